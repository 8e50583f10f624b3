// tree_schedule.cuh -- how a ragged batch of draft trees is cut into work for
// CTAs.  Plain arithmetic, written once for a warp (its lanes share the
// sequences) and for one thread of the host (tests).
//
// Sequence b has rb_b blocks of N query rows and tiles_b tiles of 128 tokens.
// Its tokens are cut into parts_b = ceil(tiles_b / S) parts of nearly equal
// length (S tiles at most), and a unit is (sequence, part, row block), row
// blocks fastest: units that read the same tokens run next to each other, so
// that a tile comes from HBM once and from L2 for the other row blocks.  Unit u
// goes to CTA u mod G, and its partial to slot u.
//
// S is chosen for the time of the longest CTA: k units one after another take
// about k (S + c) tile times, c for a unit's fixed costs (query block, pipeline
// fill, partial or output).  For each k up to kTreeMaxWaves the least S with
// units(S) <= k G is found and the best k taken; where even unsplit sequences
// make more units than that, none is split (and no slot is used).
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define LCA_HD __host__ __device__ __forceinline__
#else
#define LCA_HD inline
#endif

namespace lca {

constexpr int kTreeTile = 128;        // tokens
constexpr int kTreeMaxWaves = 4;
constexpr int kTreeUnitCost = 2;      // c, in tile times

struct TreeWork {                     // one sequence's
  int rb, tiles;
};

LCA_HD TreeWork tree_work(int n, int d, int H, int N) {
  TreeWork w;
  w.rb = (d * H + N - 1) / N;
  w.tiles = d > 0 ? (int)(((int64_t)n + d + kTreeTile - 1) / kTreeTile) : 0;
  return w;
}

struct TreeUnit {
  int b;                              // -1: there is no such unit
  int rb, part, parts;
  int t0, t1;                         // tiles
};

// First tile of part `part` of `parts` over `tiles`: the first parts have one more where it does not come out even.
LCA_HD int tree_cut(int tiles, int part, int parts) {
  const int each = tiles / parts, more = tiles - each * parts;
  return each * part + (part < more ? part : more);
}

// Units for parts of at most S tiles.  Lanes: lane() of count(), sum(), scan() (inclusive), first() (the lowest
// lane where true, -1: none), get() (a lane's value).
template <class Lanes, class Seq>
LCA_HD int64_t tree_units(const Lanes& w, const Seq& seq, int B, int S) {
  int64_t c = 0;
  for (int b = w.lane(); b < B; b += w.count()) {
    const TreeWork k = seq(b);
    c += (int64_t)k.rb * ((k.tiles + S - 1) / S);
  }
  return w.sum(c);
}

// The least S in [1, most] with units(S) <= limit; most + 1 if there is none.
template <class Lanes, class Seq>
LCA_HD int tree_least(const Lanes& w, const Seq& seq, int B, int most, int64_t limit) {
  if (tree_units(w, seq, B, most) > limit) return most + 1;
  int lo = 1, hi = most;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (tree_units(w, seq, B, mid) <= limit) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// The same for up to count() sequences, lane b with sequence b's work: every lane tries a length of its own, so
// a few rounds do.
template <class Lanes>
LCA_HD int tree_least_few(const Lanes& w, const TreeWork& own, int B, int most, int64_t limit) {
  int lo = 1, hi = most + 1;                   // the answer lies in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + w.count() - 1) / w.count();
    const int S = lo + w.lane() * step < hi ? lo + w.lane() * step : hi;     // hi: known to do (or none does)
    int64_t units = 0;
    for (int b = 0; b < B; ++b) {
      const int rb = w.get(own.rb, b), tiles = w.get(own.tiles, b);
      units += (int64_t)rb * (S <= most ? (tiles + S - 1) / S : 1);
    }
    const int at = w.first(S >= hi || units <= limit);
    if (at < 0) {                              // none tried does: it lies above the last one
      lo = lo + (w.count() - 1) * step + 1;
    } else {
      const int found = lo + at * step < hi ? lo + at * step : hi;
      lo = at == 0 ? found : lo + (at - 1) * step + 1;
      hi = found;
    }
  }
  return lo;
}

// The cost of k waves with their least S (INT64_MAX: not possible).
LCA_HD int64_t tree_cost(int k, int S, int most) {
  return S > most ? INT64_MAX : (int64_t)k * (S + kTreeUnitCost);
}

// A place in the units' order: the batch of count() sequences looked at last, of which each lane keeps its own one.
// A CTA's units follow one another, so each search goes on from the last (from the start every time, 4096
// sequences of 256 tokens took 1320 us for 600).
template <class I>
struct TreeCursor {
  int b0 = -1;                        // first sequence; -1: none looked at
  I end = 0;                          // units up to the batch's end
  I incl;                             // up to this lane's sequence's end
  TreeWork k;
  int parts;
};

// Unit u, not below the one that the cursor was used for last.  I holds the number of units.
template <class I, class Lanes, class Seq>
LCA_HD TreeUnit tree_unit(const Lanes& w, const Seq& seq, int B, int S, I u, TreeCursor<I>& at) {
  while (at.b0 < 0 || u >= at.end) {
    const int b0 = at.b0 < 0 ? 0 : at.b0 + w.count();
    if (b0 >= B) return TreeUnit{-1, 0, 0, 0, 0, 0};
    at.k = b0 + w.lane() < B ? seq(b0 + w.lane()) : TreeWork{0, 0};
    at.parts = (at.k.tiles + S - 1) / S;
    at.incl = at.end + w.scan((I)at.k.rb * at.parts);
    at.end = w.get(at.incl, w.count() - 1);
    at.b0 = b0;
  }
  const int lane = w.first(at.incl > u);
  TreeUnit r;
  r.b = at.b0 + lane;
  const int rb = w.get(at.k.rb, lane), tiles = w.get(at.k.tiles, lane);
  r.parts = w.get(at.parts, lane);
  const int i = (int)(u - (w.get(at.incl, lane) - (I)rb * r.parts));
  r.part = i / rb;
  r.rb = i - r.part * rb;
  r.t0 = tree_cut(tiles, r.part, r.parts);
  r.t1 = tree_cut(tiles, r.part + 1, r.parts);
  return r;
}
template <class I, class Lanes, class Seq>
LCA_HD TreeUnit tree_unit(const Lanes& w, const Seq& seq, int B, int S, I u) {
  TreeCursor<I> at;
  return tree_unit<I>(w, seq, B, S, u, at);
}

#ifdef __CUDACC__
struct WarpLanes {
  __device__ __forceinline__ int lane() const { return threadIdx.x & 31; }
  __device__ __forceinline__ int count() const { return 32; }
  __device__ __forceinline__ int64_t sum(int64_t v) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  template <class I>
  __device__ __forceinline__ I scan(I v) const {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const I x = __shfl_up_sync(0xffffffffu, v, o);
      if (lane() >= o) v += x;
    }
    return v;
  }
  __device__ __forceinline__ int first(bool p) const { return __ffs(__ballot_sync(0xffffffffu, p)) - 1; }
  __device__ __forceinline__ int get(int v, int from) const { return __shfl_sync(0xffffffffu, v, from); }
  __device__ __forceinline__ int64_t get(int64_t v, int from) const { return __shfl_sync(0xffffffffu, v, from); }
};
#endif

}  // namespace lca
