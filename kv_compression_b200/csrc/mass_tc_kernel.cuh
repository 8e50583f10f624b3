// mass_tc_kernel.cuh -- accumulated attention weights with tcgen05 tensor cores
// (bf16, d_c = 512, d_r = 64).
//
//   s[t] = decay prev[t] + sum_r 2^{(q[r] . [c_t | k_t] - lse[r]) log2 e}
//
// Work is a list of (sequence, 128-token tile, block of N query rows), row
// blocks fastest, and each CTA takes one contiguous range of it.  A step is
//   S^T[128 tokens x N rows] = [C | K]_tile . [q_c | q_r]^T     36 MMAs, M = 128, K = 16
// into one of two TMEM buffers, then eight warps add each token's weights up
// (a thread holds one token and half of the rows) while the next step's MMAs
// run.  Nothing is written per (row, token): a token's sum leaves once.
//
// One operand stays in shared memory and the other streams through a ring of
// [128][64] chunks:
//   up to 128 rows   the queries stay (N = 16 .. 128) and the cache streams: it is read
//                    once, at memory speed
//   more rows        a tile of the cache stays and the query blocks (N = 128) stream, from
//                    L2: the cache comes from memory once whatever the number of rows.
//                    Shared memory would bound this: an MMA of 64 cycles reads 8 KB of
//                    operands there (all of its 128 bytes a cycle) while 4 KB of
//                    queries arrive.  So the tile's C is copied into tensor memory
//                    (256 columns, a token's row in its lane) and is the A operand from
//                    there; K (64 of 576 dims) stays in shared memory.
// A tile whose row blocks are split over CTAs gets one partial sum from each;
// lca_mass_finish_kernel adds those in CTA order, so the result does not depend
// on timing.
//
// Roles (320 threads): warp 0 loads, warp 1 issues the MMAs, warps 2-9 add.
// Every wait is bounded, as in the tree kernel.
#pragma once
#include <cuda.h>

#include "tree_simt_kernel.cuh"
#include "tree_tc_kernel.cuh"

namespace lca {
namespace mtc {

using ttc::kChunk;
using ttc::Wait;
constexpr int kAddWarps = 8;
constexpr int kThreads = 32 * (2 + kAddWarps);
constexpr int kBarAdd = 1;
constexpr int kMaxSlots = 5;
constexpr uint32_t kColA = 256;      // the tile's C in TMEM: 32 columns for 64 dims

template <int N, bool kStream>       // kStream: the queries stream
struct Layout {
  static_assert(!kStream || N == 128, "streamed queries come 128 rows at a time");
  static constexpr int kQChunk = N * 128;
  static constexpr int kStay = kStream ? kChunk : 9 * kQChunk;             // what stays in shared memory: a tile's K, or Q
  // The ring: slots of three chunks, three of them, so that a step's slots are always the same ones; beside 128
  // rows of queries slots of one chunk.  (A load, a barrier and a release for each single chunk set the pace
  // elsewhere: 430 cycles a chunk for the loading warp, 400 for the MMA warp, where the MMAs take 256.)
  static constexpr int kPer = N == 128 && !kStream ? 1 : 3;
  static constexpr int kSlots = kPer == 1 ? 5 : 3;
  static constexpr int kSlot = kPer * kChunk;
  static constexpr int kOffRing = kStay;
  static constexpr int kOffOff = kOffRing + kSlots * kSlot;               // float [2][N] offsets of the rows
  static constexpr int kOffPart = kOffOff + 8 * N;                         // float [128]
  static constexpr int kOffGap = kOffPart + 512;                           // u32 [2][4] rows that add nothing
  static constexpr int kOffBar = kOffGap + 32;
  static constexpr int kBars = 2 * kMaxSlots + 8;
  static constexpr int kOffMisc = kOffBar + 8 * kBars;
  static constexpr int kBytes = kOffMisc + 16;
  static constexpr int kAlloc = kBytes + 1024;
  static constexpr uint32_t kCols = kStream ? 512 : N <= 16 ? 32 : N == 32 ? 64 : N == 64 ? 128 : 256;
  static_assert(kAlloc <= 232448, "shared memory of one CTA");
};

struct Split {                  // one per sequence, for the finishing kernel
  int64_t base;                 // first step
  int tiles, rb;
};

struct Params {
  CUtensorMap tm_c, tm_k;       // pools, box [64 rows][64]
  CUtensorMap tm_qc, tm_qr;     // queries as [B T H rows][..], box [N rows][64]
  MassParams m;
  int G;
  float* part;                  // [2 G][128]: a CTA's first and last tile, where it holds a share of it
  Split* split;
  uint64_t timeout_ns;
  int debug_skip_load;
};

// Where a step lies, and the step after it.
struct Step {
  int b, tile, rb;
  int tiles, rbs;               // of sequence b
};

template <int N, bool kStream>
__global__ void __launch_bounds__(kThreads, 1) lca_mass_tc_kernel(const __grid_constant__ Params p) {
  using L = Layout<N, kStream>;
  constexpr int kSlots = L::kSlots, kPer = L::kPer, kFills = 9 / kPer;   // slots filled for a step
  constexpr int C = N / 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t *full = bars, *empty = bars + kMaxSlots, *stay_full = bars + 2 * kMaxSlots, *stay_empty = stay_full + 1,
           *s_full = stay_full + 2, *s_empty = stay_full + 4, *drain = stay_full + 6, *a_full = stay_full + 7;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffMisc + 4);
  const TreeBatch& t = p.m.t;
  const Wait wt = {abort_flag, t.err, p.timeout_ns};
  const WarpLanes lanes;

  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      ptx::mbar_init(full + i, 1);
      ptx::mbar_init(empty + i, 1);
    }
    ptx::mbar_init(stay_full, 1);
    ptx::mbar_init(stay_empty, 1);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(s_full + i, 1);
      ptx::mbar_init(s_empty + i, kAddWarps);
    }
    ptx::mbar_init(drain, 1);
    ptx::mbar_init(a_full, kAddWarps);
    *abort_flag = 0;
    ptx::fence_mbarrier_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_slot, L::kCols);
    ptx::tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&p.tm_c);
    ptx::prefetch_tmap(&p.tm_k);
    ptx::prefetch_tmap(&p.tm_qc);
    ptx::prefetch_tmap(&p.tm_qr);
  }
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  // up to 32 sequences a lane keeps its own one's lengths
  const bool few = t.B <= 32;
  auto work = [&](const TreeLens& l) {
    TreeWork w = tree_work(l.n, l.d, t.H, N);
    if (l.d == 0 && l.n > 0) {        // nothing to add, but the old sums are scaled all the same
      w.rb = 1;
      w.tiles = (l.n + kTreeTile - 1) / kTreeTile;
    }
    return w;
  };
  const TreeLens own = few && lane < t.B ? tree_lens(t, lane) : TreeLens{0, 0, false};
  const TreeWork own_work = work(own);
  auto seq = [&](int b) { return few ? own_work : work(tree_lens(t, b)); };     // few: asked for b = lane only
  auto lens_of = [&](int b) {         // for a whole warp
    return few ? TreeLens{lanes.get(own.n, b), lanes.get(own.d, b), false} : tree_lens(t, b);
  };
  const int64_t U = tree_units(lanes, seq, t.B, 1);
  // CTA c of the G used (no more than there are steps): steps [c U / G, (c + 1) U / G)
  const int64_t G = U < p.G ? U : p.G, c0 = blockIdx.x;
  const int64_t u0 = c0 < G ? c0 * U / G : 0, u1 = c0 < G ? (c0 + 1) * U / G : 0;
  Step st0 = {0, 0, 0, 1, 1};
  if (u0 < u1) {
    const TreeUnit x = tree_unit<int64_t>(lanes, seq, t.B, 1, u0);
    const TreeWork w = work(lens_of(x.b));
    st0 = Step{x.b, x.t0, x.rb, w.tiles, w.rb};
  }
  auto next = [&](Step& s) {
    if (++s.rb < s.rbs) return;
    s.rb = 0;
    if (++s.tile < s.tiles) return;
    s.tile = 0;
    s.tiles = 0;
    while (s.tiles == 0 && ++s.b < t.B) {
      const TreeWork w = work(lens_of(s.b));
      s.tiles = w.tiles;
      s.rbs = w.rb;
    }
  };
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    // Converged, with one elected lane; a step's rows are looked up a step ahead.
    int ns = 0, slot = 0, use = 0, sent = 0;
    bool ok = true, skip = p.debug_skip_load != 0;
    Step s = st0;
    int last_b = -1, last_tile = -1;
    int r0 = 0, r1 = 0;
    auto rows_of = [&](const Step& x, int& a, int& b) {
      const TreeLens l = lens_of(x.b);
      const int pos = x.tile * kTreeTile;
      a = (int)tree_row(t, x.b, pos, 0xB06);
      b = pos + 64 < l.n + l.d ? (int)tree_row(t, x.b, pos + 64, 0xB06) : a;
    };
    if (u0 < u1) rows_of(s, r0, r1);
    for (int64_t u = u0; u < u1 && ok; ++u) {
      const int b = s.b, tile = s.tile;
      const int qrow = (int)((int64_t)s.b * t.T * t.H + (int64_t)s.rb * N);
      int n0 = r0, n1 = r1;
      next(s);
      if (u + 1 < u1 && (s.b != b || s.tile != tile)) rows_of(s, n0, n1);
      auto load_tile = [&](uint8_t* dst, int c, uint64_t* bar) {
        const CUtensorMap* map = c < 8 ? &p.tm_c : &p.tm_k;
        const int x = c < 8 ? 64 * c : 0;
        ptx::tma_load_2d(dst, map, x, r0, bar);
        ptx::tma_load_2d(dst + kChunk / 2, map, x, r1, bar);
      };
      auto load_q = [&](uint8_t* dst, int c, uint64_t* bar) {
        ptx::tma_load_2d(dst, c < 8 ? &p.tm_qc : &p.tm_qr, c < 8 ? 64 * c : 0, qrow, bar);
      };
      // chunks kPer f .. of the tile (up to `count`) or of the queries into the ring
      auto fill = [&](bool tiles, int f, int count) {
        if (use > 0) ok = ttc::warp_wait(empty + slot, (use - 1) & 1, wt, 0xC41);
        if (!ok) return;
        if (!skip && ptx::elect_one()) {
          ptx::mbar_arrive_expect_tx(full + slot, min(kPer, count - kPer * f) * kChunk);
          uint8_t* dst = smem + L::kOffRing + slot * L::kSlot;
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            const int c = kPer * f + k;
            if (c >= count || !LCA_CHECK(t.err, slot < kSlots && c < 9, 0xD60)) break;
            if (tiles) load_tile(dst + k * kChunk, c, full + slot);
            else load_q(dst + k * kChunk, c, full + slot);
          }
        }
        __syncwarp();
        if (!skip && use == 0) sent |= 1 << slot;
        skip = false;
        if (++slot == kSlots) {
          slot = 0;
          ++use;
        }
      };
      if (b != last_b || (kStream && tile != last_tile)) {
        last_b = b;
        last_tile = tile;
        if constexpr (kStream) {
#pragma unroll 1
          for (int f = 0; f < kFills && ok; ++f) fill(true, f, 8);       // on its way to TMEM
        }
        if (ok && ns > 0) ok = ttc::warp_wait(stay_empty, (ns - 1) & 1, wt, 0xC40);
        if (!ok) break;
        if (ptx::elect_one()) {
          ptx::mbar_arrive_expect_tx(stay_full, L::kStay);
          if constexpr (kStream) {
            load_tile(smem, 8, stay_full);
          } else {
#pragma unroll
            for (int c = 0; c < 9; ++c) load_q(smem + c * L::kQChunk, c, stay_full);
          }
        }
        __syncwarp();
        ++ns;
      }
#pragma unroll 1
      for (int f = 0; f < kFills && ok; ++f) fill(!kStream, f, 9);
      r0 = n0;
      r1 = n1;
    }
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const int fills = use + (i < slot ? 1 : 0);
      if (fills > 1 || (fills == 1 && ((sent >> i) & 1))) ttc::wait(full + i, (fills - 1) & 1, wt, 0xC4F, false);
    }
    if (ns > 0) ttc::wait(stay_full, (ns - 1) & 1, wt, 0xC4F, false);
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMAs
    // The whole warp runs this and one elected lane issues; the next chunk's barrier is probed
    // before the MMAs of the chunk at hand (as in the tree kernel).
    constexpr uint32_t kId = ptx::idesc_bf16_f32(128, N, 0, 0);
    const uint64_t d_stay = ptx::smem_desc(ptx::smem_u32(smem), 16, 1024, ptx::kSwizzle128B);
    const uint64_t d_ring = ptx::smem_desc(ptx::smem_u32(smem + L::kOffRing), 16, 1024, ptx::kSwizzle128B);
    int64_t i = 0;
    int ns = 0, slot = 0, ph = 0;
    bool ok = true, ready = false;
    Step s = st0;
    int last_b = -1, last_tile = -1;
    for (int64_t u = u0; u < u1 && ok; ++u, ++i) {
      if (s.b != last_b || (kStream && s.tile != last_tile)) {
        last_b = s.b;
        last_tile = s.tile;
        ok = ttc::warp_wait(stay_full, ns & 1, wt, 0xC42);
        if constexpr (kStream) {                       // a round of the ring went to TMEM
          ok = ok && ttc::warp_wait(a_full, ns & 1, wt, 0xC46);
          ready = false;
          ph ^= 1;
        }
        ++ns;
      }
      const int b = s.b, tile = s.tile;
      next(s);
      const bool leaves = u + 1 < u1 && (s.b != b || (kStream && s.tile != tile));   // the operand that stays does not
      const int buf = (int)(i & 1);
      if (i >= 2) ok = ttc::warp_wait(s_empty + buf, (uint32_t)((i >> 1) - 1) & 1, wt, 0xC43) && ok;
#pragma unroll
      for (int f = 0; f < kFills; ++f) {
        const int at = kSlots == kFills ? f : slot;
        if (!__all_sync(0xffffffffu, ready)) ok = ttc::warp_wait(full + at, ph, wt, 0xC44) && ok;
        ptx::tc_fence_after();
        const int ahead = at + 1 == kSlots ? 0 : at + 1, aph = at + 1 == kSlots ? ph ^ 1 : ph;
        ready = ptx::mbar_test_wait(full + ahead, aph);
        if (!ok) break;
        if (ptx::elect_one()) {
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            const int c = kPer * f + j;
            const uint64_t r = d_ring + (uint64_t)((at * L::kSlot + j * kChunk) >> 4);
            const uint64_t q = d_stay + (uint64_t)((kStream ? 0 : c * L::kQChunk) >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint64_t o = (uint64_t)((32 * k) >> 4);
              if constexpr (!kStream) ptx::mma_bf16_ss(tmem + N * buf, r + o, q + o, kId, (c | k) != 0);
              else if (c < 8) ptx::mma_bf16_ts(tmem + N * buf, tmem + kColA + 32 * c + 8 * k, r + o, kId, (c | k) != 0);
              else ptx::mma_bf16_ss(tmem + N * buf, q + o, r + o, kId, 1u);
            }
          }
          ptx::mma_commit(empty + at);
          if (f == kFills - 1) {
            ptx::mma_commit(s_full + buf);
            if (leaves) ptx::mma_commit(stay_empty);
          }
        }
        __syncwarp();
        slot = ahead;
        ph = aph;
      }
    }
    if (ptx::elect_one()) ptx::mma_commit(drain);
    ttc::wait(drain, 0, wt, 0xC4E, false);
  } else {
    // ---------------------------------------------------------------- sums
    const int sw = warp - 2, sid = tid - 64;
    const int quarter = warp & 3, half = sw >> 2;
    const int tok = 32 * quarter + lane;
    const uint32_t addr = tmem + ((uint32_t)(32 * quarter) << 16) + C * half;
    float* off = reinterpret_cast<float*>(smem + L::kOffOff);
    float* part = reinterpret_cast<float*>(smem + L::kOffPart);
    uint32_t* gap = reinterpret_cast<uint32_t*>(smem + L::kOffGap);
    if (blockIdx.x == 0 && sw == 7) {
      int64_t base = 0;
      for (int b0 = 0; b0 < t.B; b0 += 32) {
        const int b = b0 + lane;
        TreeWork k = {0, 0};
        if (b < t.B) {
          k = seq(b);
          if (tree_lens(t, b).bad) input_error(t.err, 0xB03);
        }
        const int64_t mine = (int64_t)k.rb * k.tiles, incl = base + lanes.scan(mine);
        if (b < t.B) p.split[b] = Split{incl - mine, k.tiles, k.rb};
        base = lanes.get(incl, 31);
      }
    }
    Step s = st0;
    int64_t i = 0;
    int segment = 0;
    bool from_start = s.rb == 0, fresh = true;
    float acc = 0.f;
    TreeLens l = lens_of(s.b);
    // a row's -lse; rows that add nothing have -inf.  Read a step ahead.
    auto offset = [&](const Step& at, int d) {
      const int r = at.rb * N + sid;
      return sid < N && r < d * t.H ? mass_offset(p.m.lse[(int64_t)at.b * t.T * t.H + r]) : -INFINITY;
    };
    float o_next = u0 < u1 ? offset(s, l.d) : -INFINITY;
    unsigned long long vis = ~0ull;                    // the nodes that see this thread's token
    int64_t rounds = 0;                                // of the ring
    for (int64_t u = u0; u < u1; ++u, ++i) {
      const int buf = (int)(i & 1);
      bool live = true;
      if constexpr (kStream) {
        if (fresh) {
          // the tile's C from a round of the ring into TMEM, every other chunk by each half of the warps; the MMAs
          // that read the last one are done (their last step has been added up)
#pragma unroll 1
          for (int f = 0; f < kFills; ++f) {
            live = ttc::warp_wait(full + f, (uint32_t)rounds & 1, wt, 0xC47) && live;
#pragma unroll 1
            for (int c = kPer * f; c < min(8, kPer * f + kPer); ++c) {
              if ((c & 1) != half) continue;
              const uint8_t* from = smem + L::kOffRing + c * kChunk + tok * 128;
              float v[32];
#pragma unroll
              for (int j = 0; j < 8; ++j) {            // the 16-byte units of a row are swizzled by its number
                const float4 w = *reinterpret_cast<const float4*>(from + ((j ^ (tok & 7)) << 4));
                v[4 * j] = w.x; v[4 * j + 1] = w.y; v[4 * j + 2] = w.z; v[4 * j + 3] = w.w;
              }
              ptx::tmem_st32(tmem + ((uint32_t)(32 * quarter) << 16) + kColA + 32 * c, v);
            }
            ptx::named_bar_sync(kBarAdd, 32 * kAddWarps);          // the slot is read
            if (sid == 0 && live) ptx::mbar_arrive(empty + f);     // (not after an error: nothing is loaded any more)
          }
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(a_full);
          ++rounds;
        }
        ++rounds;
      }
      const int pos0 = s.tile * kTreeTile;
      const bool special = pos0 + kTreeTile > l.n;     // drafted tokens, or the end, in this tile
      if (sid < N) off[buf * N + sid] = o_next;
      const uint32_t empty_rows = __ballot_sync(0xffffffffu, o_next == -INFINITY);
      if (sid < N && lane == 0) gap[4 * buf + sw] = empty_rows;
      const Step at = s;
      const TreeLens lat = l;
      next(s);
      if (u + 1 < u1) {
        if (s.b != at.b) l = lens_of(s.b);
        o_next = offset(s, l.d);
      }
      if (fresh && special) {
        const int node = pos0 + tok - lat.n;
        vis = node < 0 ? ~0ull : 0ull;
        if (node >= 0 && node < lat.d)
          for (int j = 0; j < lat.d; ++j) vis |= ((tree_word(t, at.b, j) >> node) & 1ull) << j;
      }
      fresh = false;
      live = ttc::warp_wait(s_full + buf, (uint32_t)(i >> 1) & 1, wt, 0xC45) && live;
      if (ptx::named_bar_or(kBarAdd, 32 * kAddWarps, !live)) break;
      ptx::tc_fence_after();
      float a0 = 0.f, a1 = 0.f;
      constexpr int W = C < 32 ? C : 32;
#pragma unroll
      for (int c0 = 0; c0 < C; c0 += W) {
        float x[W];
        ttc::tmem_load<W>(addr + N * buf + c0, x);
        ptx::tmem_wait_ld();
        const int col0 = C * half + c0;
        const float* o = off + buf * N + col0;
        const uint32_t all = W == 32 ? ~0u : (1u << (W & 31)) - 1u;
        if (!LCA_CHECK(t.err, col0 >= 0 && col0 + W <= N && buf < 2, 0xD62)) break;
        const uint32_t gaps = (gap[4 * buf + col0 / 32] >> (col0 % 32)) & all;
        if (special || gaps != 0u) {
          // the rows of these that see this thread's token, and are there; the others' logits become -inf
          // (rows of nodes from 64 on, in a last block that is not full, are gaps)
          uint32_t sees = ~gaps;
          if (special) {
            int node = (at.rb * N + col0) / t.H, left = t.H - (at.rb * N + col0 - node * t.H);
            for (int c = 0; c < W; ++node, left = t.H) {
              const int n = min(left, W - c);
              if (!((vis >> (node & 63)) & 1ull)) sees &= ~((n == 32 ? ~0u : (1u << n) - 1u) << c);
              c += n;
            }
          }
#pragma unroll
          for (int c = 0; c < W; ++c) x[c] = (sees >> c) & 1u ? x[c] : -INFINITY;
        }
        const uint64_t log2e = ptx::f32x2(kTreeLog2e, kTreeLog2e), scale = ptx::f32x2(ttc::kLogitScale, ttc::kLogitScale);
#pragma unroll
        for (int c = 0; c < W; c += 4) {
          const float4 o4 = *reinterpret_cast<const float4*>(o + c);
          float e0, e1, e2, e3;
          ptx::f32x2_split(ptx::mul_f32x2(ptx::fma_f32x2(ptx::f32x2(x[c], x[c + 1]), scale, ptx::f32x2(o4.x, o4.y)), log2e), e0, e1);
          ptx::f32x2_split(ptx::mul_f32x2(ptx::fma_f32x2(ptx::f32x2(x[c + 2], x[c + 3]), scale, ptx::f32x2(o4.z, o4.w)), log2e), e2, e3);
          a0 += ttc::ex2(e0);
          a1 += ttc::ex2(e1);
          a0 += ttc::ex2(e2);
          a1 += ttc::ex2(e3);
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(s_empty + buf);
      acc += a0 + a1;
      if (u + 1 == u1 || s.tile != at.tile || s.b != at.b) {
        // the end of this CTA's share of a tile
        if (half == 1) part[tok] = acc;
        ptx::named_bar_sync(kBarAdd, 32 * kAddWarps);
        if (half == 0) {
          const float sum = acc + part[tok];
          if (from_start && at.rb + 1 == at.rbs) {
            if (pos0 + tok < lat.n + lat.d) mass_store(p.m, at.b, pos0 + tok, lat.n, sum);
          } else if (LCA_CHECK(t.err, (int)blockIdx.x < p.G, 0xD61)) {
            p.part[(2 * (int64_t)blockIdx.x + (segment > 0 ? 1 : 0)) * kTreeTile + tok] = sum;
          }
        }
        acc = 0.f;
        vis = ~0ull;
        ++segment;
        from_start = fresh = true;
      }
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc(tmem, L::kCols);
}

struct FinishParams {
  MassParams m;
  int G;
  const float* part;
  const Split* split;
};

// The tiles that more than one CTA had a share of: their shares added in CTA
// order.  grid (blocks, B), a thread per token.
__global__ void __launch_bounds__(kTreeTile) lca_mass_finish_kernel(const FinishParams p) {
  ptx::griddep_wait();
  const int b = blockIdx.y, tok = threadIdx.x;
  const Split sp = p.split[b], last = p.split[p.m.t.B - 1];
  const int64_t U = last.base + (int64_t)last.tiles * last.rb;
  const int64_t G = U < p.G ? U : p.G;
  const TreeLens l = tree_lens(p.m.t, b);
  for (int tile = blockIdx.x; tile < sp.tiles; tile += gridDim.x) {
    const int64_t u = sp.base + (int64_t)tile * sp.rb;
    const int64_t lo = ((u + 1) * G - 1) / U, hi = ((u + sp.rb) * G - 1) / U;   // the CTAs of its first and last step
    if (lo == hi || !LCA_CHECK(p.m.t.err, lo >= 0 && hi < p.G, 0xD63)) continue;
    float sum = 0.f;
    for (int64_t c = lo; c <= hi; ++c) sum += p.part[(2 * c + (c * U / G < u ? 1 : 0)) * kTreeTile + tok];
    const int pos = tile * kTreeTile + tok;
    if (pos < l.n + l.d) mass_store(p.m, b, pos, l.n, sum);
  }
}

}  // namespace mtc
}  // namespace lca
