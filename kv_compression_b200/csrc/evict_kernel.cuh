// evict_kernel.cuh -- which rows an eviction keeps, and moving kept rows to the
// front of their sequence.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"
#include "tree_common.cuh"

namespace lca {

// ---------------------------------------------------------------- choice
// Of a sequence's n rows, `budget` stay: the first n_sink, the last n_recent,
// and of the rows between those with the largest sums, the lower row first
// where sums are equal.  A sum that is not a number counts as the smallest.
// All rows stay where n <= budget.  The kept rows are written in rising order.
//
// The sums map to unsigned keys of the same order.  A sequence belongs to a
// cluster of CTAs, each with a contiguous run of its rows, whose keys it reads
// once and keeps in shared memory.  The key of the last row kept is found 11, 11
// and 10 bits at a time: a histogram per CTA of the keys that share the bits
// found so far, added up over the cluster by every CTA for itself.  Then each
// warp counts the kept rows of its run, the counts before it (its CTA's, and
// the lower CTAs' totals) say where its rows go, and it writes them in order.
// What bounds it is latency: five cluster barriers and three histograms.
struct SelectParams {
  const float* scores;          // [B][stride]
  int64_t stride;
  const int32_t* seq_lens;      // [B]
  int B;
  int64_t cap;                  // the longest valid length
  int n_sink, n_recent;
  int budget;                   // entries a row of `kept` has
  int32_t* kept;                // [B][budget]
  int32_t* kept_lens;           // [B]
  int ctas;                     // of a cluster, which takes one sequence
  int* err;
};

__device__ __forceinline__ uint32_t select_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);                  // -0 counts as 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kSelectBins = 2048;
constexpr int kSelectKeep = 40960;          // keys of a CTA in shared memory; later ones are read again
constexpr int kSelectMaxCtas = 8;

__host__ __device__ inline size_t select_smem(int64_t run) {
  const int64_t keys = run < kSelectKeep ? run : kSelectKeep;
  return sizeof(int) * (3 * kSelectBins + (size_t)keys);
}

// Rows a CTA of `ctas` takes of n: a multiple of 32 x warps, so that every warp's run starts on a 128-byte line.
__host__ __device__ inline int64_t select_run(int64_t n, int ctas) {
  const int64_t per = (n + ctas - 1) / ctas;
  return (per + kSelectThreads - 1) / kSelectThreads * kSelectThreads;
}

__device__ __forceinline__ int ld_cluster(const int* p, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(ptx::mapa(ptx::smem_u32(p), rank)) : "memory");
  return v;
}

__device__ __forceinline__ int4 ld_cluster4(const int* p, uint32_t rank) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(ptx::mapa(ptx::smem_u32(p), rank))
               : "memory");
  return v;
}
// The sum of the warps' values below `warp`.
__device__ __forceinline__ int warp_prefix(const int* sums, int warp, int lane) {
  int v = lane < warp ? sums[lane] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__global__ void __launch_bounds__(kSelectThreads) lca_select_kernel(const SelectParams p) {
  extern __shared__ int select_dyn[];
  int* hist = select_dyn;                                       // [3][2048]
  uint32_t* keys = reinterpret_cast<uint32_t*>(select_dyn + 3 * kSelectBins);
  __shared__ int warp_sum[kSelectWarps], warp_eq[kSelectWarps];
  __shared__ int s_bin, s_above;
  __shared__ int totals[2];                                     // rows kept for sure, rows of the last key
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = p.ctas, rank = blockIdx.x % ctas, b = blockIdx.x / ctas;
  const int n = p.seq_lens[b];
  int32_t* kept = p.kept + (int64_t)b * p.budget;
  if (n < 0 || n > p.cap) {
    if (rank == 0 && tid == 0) {
      input_error(p.err, 0xB10);
      p.kept_lens[b] = 0;
    }
    return;
  }
  if (rank == 0 && tid == 0) p.kept_lens[b] = min(n, p.budget);
  if (n <= p.budget) {
    for (int i = rank * kSelectThreads + tid; i < n; i += ctas * kSelectThreads) kept[i] = i;
    return;
  }
  const float* x = p.scores + (int64_t)b * p.stride;
  const int run = (int)select_run(n, ctas);                     // this CTA: rows [r0, r1)
  const int r0 = (int)min((int64_t)n, (int64_t)rank * run), r1 = min(n, r0 + run);
  const int lo = p.n_sink, hi = n - p.n_recent;                 // rows that compete
  auto key_of = [&](int i) { return i - r0 < kSelectKeep ? keys[i - r0] : select_key(x[i]); };
  for (int i = tid; i < 3 * kSelectBins; i += kSelectThreads) hist[i] = 0;
  __syncthreads();
  int need = p.budget - p.n_sink - p.n_recent;                  // rows to take of [lo, hi)
  const bool any = need > 0;
  uint32_t prefix = 0, have = 0;                                // bits of the last key found; their mask
  constexpr int kShift[3] = {21, 10, 0}, kBits[3] = {11, 11, 10};
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    int* h = hist + pass * kSelectBins;
    constexpr int kUnroll = 16;
    for (int i0 = r0; i0 < r1; i0 += kUnroll * kSelectThreads) {
      uint32_t k[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = i0 + u * kSelectThreads + tid;
        k[u] = 0;
        if (i < r1) k[u] = pass == 0 ? select_key(x[i]) : key_of(i);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = i0 + u * kSelectThreads + tid;
        if (i >= r1) continue;
        if (pass == 0 && i - r0 < kSelectKeep) keys[i - r0] = k[u];
        if (i >= lo && i < hi && (k[u] & have) == prefix) atomicAdd(&h[(k[u] >> kShift[pass]) & ((1u << kBits[pass]) - 1u)], 1);
      }
    }
    ptx::cluster_sync();                                        // (also the CTA's own barrier)
    if (any) {
      // thread t < 512 has the four bins from 2047 - 4t down; their counts over the cluster, scanned from the top
      int4 c = make_int4(0, 0, 0, 0);                           // .w the highest bin
      const int bin0 = kSelectBins - 4 - 4 * tid;
      if (tid < kSelectBins / 4) {
        int4 v[kSelectMaxCtas];
#pragma unroll
        for (int r = 0; r < kSelectMaxCtas; ++r) v[r] = r < ctas ? ld_cluster4(h + bin0, r) : make_int4(0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < kSelectMaxCtas; ++r) {
          c.x += v[r].x; c.y += v[r].y; c.z += v[r].z; c.w += v[r].w;
        }
      }
      int incl = c.x + c.y + c.z + c.w;
      const int mine = incl;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) warp_sum[warp] = incl;
      __syncthreads();
      int above = warp_prefix(warp_sum, warp, lane) + incl - mine;      // rows in higher bins
      const int count[4] = {c.w, c.z, c.y, c.x};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (above < need && need <= above + count[q]) {
          s_bin = bin0 + 3 - q;
          s_above = above;
        }
        above += count[q];
      }
      __syncthreads();
      prefix |= (uint32_t)s_bin << kShift[pass];
      have |= ((1u << kBits[pass]) - 1u) << kShift[pass];
      need -= s_above;
    }
  }
  // a warp's rows: kept for sure (by place, or by a larger key), or of the last key
  const int per_warp = run / kSelectWarps;
  const int w0 = min(r1, r0 + warp * per_warp), w1 = min(r1, w0 + per_warp);
  auto judge = [&](int i, bool& sure, bool& eq) {
    sure = eq = false;
    if (i >= w1) return;
    if (i < lo || i >= hi) {
      sure = true;
    } else if (any) {
      const uint32_t k = key_of(i);
      sure = k > prefix;
      eq = k == prefix;
    }
  };
  // lane j keeps the votes on the warp's j-th 32 rows (a warp of more than 1024 rows votes twice)
  const bool votes_kept = per_warp <= 1024;
  uint32_t my_sure = 0, my_eq = 0;
  int n_sure = 0, n_eq = 0;
  for (int i0 = w0, j = 0; i0 < w1; i0 += 32, ++j) {
    bool sure, eq;
    judge(i0 + lane, sure, eq);
    const uint32_t sb = __ballot_sync(0xffffffffu, sure), eb = __ballot_sync(0xffffffffu, eq);
    if (lane == j) {
      my_sure = sb;
      my_eq = eb;
    }
    n_sure += __popc(sb);
    n_eq += __popc(eb);
  }
  if (lane == 0) {
    warp_sum[warp] = n_sure;
    warp_eq[warp] = n_eq;
  }
  __syncthreads();
  if (warp == 0) {
    int s = warp_sum[lane], e = warp_eq[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      e += __shfl_xor_sync(0xffffffffu, e, o);
    }
    if (lane == 0) {
      totals[0] = s;
      totals[1] = e;
    }
  }
  ptx::cluster_sync();
  int sure_before = warp_prefix(warp_sum, warp, lane), eq_before = warp_prefix(warp_eq, warp, lane);
#pragma unroll
  for (int r = 0; r < kSelectMaxCtas - 1; ++r)
    if (r < rank) {
      sure_before += ld_cluster(totals, r);
      eq_before += ld_cluster(totals + 1, r);
    }
  for (int i0 = w0, j = 0; i0 < w1; i0 += 32, ++j) {
    uint32_t sb, eb;
    if (votes_kept) {
      sb = __shfl_sync(0xffffffffu, my_sure, j);
      eb = __shfl_sync(0xffffffffu, my_eq, j);
    } else {
      bool sure, eq;
      judge(i0 + lane, sure, eq);
      sb = __ballot_sync(0xffffffffu, sure);
      eb = __ballot_sync(0xffffffffu, eq);
    }
    const uint32_t below = (1u << lane) - 1u;
    // of the rows with the last key the first `need` stay
    const int eq_rank = eq_before + __popc(eb & below);
    const int at = sure_before + __popc(sb & below) + min(eq_rank, need);
    if (((sb >> lane) & 1u) || (((eb >> lane) & 1u) && eq_rank < need)) kept[at] = i0 + lane;
    sure_before += __popc(sb);
    eq_before += __popc(eb);
  }
  ptx::cluster_sync();                                          // no CTA leaves while its counts may be read
}

// ---------------------------------------------------------------- moving rows
// Row dst0 + j of a sequence becomes its row src[j], j = 0 .. m - 1, in place;
// src rises strictly and src[j] >= dst0 + j.  A block moves one strip of columns
// (2, 4 or 8 times 16 bytes) of one sequence, tile after tile of rows in order.
// No row is overwritten before it is read: the rows of a tile are in registers
// of the whole block before any of them is written, later tiles read only rows
// above all those written so far (src[j] >= dst0 + j), and strips do not meet.
// For the same reason the next tile's reads may be under way while this tile is
// written, so two tiles (16 reads of 16 bytes a thread) are in flight.
//
// It is bound by memory latency and then bandwidth: a strip is as wide as
// leaves about one block per SM (narrower ones cost DRAM and L2 efficiency, wider
// ones leave SMs idle).  Rows at their place already (src[j] = dst0 + j, the
// first ones, since src[j] - j never falls) are passed over.
struct CompactParams {
  TreeBatch t;                  // the cache; lengths and masks unused
  int elem;                     // bytes of an element
  const int32_t* src;           // [B][src_stride]
  int64_t src_stride;
  const int32_t* n_src;         // [B]
  const int32_t* dst0;          // [B]; null: 0
  float* scores;                // [B][score_stride]; null: none
  int64_t score_stride;
  int strip;                    // 16-byte columns of a block
  int strips_c, strips_k;       // blocks for a row of c, of k; one more for the scores
};

// The pool row of position `pos`, -1 where its table entry is out of range (the row is then left alone).
__device__ __forceinline__ int64_t compact_row(const TreeBatch& t, int b, int pos) {
  if (!t.table) return (int64_t)b * t.page_size + pos;
  const uint32_t ps = (uint32_t)t.page_size, i = (uint32_t)pos / ps;
  const int64_t page = t.table[(int64_t)b * t.max_pages + i];
  if (page < 0 || page >= t.num_pages) {
    input_error(t.err, 0xB22);
    return -1;
  }
  return page * t.page_size + ((uint32_t)pos - i * ps);
}

constexpr int kCompactThreads = 256;
constexpr int kCompactUnroll = 8;
constexpr int kCompactMaxStrip = 8, kCompactMinStrip = 2;

__global__ void __launch_bounds__(kCompactThreads) lca_compact_kernel(const CompactParams p) {
  const TreeBatch& t = p.t;
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  const int m = p.n_src[b];
  const int d0 = p.dst0 ? p.dst0[b] : 0;
  if (m < 0 || m > p.src_stride || d0 < 0 || (int64_t)d0 + m > t.cap) {
    if (blockIdx.x == 0 && tid == 0) input_error(t.err, 0xB20);
    return;
  }
  const int32_t* src = p.src + (int64_t)b * p.src_stride;
  // rows at their place: the first j with src[j] != dst0 + j, 32 probes at a time
  int first = 0;
  for (int span = m; span > 0;) {
    const int step = (span + 31) / 32, j = first + lane * step;
    const bool moved = j >= first + span || src[j] != d0 + j;
    const uint32_t vote = __ballot_sync(0xffffffffu, moved);
    const int hit = vote ? __ffs(vote) - 1 : 32;               // probes before it are at their place
    if (hit == 0) break;
    const int end = first + span;
    first += (hit - 1) * step + 1;
    span = min(step - 1, end - first);
  }
  // row j of the list: where it is and where it goes; -1 where it stays put
  auto check = [&](int j, int& s) {
    s = src[j];
    const bool ok = s >= d0 + j && s < t.cap && (j == 0 || s > src[j - 1]);
    if (!ok) input_error(t.err, 0xB21);
    return ok;
  };
  int sx = blockIdx.x;
  if (sx >= p.strips_c + p.strips_k) {
    float* sc = p.scores + (int64_t)b * p.score_stride;
    for (int j0 = first; j0 < m; j0 += kCompactThreads * kCompactUnroll) {
      float v[kCompactUnroll];
      bool ok[kCompactUnroll];
#pragma unroll
      for (int u = 0; u < kCompactUnroll; ++u) {
        const int j = j0 + u * kCompactThreads + tid;
        int s = 0;
        ok[u] = j < m && check(j, s);
        v[u] = ok[u] ? sc[s] : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kCompactUnroll; ++u)
        if (ok[u]) sc[d0 + j0 + u * kCompactThreads + tid] = v[u];
      __syncthreads();
    }
    return;
  }
  uint8_t* base;
  int row_bytes;
  if (sx < p.strips_c) {
    base = static_cast<uint8_t*>(const_cast<void*>(t.c));
    row_bytes = t.d_c * p.elem;
  } else {
    sx -= p.strips_c;
    base = static_cast<uint8_t*>(const_cast<void*>(t.k));
    row_bytes = t.d_r * p.elem;
  }
  constexpr int kMaxRows = kCompactThreads / kCompactMinStrip * kCompactUnroll;
  __shared__ int from_s[2][kMaxRows], to_s[2][kMaxRows];        // pool rows of a tile
  const int step = kCompactThreads / p.strip;                   // rows a block reads at once
  const int rows = step * kCompactUnroll;                       // of a tile
  const int x = tid % p.strip, y = tid / p.strip;
  const bool act = x < row_bytes / 16 - sx * p.strip;
  base += (sx * p.strip + x) * 16;
  auto look_up = [&](int j0, int buf) {
    for (int i = tid; i < rows; i += kCompactThreads) {
      const int j = j0 + i;
      int64_t from = -1, to = -1;
      int s;
      if (j < m && check(j, s)) {
        from = compact_row(t, b, s);
        to = from < 0 ? -1 : compact_row(t, b, d0 + j);
      }
      from_s[buf][i] = (int)from;
      to_s[buf][i] = (int)to;
    }
  };
  uint4 v[kCompactUnroll], w[kCompactUnroll];
  int to[kCompactUnroll], to_w[kCompactUnroll];
  auto read = [&](int buf, uint4 (&d)[kCompactUnroll], int (&g)[kCompactUnroll]) {
#pragma unroll
    for (int u = 0; u < kCompactUnroll; ++u) {
      const int i = u * step + y;
      g[u] = act ? to_s[buf][i] : -1;
      if (g[u] >= 0) d[u] = *reinterpret_cast<const uint4*>(base + (int64_t)from_s[buf][i] * row_bytes);
    }
  };
  look_up(first, 0);
  __syncthreads();
  read(0, v, to);
  int buf = 0;
  for (int j0 = first; j0 < m; j0 += rows) {
    buf ^= 1;
    look_up(j0 + rows, buf);
    __syncthreads();            // this tile's rows are read, the next one's are looked up
    read(buf, w, to_w);
#pragma unroll
    for (int u = 0; u < kCompactUnroll; ++u)
      if (to[u] >= 0) *reinterpret_cast<uint4*>(base + (int64_t)to[u] * row_bytes) = v[u];
#pragma unroll
    for (int u = 0; u < kCompactUnroll; ++u) {
      v[u] = w[u];
      to[u] = to_w[u];
    }
  }
}

}  // namespace lca
