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
// cluster of CTAs, each with a contiguous run of its rows and each thread with
// E consecutive ones, whose keys are read once (128-byte lines) and kept in
// shared memory, thread t's e-th at [e][t].  The key of the last row kept is found 8 bits at a
// time: a histogram per CTA of the keys that share the bits found so far, added
// up over the cluster by every CTA for itself; it ends early once all rows that
// share the bits found are to stay.  A scan of the threads' counts (and the
// lower CTAs' totals) then says where each thread's rows go.
// What bounds it is latency: up to four histograms, each with a cluster barrier.
// (11 bits at a time, three histograms, took 30 us instead of 20 at 8 x 131072
// rows: adding 2048 bins over 8 CTAs costs more than a further round.)
struct SelectParams {
  const float* scores;          // [B][stride]
  int64_t stride;
  const int32_t* seq_lens;      // [B]
  int B;
  int64_t cap;                  // the longest valid length
  int n_sink, n_recent;
  int budget;                   // entries a row of `kept` has
  int32_t* kept;                // [B][budget]
  int32_t* kept_lens;           // [B]; may be seq_lens
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
constexpr int kSelectBins = 256;
constexpr int kSelectKeep = 40;             // rows of a thread whose keys stay in shared memory; later ones are read again
constexpr int kSelectStride = kSelectThreads + 1;   // of keys[e]: what one warp reads from memory falls into all banks
constexpr int kSelectMaxCtas = 8;

// Rows of a thread, of n over `ctas` CTAs.
__host__ __device__ inline int select_each(int64_t n, int ctas) {
  const int64_t per = (n + ctas - 1) / ctas;
  return (int)((per + kSelectThreads - 1) / kSelectThreads);
}
__host__ __device__ inline size_t select_smem(int each) {
  return sizeof(int) * (4 * kSelectBins + (size_t)(each < kSelectKeep ? each : kSelectKeep) * kSelectStride);
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
__device__ __forceinline__ int warp_scan(int v, int lane) {     // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
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
  int* hist = select_dyn;                                       // [4][256]
  uint32_t* keys = reinterpret_cast<uint32_t*>(select_dyn + 4 * kSelectBins);
  __shared__ int warp_sum[kSelectWarps], warp_eq[kSelectWarps];
  __shared__ int s_bin, s_above, s_count;
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
  if (n <= p.budget) {
    if (rank == 0 && tid == 0) p.kept_lens[b] = n;              // (what others may still read there, in place)
    for (int i = rank * kSelectThreads + tid; i < n; i += ctas * kSelectThreads) kept[i] = i;
    return;
  }
  const float* x = p.scores + (int64_t)b * p.stride;
  const int each = select_each(n, ctas), run = each * kSelectThreads;
  const int r0 = (int)min((int64_t)n, (int64_t)rank * run), r1 = (int)min((int64_t)n, (int64_t)r0 + run);   // this CTA's rows
  const int lo = p.n_sink, hi = n - p.n_recent;                 // rows that compete
  const int first = r0 + tid * each;                            // this thread's rows
  const int mine = max(0, min(each, r1 - first));
  auto key_of = [&](int e) { return e < kSelectKeep ? keys[e * kSelectStride + tid] : select_key(x[first + e]); };
  hist[tid] = 0;
  __syncthreads();
  int need = p.budget - p.n_sink - p.n_recent;                  // rows to take of [lo, hi)
  const bool any = need > 0;
  uint32_t prefix = 0, have = 0;                                // bits of the last key found; their mask
  {
    // the run's keys, line by line; row j of it is thread j / each's e = j % each
    const uint32_t magic = (uint32_t)(((1ull << 32) + each - 1) / each);   // j magic >> 32 is j / each, or one more
    constexpr int kUnroll = 16;
    for (int u0 = 0; u0 < each; u0 += kUnroll) {
      float v[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = r0 + (u0 + u) * kSelectThreads + tid;
        v[u] = u0 + u < each && i < r1 ? x[i] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int j = (u0 + u) * kSelectThreads + tid, i = r0 + j;
        if (u0 + u >= each || i >= r1) continue;
        const uint32_t k = select_key(v[u]);
        int c = each == 1 ? j : (int)__umulhi((uint32_t)j, magic), e = j - c * each;
        if (e < 0) {                                            // one more: only with more than 2048 rows a thread
          --c;
          e += each;
        }
        if (!LCA_CHECK(p.err, e >= 0 && e < each && c >= 0 && c < kSelectThreads, 0xD70)) continue;
        if (e < kSelectKeep) keys[e * kSelectStride + c] = k;
        if (i >= lo && i < hi) atomicAdd(&hist[k >> 24], 1);
      }
    }
  }
#pragma unroll 1
  for (int pass = 0; any; ++pass) {
    int* h = hist + pass * kSelectBins;
    const int shift = 24 - 8 * pass;
    if (pass > 0) {
      for (int e = 0; e < mine; ++e) {
        const uint32_t k = key_of(e);
        const int i = first + e;
        if ((k & have) == prefix && i >= lo && i < hi) atomicAdd(&h[(k >> shift) & 255u], 1);
      }
    }
    ptx::cluster_sync();                                        // (also the CTA's own barrier)
    if (warp < 2) {
      // thread t < 64 has the four bins from 255 - 4t down; their counts over the cluster, scanned from the top
      const int bin0 = kSelectBins - 4 - 4 * tid;
      int4 v[kSelectMaxCtas], c = make_int4(0, 0, 0, 0);        // .w the highest bin
#pragma unroll
      for (int r = 0; r < kSelectMaxCtas; ++r) v[r] = r < ctas ? ld_cluster4(h + bin0, r) : make_int4(0, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < kSelectMaxCtas; ++r) {
        c.x += v[r].x; c.y += v[r].y; c.z += v[r].z; c.w += v[r].w;
      }
      const int sum = c.x + c.y + c.z + c.w, incl = warp_scan(sum, lane);
      if (warp == 0 && lane == 31) warp_sum[0] = incl;
      ptx::named_bar_sync(1, 64);
      int above = incl - sum + (warp == 1 ? warp_sum[0] : 0);   // rows in higher bins
      const int count[4] = {c.w, c.z, c.y, c.x};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (above < need && need <= above + count[q]) {
          s_bin = bin0 + 3 - q;
          s_above = above;
          s_count = count[q];
        }
        above += count[q];
      }
    }
    __syncthreads();
    prefix |= (uint32_t)s_bin << shift;
    have |= 255u << shift;
    need -= s_above;
    if (s_count == need || pass == 3) break;
  }
  // a thread's rows: kept for sure (by place, or by a larger key), or of the last key
  auto judge = [&](int e, bool& sure, bool& eq) {
    const int i = first + e;
    const bool place = i < lo || i >= hi;
    const uint32_t k = any && !place ? key_of(e) & have : 0u;
    sure = place || (any && k > prefix);
    eq = !place && any && k == prefix;
  };
  int n_sure = 0, n_eq = 0;
  for (int e = 0; e < mine; ++e) {
    bool sure, eq;
    judge(e, sure, eq);
    n_sure += sure;
    n_eq += eq;
  }
  const int in_sure = warp_scan(n_sure, lane), in_eq = warp_scan(n_eq, lane);
  __syncthreads();                                              // (warp_sum[0] is read)
  if (lane == 31) {
    warp_sum[warp] = in_sure;
    warp_eq[warp] = in_eq;
  }
  __syncthreads();
  int sure_before = warp_prefix(warp_sum, warp, lane) + in_sure - n_sure;
  int eq_before = warp_prefix(warp_eq, warp, lane) + in_eq - n_eq;
  if (tid == kSelectThreads - 1) {
    totals[0] = sure_before + n_sure;
    totals[1] = eq_before + n_eq;
  }
  ptx::cluster_sync();
#pragma unroll
  for (int r = 0; r < kSelectMaxCtas - 1; ++r)
    if (r < rank) {
      sure_before += ld_cluster(totals, r);
      eq_before += ld_cluster(totals + 1, r);
    }
  if (n_sure + n_eq > 0)
    for (int e = 0; e < mine; ++e) {
      bool sure, eq;
      judge(e, sure, eq);
      // of the rows with the last key the first `need` stay
      if (sure || (eq && eq_before < need)) {
        const int at = sure_before + min(eq_before, need);
        if (LCA_CHECK(p.err, at >= 0 && at < p.budget && first + e < n, 0xD71)) kept[at] = first + e;
      }
      sure_before += sure;
      eq_before += eq;
    }
  ptx::cluster_sync();                                          // no CTA leaves while its counts may be read
  if (rank == 0 && tid == 0) p.kept_lens[b] = p.budget;         // kept_lens may be seq_lens: every thread has read it
}

// ---------------------------------------------------------------- moving rows
// Row dst0 + j of a sequence becomes its row src[j], j = 0 .. m - 1, in place;
// src rises strictly and src[j] >= dst0 + j.  A block moves one strip of columns
// (2 or 8 times 16 bytes) of one sequence, tile after tile of rows in order.
// No row is overwritten before it is read: the rows of a tile are in registers
// of the whole block before any of them is written, later tiles read only rows
// above all those written so far (src[j] >= dst0 + j), and strips do not meet.
// For the same reason the next tile's reads may be under way while this tile is
// written, so two tiles (16 reads of 16 bytes a thread) are in flight.
//
// It is bound by memory latency with few sequences and comes to 5.2 TB/s, read
// and written, with 64 (8192 of 32768 rows each: 231 us).  Wide strips suit DRAM and L2, but a block for each SM
// comes first: narrow ones as long as an SM gets no second block (4 sequences,
// 16384 of 32768 rows each: 49 us, 61 with wide ones; 8 sequences, 8192 rows: 57,
// wide 41), and 512 threads instead of 256 as long as all wide ones are resident
// too (8 sequences: 41 instead of 54; with 32 37 instead of 35).  Two divisions a
// row, for its page and place in it, had cost 10%.  Rows from behind the destination
// copied whole by a second kernel, once this one has done the others, did not pay
// (48 -> 51 to 54 us).  Rows at their place already (src[j] = dst0 + j, the first
// ones, since src[j] - j never falls) are passed over, and one block checks that
// they are.
struct CompactParams {
  TreeBatch t;                  // the cache; lengths and masks unused
  int elem;                     // bytes of an element
  const int32_t* src;           // [B][src_stride]
  int64_t src_stride;
  const int32_t* n_src;         // [B]
  const int32_t* dst0;          // [B]; null: 0
  float* scores;                // [B][score_stride]; null: none
  int64_t score_stride;
  int strips_c, strips_k;       // blocks for a row of c, of k; one more for the scores
  uint32_t page_mul;            // of compact_page
  int page_shift;
};

// A position's page, pos / page_size for 0 <= pos < 2^31, with mul = floor(2^(31 + l) / page_size) + 1 (below 2^32)
// and shift = l - 1, l = ceil(log2 page_size) >= 1: mul page_size / 2^(31 + l) is above 1 by at most
// page_size / 2^(31 + l) <= 2^-31, so the product's error stays below 1 / page_size.
__device__ __forceinline__ uint32_t compact_page(const CompactParams& p, uint32_t pos) {
  return __umulhi(pos, p.page_mul) >> p.page_shift;
}

constexpr int kCompactUnroll = 8;
constexpr int kCompactWide = 8, kCompactNarrow = 2;          // strips, in 16 bytes

// A row of the list on its way from the list to the copy: its loads are issued a
// tile apart, so that none is waited for when it is needed.
struct CompactRow {
  int s, before;                // src[j], src[j - 1]; s = -1: no such row
  int page_from, page_to;       // table entries
};

template <int kStrip, int kThreads>
__global__ void __launch_bounds__(kThreads, 512 / kThreads) lca_compact_kernel(const CompactParams p) {
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
  if (blockIdx.x == 0)          // (the probes took the order on trust)
    for (int j = tid; j < first; j += kThreads)
      if (src[j] != d0 + j) input_error(t.err, 0xB21);
  if (first >= m) return;
  auto valid = [&](int j, int s, int before) {
    const bool ok = s >= d0 + j && s < t.cap && (j == 0 || s > before);
    if (!ok) input_error(t.err, 0xB21);
    return ok;
  };
  int sx = blockIdx.x;
  if (sx >= p.strips_c + p.strips_k) {
    float* sc = p.scores + (int64_t)b * p.score_stride;
    for (int j0 = first; j0 < m; j0 += kThreads * kCompactUnroll) {
      float v[kCompactUnroll];
      bool ok[kCompactUnroll];
#pragma unroll
      for (int u = 0; u < kCompactUnroll; ++u) {
        const int j = j0 + u * kThreads + tid;
        const int s = j < m ? src[j] : 0;
        ok[u] = j < m && valid(j, s, j > 0 ? src[j - 1] : -1);
        ok[u] = ok[u] && LCA_CHECK(t.err, s < p.score_stride && d0 + j < p.score_stride, 0xD72);
        v[u] = ok[u] ? sc[s] : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kCompactUnroll; ++u)
        if (ok[u]) sc[d0 + j0 + u * kThreads + tid] = v[u];
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
  constexpr int kStep = kThreads / kStrip;                      // rows a block reads at once
  constexpr int kRows = kStep * kCompactUnroll;                 // of a tile
  constexpr int kEach = kRows / kThreads;                       // rows a thread looks up
  static_assert(kRows % kThreads == 0, "every row of a tile is looked up");
  __shared__ int from_s[2][kRows], to_s[2][kRows];              // pool rows of a tile; -1: the row is left alone
  const int x = tid % kStrip, y = tid / kStrip;
  const bool act = x < row_bytes / 16 - sx * kStrip;
  base += (sx * kStrip + x) * 16;
  const uint32_t ps = (uint32_t)t.page_size;
  const int32_t* table = t.table ? t.table + (int64_t)b * t.max_pages : nullptr;
  CompactRow r[kEach], nx[kEach];
  auto list = [&](uint32_t j0, CompactRow (&q)[kEach]) {        // the list's entries of the tile at j0
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const uint32_t j = j0 + k * kThreads + tid;
      q[k].s = j < (uint32_t)m ? src[j] : -1;
      q[k].before = j < (uint32_t)m && j > 0 ? src[j - 1] : -1;
    }
  };
  auto pages = [&](uint32_t j0, CompactRow (&q)[kEach]) {       // their pages' table entries
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const uint32_t j = j0 + k * kThreads + tid;
      if (j < (uint32_t)m) q[k].s = valid(j, q[k].s, q[k].before) ? q[k].s : -1;
      q[k].page_from = q[k].page_to = b;
      if (table && q[k].s >= 0) {
        q[k].page_from = table[compact_page(p, q[k].s)];
        q[k].page_to = table[compact_page(p, d0 + j)];
      }
    }
  };
  auto rows = [&](uint32_t j0, const CompactRow (&q)[kEach], int buf) {   // and their pool rows
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const uint32_t i = k * kThreads + tid, to = d0 + j0 + i;
      int from = -1, dst = -1;
      if (q[k].s >= 0) {
        if (table && (q[k].page_from < 0 || q[k].page_from >= t.num_pages || q[k].page_to < 0 || q[k].page_to >= t.num_pages)) {
          input_error(t.err, 0xB22);
        } else {
          // page' page_size + pos mod page_size
          from = (int)((q[k].page_from - (table ? compact_page(p, q[k].s) : 0u)) * ps + q[k].s);
          dst = (int)((q[k].page_to - (table ? compact_page(p, to) : 0u)) * ps + to);
          if (!LCA_CHECK(t.err, from >= 0 && from < t.num_pages * t.page_size && dst >= 0 && dst < t.num_pages * t.page_size, 0xD73))
            from = dst = -1;
        }
      }
      from_s[buf][i] = from;
      to_s[buf][i] = dst;
    }
  };
  uint4 v[kCompactUnroll], w[kCompactUnroll];
  int to[kCompactUnroll], to_w[kCompactUnroll];
  auto read = [&](int buf, uint4 (&d)[kCompactUnroll], int (&g)[kCompactUnroll]) {
#pragma unroll
    for (int u = 0; u < kCompactUnroll; ++u) {
      const int i = u * kStep + y;
      g[u] = act ? to_s[buf][i] : -1;
      if (g[u] >= 0) d[u] = *reinterpret_cast<const uint4*>(base + (int64_t)from_s[buf][i] * row_bytes);
    }
  };
  const uint32_t j1 = first;
  list(j1, r);
  list(j1 + kRows, nx);
  pages(j1, r);
  rows(j1, r, 0);
  pages(j1 + kRows, nx);
#pragma unroll
  for (int k = 0; k < kEach; ++k) r[k] = nx[k];                 // r: the next tile, its pages under way
  list(j1 + 2 * kRows, nx);                                     // nx: the one after it, its list under way
  __syncthreads();
  read(0, v, to);
  int buf = 0;
  for (uint32_t j0 = first; j0 < (uint32_t)m; j0 += kRows) {
    buf ^= 1;
    rows(j0 + kRows, r, buf);
#pragma unroll
    for (int k = 0; k < kEach; ++k) r[k] = nx[k];
    pages(j0 + 2 * kRows, r);
    list(j0 + 3 * kRows, nx);
    __syncthreads();            // this tile's rows are read, the next one's are known
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
