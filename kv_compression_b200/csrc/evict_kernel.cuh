// evict_kernel.cuh -- which rows an eviction keeps, and moving kept rows to the
// front of their sequence.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "tree_common.cuh"

namespace lca {

// ---------------------------------------------------------------- choice
// Of a sequence's n rows, `budget` stay: the first n_sink, the last n_recent,
// and of the rows between those with the largest sums, the lower row first
// where sums are equal.  A sum that is not a number counts as the smallest.
// All rows stay where n <= budget.  The kept rows are written in rising order.
//
// The sums map to unsigned keys of the same order; the key of the last row kept
// is found 8 bits at a time (a histogram of the keys that share the bits found
// so far), then one pass in row order writes the rows.
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
  int* err;
};

__device__ __forceinline__ uint32_t select_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);                  // -0 counts as 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kSelectThreads = 1024;

__global__ void __launch_bounds__(kSelectThreads) lca_select_kernel(const SelectParams p) {
  __shared__ int hist[256];
  __shared__ int s_bin, s_above;
  __shared__ int wk[kSelectThreads / 32], we[kSelectThreads / 32];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = p.seq_lens[b];
  if (n < 0 || n > p.cap) {
    if (tid == 0) {
      input_error(p.err, 0xB10);
      p.kept_lens[b] = 0;
    }
    return;
  }
  const float* x = p.scores + (int64_t)b * p.stride;
  int32_t* kept = p.kept + (int64_t)b * p.budget;
  if (tid == 0) p.kept_lens[b] = min(n, p.budget);
  if (n <= p.budget) {
    for (int i = tid; i < n; i += kSelectThreads) kept[i] = i;
    return;
  }
  const int lo = p.n_sink, hi = n - p.n_recent;
  int need = p.budget - p.n_sink - p.n_recent;                  // rows to take from [lo, hi)
  uint32_t prefix = 0, have = 0;                                // key bits found; their mask
  if (need > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int i = lo + tid; i < hi; i += kSelectThreads) {
        const uint32_t k = select_key(x[i]);
        if ((k & have) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int above = 0, bin = 255;
        for (; bin > 0; --bin) {
          if (above + hist[bin] >= need) break;
          above += hist[bin];
        }
        s_bin = bin;
        s_above = above;
      }
      __syncthreads();
      prefix |= (uint32_t)s_bin << shift;
      have |= 255u << shift;
      need -= s_above;
      __syncthreads();
    }
  }
  // rows in order: kept by place, by a larger key, or among the first `need` of the equal ones
  const bool any = p.budget - p.n_sink - p.n_recent > 0;
  int done = 0, equal = 0;
  for (int i0 = 0; i0 < n; i0 += kSelectThreads) {
    const int i = i0 + tid;
    bool keep = false, eq = false;
    if (i < n) {
      if (i < lo || i >= hi) {
        keep = true;
      } else if (any) {
        const uint32_t k = select_key(x[i]);
        keep = k > prefix;
        eq = k == prefix;
      }
    }
    const uint32_t eb = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) we[warp] = __popc(eb);
    __syncthreads();
    int before = equal, all = 0;
    for (int w = 0; w < kSelectThreads / 32; ++w) {
      if (w < warp) before += we[w];
      all += we[w];
    }
    if (eq) keep = before + __popc(eb & ((1u << lane) - 1u)) < need;
    equal += all;
    const uint32_t kb = __ballot_sync(0xffffffffu, keep);
    if (lane == 0) wk[warp] = __popc(kb);
    __syncthreads();
    int at = done, sum = 0;
    for (int w = 0; w < kSelectThreads / 32; ++w) {
      if (w < warp) at += wk[w];
      sum += wk[w];
    }
    if (keep) kept[at + __popc(kb & ((1u << lane) - 1u))] = i;
    done += sum;
    __syncthreads();
  }
}

// ---------------------------------------------------------------- moving rows
// Row dst0 + j of a sequence becomes its row src[j], j = 0 .. m - 1, in place;
// src rises strictly and src[j] >= dst0 + j.  A block moves one 16-byte-wide
// strip of columns (or a few) of one sequence, tile after tile of rows in
// order: the rows of a tile are read into registers by the whole block before
// any of them is written, and every later tile reads only rows above those
// written so far (src[j] >= dst0 + j), so no row is overwritten before it is
// read; different strips do not meet.  Rows at their place already (src[j] =
// dst0 + j, the first ones, since src[j] - j never falls) are passed over.
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

__global__ void __launch_bounds__(kCompactThreads) lca_compact_kernel(const CompactParams p) {
  const TreeBatch& t = p.t;
  const int b = blockIdx.y, tid = threadIdx.x;
  const int m = p.n_src[b];
  const int d0 = p.dst0 ? p.dst0[b] : 0;
  if (m < 0 || m > p.src_stride || d0 < 0 || (int64_t)d0 + m > t.cap) {
    if (blockIdx.x == 0 && tid == 0) input_error(t.err, 0xB20);
    return;
  }
  const int32_t* src = p.src + (int64_t)b * p.src_stride;
  int first = 0;
  for (int hi = m; first < hi;) {
    const int mid = (first + hi) >> 1;
    if (src[mid] == d0 + mid) first = mid + 1; else hi = mid;
  }
  int sx = blockIdx.x;
  uint8_t* base;
  int row_bytes, col, cols;     // this block's columns: [col, col + cols) of 16 bytes
  const bool is_score = sx >= p.strips_c + p.strips_k;
  if (sx < p.strips_c) {
    base = static_cast<uint8_t*>(const_cast<void*>(t.c));
    row_bytes = t.d_c * p.elem;
  } else {
    sx -= p.strips_c;
    base = static_cast<uint8_t*>(const_cast<void*>(t.k));
    row_bytes = t.d_r * p.elem;
  }
  if (is_score) {
    for (int j0 = first; j0 < m; j0 += kCompactThreads * kCompactUnroll) {
      float v[kCompactUnroll];
      bool ok[kCompactUnroll];
      float* sc = p.scores + (int64_t)b * p.score_stride;
#pragma unroll
      for (int u = 0; u < kCompactUnroll; ++u) {
        const int j = j0 + u * kCompactThreads + tid;
        const int s = j < m ? src[j] : 0;
        ok[u] = j < m && s >= d0 + j && s < t.cap && (j == 0 || s > src[j - 1]);
        if (j < m && !ok[u]) input_error(t.err, 0xB21);
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
  col = sx * p.strip;
  cols = min(p.strip, row_bytes / 16 - col);
  const int rows_step = kCompactThreads / p.strip;
  const int x = tid % p.strip, y = tid / p.strip;
  const bool act = x < cols && y < rows_step;
  for (int j0 = first; j0 < m; j0 += rows_step * kCompactUnroll) {
    uint4 v[kCompactUnroll];
    int64_t to[kCompactUnroll];             // where the row goes; -1: nowhere
#pragma unroll
    for (int u = 0; u < kCompactUnroll; ++u) {
      const int j = j0 + u * rows_step + y;
      const int s = act && j < m ? src[j] : 0;
      const bool ok = act && j < m && s >= d0 + j && s < t.cap && (j == 0 || s > src[j - 1]);
      if (act && j < m && !ok) input_error(t.err, 0xB21);
      const int64_t from = ok ? compact_row(t, b, s) : -1;
      to[u] = from >= 0 ? compact_row(t, b, d0 + j) : -1;
      if (to[u] >= 0) v[u] = *reinterpret_cast<const uint4*>(base + from * row_bytes + (col + x) * 16);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kCompactUnroll; ++u)
      if (to[u] >= 0) *reinterpret_cast<uint4*>(base + to[u] * row_bytes + (col + x) * 16) = v[u];
    __syncthreads();
  }
}

}  // namespace lca
