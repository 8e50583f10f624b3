// tree_common.cuh -- what the kernels of the draft-tree operators share: the
// batch they work on, its lengths and masks, and where a token's row lies.
//
// A sequence b holds n_b cached tokens (positions 0 .. n_b - 1) and d_b <= T
// drafted ones (positions n_b .. n_b + d_b - 1, the nodes of a tree, parents
// before children).  Node i sees every cached token and the drafted tokens j
// whose bit is set in its mask word (bit j of mask[b][i]); without masks the
// nodes are a chain and node i sees nodes 0 .. i.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "checks.cuh"
#include "device_input.cuh"

namespace lca {

constexpr int kTreeMaxDraft = 64;     // one mask word per node

struct TreeBatch {
  const void* c;                // rows of d_c, rows of d_r: pages of page_size rows
  const void* k;
  int64_t num_pages;
  int page_size;
  const int32_t* table;         // [B][max_pages]; null: sequence b is page b (a contiguous cache)
  int64_t max_pages;
  const int32_t* seq_lens;      // [B] n_b
  const int32_t* draft_lens;    // [B] d_b; null: T
  const unsigned long long* mask;  // [B][T]; null: a chain
  int B, H, T;
  int d_c, d_r;
  int64_t cap;                  // n_b + d_b may not exceed it
  int* err;
};

struct TreeLens {
  int n, d;                     // d = 0: nothing to do; bad: a length was out of range
  bool bad;
};

// The lengths of sequence b; one out of range gives an empty, bad sequence.
__device__ __forceinline__ TreeLens tree_lens(const TreeBatch& t, int b) {
  TreeLens r;
  r.n = t.seq_lens[b];
  r.d = t.draft_lens ? t.draft_lens[b] : t.T;
  r.bad = r.n < 0 || r.d < 0 || r.d > t.T || (int64_t)r.n + r.d > t.cap;
  if (r.bad) r.n = r.d = 0;
  return r;
}

// The mask word of node i: bit j says that it sees node j.
__device__ __forceinline__ unsigned long long tree_word(const TreeBatch& t, int b, int i) {
  return t.mask ? t.mask[(int64_t)b * t.T + i] : (2ull << i) - 1ull;
}

// The pool row of position `pos` of sequence b.
__device__ __forceinline__ int64_t tree_row(const TreeBatch& t, int b, int pos, int where) {
  if (!LCA_CHECK(t.err, pos >= 0 && pos < t.cap && b < t.B, 0xD50)) return 0;
  const int64_t row = t.table ? paged_row(t.table, t.max_pages, t.page_size, t.num_pages, b, pos, t.err, where)
                              : (int64_t)b * t.page_size + pos;
  return LCA_CHECK(t.err, row >= 0 && row < t.num_pages * t.page_size, 0xD51) ? row : 0;
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// Four consecutive elements (16- or 8-byte aligned) as fp32.
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u));
}

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// ---------------------------------------------------------------- merge of partial softmax sums
// Row r = (node, head) of sequence b has n_part(b) partials (M, Z, O = sum
// e^{x - M} c), M and Z in units of log2; they merge to
//   out = sum_s 2^{M_s - M} O_s / Z,  Z = sum_s 2^{M_s - M} Z_s,  lse = ln 2 (M + log2 Z).
// A row that saw nothing (Z = 0) gives 0 and -inf; one of a bad sequence NaN.
constexpr float kTreeLog2e = 1.4426950408889634f;
constexpr float kTreeLn2 = 0.6931471805599453f;

// 2^{m - top} for m <= top; 1 where they are equal, infinite ones among them.
__device__ __forceinline__ float tree_scale(float m, float top) { return m == top ? 1.f : exp2f(m - top); }

// What a row's logits are counted from: their maximum, 0 while all of them are -inf (weights of 0, not NaN).
__device__ __forceinline__ float tree_origin(float top) { return top == -INFINITY ? 0.f : top; }

struct TreeSplit {              // one per sequence, written by the main kernel
  int base;                     // slot of row block 0 of part 0
  int parts;                    // partials of each row; 0: none; 1: the main kernel wrote the output itself
  int rb;                       // row blocks of a part
  int bad;
};

struct TreeMergeParams {
  TreeBatch t;
  const float* part_o;          // [slots][rows a block][d_c]
  const float* part_mz;         // [slots][rows a block][2]
  const TreeSplit* split;
  int64_t slot_rows;            // rows of part_o and part_mz
  int rows_per_block;
  bool direct;                  // parts == 1 was written by the main kernel
  void* out;                    // [B][T][H][d_c] in the cache's type
  float* lse;                   // [B][T][H]; null: not wanted
};

constexpr int kTreeMergeThreads = 128;
constexpr int kTreeMaxParts = 1024;

// One CTA per (node, head) row of one sequence and run of its dims: a lane has
// four of 128, and kSplit warps share those 128, each with every kSplit-th part,
// eight of them at a time; their sums are added in warp order, so the result
// does not depend on timing.  Every part's (M, Z) is read at once by a thread of
// its own.  What it costs is latency: with few rows 4 warps share (82 parts of
// 64 rows: 49 -> 34 us for the whole call), with rows for several CTAs an SM one
// warp does it alone and a CTA takes 512 dims (9 parts of 4096 rows: sharing
// took 25 us more).
constexpr int tree_merge_dims(int split) { return 128 * (kTreeMergeThreads / 32) / split; }

template <typename T, int kSplit>
__global__ void __launch_bounds__(kTreeMergeThreads) lca_tree_merge_kernel(const TreeMergeParams p) {
  constexpr int kWarps = kTreeMergeThreads / 32;
  __shared__ float weight[kTreeMaxParts];
  __shared__ float2 warp_mz[kWarps];
  __shared__ float4 sums[kWarps][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const TreeSplit sp = p.split[b];
  if (!sp.bad && (sp.parts == 0 || (p.direct && sp.parts == 1))) return;
  const TreeLens ln = tree_lens(p.t, b);
  const int64_t R = (int64_t)p.t.T * p.t.H, live = sp.bad ? R : (int64_t)ln.d * p.t.H;
  constexpr int kDims = tree_merge_dims(kSplit);
  const int chunks = (p.t.d_c + kDims - 1) / kDims, turn = warp % kSplit;
  for (int64_t g = blockIdx.x; g < live * chunks; g += gridDim.x) {
    const int64_t r = g / chunks;
    const int chunk = (int)(g - r * chunks), dim = chunk * kDims + 128 * (warp / kSplit) + 4 * lane;
    const bool has = dim < p.t.d_c;
    T* out = static_cast<T*>(p.out) + ((int64_t)b * R + r) * p.t.d_c + dim;
    float* lse = p.lse && chunk == 0 ? p.lse + (int64_t)b * R + r : nullptr;
    if (sp.bad) {
      const float nan = __int_as_float(0x7fc00000);
      if (has && turn == 0) store4(out, make_float4(nan, nan, nan, nan));
      if (lse && tid == 0) *lse = nan;
      continue;
    }
    const int rb = (int)(r / p.rows_per_block), col = (int)(r - (int64_t)rb * p.rows_per_block);
    const int64_t i0 = (int64_t)(sp.base + rb) * p.rows_per_block + col;     // the row in part 0's slot
    const int64_t step = (int64_t)sp.rb * p.rows_per_block;
    if (!LCA_CHECK(p.t.err, sp.parts <= kTreeMaxParts && r < R && i0 + (sp.parts - 1) * step < p.slot_rows, 0xD52)) return;
    // M and Z over the parts: each thread its own, then the block's
    float M = -INFINITY, Z = 0.f;
    for (int s = tid; s < sp.parts; s += kTreeMergeThreads) {
      const float2 mz = *reinterpret_cast<const float2*>(p.part_mz + 2 * (i0 + s * step));
      const float top = fmaxf(M, mz.x);
      Z = Z * tree_scale(M, top) + mz.y * tree_scale(mz.x, top);
      M = top;
      weight[s] = mz.x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float m = __shfl_xor_sync(0xffffffffu, M, o), z = __shfl_xor_sync(0xffffffffu, Z, o);
      const float top = fmaxf(M, m);
      Z = Z * tree_scale(M, top) + z * tree_scale(m, top);
      M = top;
    }
    if (lane == 0) warp_mz[warp] = make_float2(M, Z);
    __syncthreads();
    M = -INFINITY;
    Z = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 mz = warp_mz[w];
      const float top = fmaxf(M, mz.x);
      Z = Z * tree_scale(M, top) + mz.y * tree_scale(mz.x, top);
      M = top;
    }
    const float inv = Z == 0.f ? 0.f : 1.f / Z;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const float* o = p.part_o + i0 * p.t.d_c + dim;
    constexpr int kAtOnce = 8;
    for (int s0 = turn; s0 < sp.parts; s0 += kAtOnce * kSplit) {
      float4 v[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
        if (has && s0 + u * kSplit < sp.parts) v[u] = *reinterpret_cast<const float4*>(o + (s0 + u * kSplit) * step * p.t.d_c);
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
        if (has && s0 + u * kSplit < sp.parts) {
          const float w = tree_scale(weight[s0 + u * kSplit], M) * inv;
          acc.x = fmaf(w, v[u].x, acc.x); acc.y = fmaf(w, v[u].y, acc.y);
          acc.z = fmaf(w, v[u].z, acc.z); acc.w = fmaf(w, v[u].w, acc.w);
        }
    }
    if constexpr (kSplit > 1) {
      sums[warp][lane] = acc;
      __syncthreads();
#pragma unroll
      for (int w = 1; w < kSplit; ++w) {
        const float4 v = sums[(warp + w) % kWarps][lane];
        if (turn == 0) {
          acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
        }
      }
    }
    if (turn == 0 && has) store4(out, acc);
    if (lse && tid == 0) *lse = Z == 0.f ? -INFINITY : kTreeLn2 * (M + log2f(Z));
    __syncthreads();             // the shared values are free again
  }
}

}  // namespace lca
