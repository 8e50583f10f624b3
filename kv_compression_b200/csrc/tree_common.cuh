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
  if (!t.table) return (int64_t)b * t.page_size + pos;
  return paged_row(t.table, t.max_pages, t.page_size, t.num_pages, b, pos, t.err, where);
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

// ---------------------------------------------------------------- merge of partial softmax sums
// Row r = (node, head) of sequence b has n_part(b) partials (M, Z, O = sum
// e^{x - M} c), M and Z in units of log2; they merge to
//   out = sum_s 2^{M_s - M} O_s / Z,  Z = sum_s 2^{M_s - M} Z_s,  lse = ln 2 (M + log2 Z).
// A row that saw nothing (Z = 0) gives 0 and -inf; one of a bad sequence NaN.
constexpr float kTreeLog2e = 1.4426950408889634f;
constexpr float kTreeLn2 = 0.6931471805599453f;

// 2^{m - top} for m <= top; 1 where they are equal, infinite ones among them.
__device__ __forceinline__ float tree_scale(float m, float top) { return m == top ? 1.f : exp2f(m - top); }

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
  int rows_per_block;
  bool direct;                  // parts == 1 was written by the main kernel
  void* out;                    // [B][T][H][d_c] in the cache's type
  float* lse;                   // [B][T][H]; null: not wanted
};

constexpr int kTreeMergeThreads = 128;

// One CTA per (node, head) row of one sequence; the parts are added in order.
template <typename T>
__global__ void __launch_bounds__(kTreeMergeThreads) lca_tree_merge_kernel(const TreeMergeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.y;
  const TreeSplit sp = p.split[b];
  const TreeLens ln = tree_lens(p.t, b);
  const int64_t R = (int64_t)p.t.T * p.t.H;
  for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
    T* out = static_cast<T*>(p.out) + ((int64_t)b * R + r) * p.t.d_c;
    float* lse = p.lse ? p.lse + (int64_t)b * R + r : nullptr;
    if (sp.bad) {
      for (int d = threadIdx.x; d < p.t.d_c; d += kTreeMergeThreads) out[d] = from_f32<T>(__int_as_float(0x7fc00000));
      if (lse && threadIdx.x == 0) *lse = __int_as_float(0x7fc00000);
      continue;
    }
    if (r >= (int64_t)ln.d * p.t.H || (p.direct && sp.parts == 1)) continue;
    const int rb = (int)(r / p.rows_per_block), col = (int)(r - (int64_t)rb * p.rows_per_block);
    float M = -INFINITY, Z = 0.f;
    for (int s = 0; s < sp.parts; ++s) {
      const int64_t i = (int64_t)(sp.base + s * sp.rb + rb) * p.rows_per_block + col;
      const float m = p.part_mz[2 * i], z = p.part_mz[2 * i + 1];
      const float top = fmaxf(M, m);
      Z = Z * tree_scale(M, top) + z * tree_scale(m, top);
      M = top;
    }
    const float inv = Z == 0.f ? 0.f : 1.f / Z;
    for (int d = threadIdx.x; d < p.t.d_c; d += kTreeMergeThreads) {
      float acc = 0.f;
      for (int s = 0; s < sp.parts; ++s) {
        const int64_t i = (int64_t)(sp.base + s * sp.rb + rb) * p.rows_per_block + col;
        acc += tree_scale(p.part_mz[2 * i], M) * p.part_o[i * p.t.d_c + d];
      }
      out[d] = from_f32<T>(acc * inv);
    }
    if (lse && threadIdx.x == 0) *lse = Z == 0.f ? -INFINITY : kTreeLn2 * (M + log2f(Z));
  }
}

}  // namespace lca
