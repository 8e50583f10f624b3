// tree_simt_kernel.cuh -- the draft-tree attention and the attention weights on
// CUDA cores, fp32 arithmetic: fp32 caches and the shapes that the tensor-core
// kernels do not take.
//
//   x[r][t] = q_c[r] . c_t + q_r[r] . k_t        r = (node, head), t a token it sees
//   tree    out[r] = sum_t softmax_t(x[r][t]) c_t, lse[r] = log sum_t e^{x[r][t]}
//   mass    s[t] = decay prev[t] + sum_r e^{x[r][t] - lse[r]}
//
// A block holds 32 tokens' rows in shared memory as fp32 and works on 8 rows r
// at a time: a warp per row and a lane per token for the products and the
// running maximum and sum; then a thread per latent dim for the sum of values.
// Tokens that a row does not see are left out of every sum (no 0 x value), so
// whatever their rows hold is not felt.
#pragma once
#include "tree_common.cuh"

namespace lca {

constexpr int kTreeSimtRows = 8;       // warps
constexpr int kTreeSimtTile = 32;      // tokens: lanes
constexpr int kTreeSimtThreads = 256;
constexpr int kTreeSimtMaxDims = 4;    // d_c <= 1024: dims of a thread

__host__ __device__ inline size_t tree_simt_smem(int d_c, int d_r) {
  const size_t d = (size_t)d_c + d_r;
  // the tile's rows are 4 floats longer: 16-byte reads of 32 rows then spread over the banks
  return sizeof(float) * (kTreeSimtRows * d + kTreeSimtTile * (d + 4) + kTreeSimtRows * kTreeSimtTile + kTreeSimtRows);
}

// Stage tokens [t0, t0 + 32) of sequence b (those below `end`; zeros behind).
template <typename T>
__device__ __forceinline__ void tree_stage_tile(const TreeBatch& t, int b, int t0, int end, float* tile, int where) {
  const int dq = (t.d_c + t.d_r) / 4, cq = t.d_c / 4, stride = t.d_c + t.d_r + 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int j = warp; j < kTreeSimtTile; j += kTreeSimtThreads / 32) {
    float* dst = tile + (size_t)j * stride;
    if (t0 + j >= end) {
      for (int i = lane; i < dq; i += 32) *reinterpret_cast<float4*>(dst + 4 * i) = make_float4(0.f, 0.f, 0.f, 0.f);
      continue;
    }
    const int64_t row = tree_row(t, b, t0 + j, where);
    const T* c = static_cast<const T*>(t.c) + row * t.d_c;
    const T* k = static_cast<const T*>(t.k) + row * t.d_r;
    for (int i = lane; i < dq; i += 32)
      *reinterpret_cast<float4*>(dst + 4 * i) = i < cq ? load4(c + 4 * i) : load4(k + 4 * (i - cq));
  }
}

// Stage query rows [r0, r0 + 8) of sequence b (those below `rows`).
template <typename T>
__device__ __forceinline__ void tree_stage_q(const TreeBatch& t, const void* q_c, const void* q_r, int b, int64_t r0,
                                             int64_t rows, float* q) {
  const int d = t.d_c + t.d_r, dq = d / 4, cq = t.d_c / 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t r = r0 + warp;
  if (r >= rows) return;
  const int64_t row = (int64_t)b * t.T * t.H + r;
  const T* c = static_cast<const T*>(q_c) + row * t.d_c;
  const T* k = static_cast<const T*>(q_r) + row * t.d_r;
  for (int i = lane; i < dq; i += 32)
    *reinterpret_cast<float4*>(q + (size_t)warp * d + 4 * i) = i < cq ? load4(c + 4 * i) : load4(k + 4 * (i - cq));
}

__device__ __forceinline__ float tree_dot(const float* q, const float* x, int d) {
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < d; i += 4) {
    const float4 u = *reinterpret_cast<const float4*>(q + i), v = *reinterpret_cast<const float4*>(x + i);
    a.x = fmaf(u.x, v.x, a.x); a.y = fmaf(u.y, v.y, a.y); a.z = fmaf(u.z, v.z, a.z); a.w = fmaf(u.w, v.w, a.w);
  }
  return (a.x + a.y) + (a.z + a.w);
}

// Whether row r (node r / H, mask word w) sees position pos: a cached token, or a drafted one of its mask.
__device__ __forceinline__ bool tree_sees(const TreeLens& ln, unsigned long long w, int pos) {
  return pos < ln.n || (pos < ln.n + ln.d && ((w >> (pos - ln.n)) & 1ull));
}

struct TreeSimtParams {
  TreeBatch t;
  const void* q_c;              // [B][T][H][d_c]
  const void* q_r;
  int n_split;                  // parts of a sequence (8 rows a slot); one part: the output is written here
  float* part_o;
  float* part_mz;
  TreeSplit* split;
  void* out;
  float* lse;
};

// grid (n_split, ceil(T H / 8), B).
template <typename T>
__global__ void __launch_bounds__(kTreeSimtThreads) lca_tree_simt_kernel(const TreeSimtParams p) {
  extern __shared__ float tree_smem[];
  const TreeBatch& t = p.t;
  const int b = blockIdx.z, rb = blockIdx.y, s = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int d = t.d_c + t.d_r, stride = d + 4;
  float* q = tree_smem;
  float* tile = q + kTreeSimtRows * d;
  float* pw = tile + (size_t)kTreeSimtTile * stride;            // [8][32] weights
  float* fac = pw + kTreeSimtRows * kTreeSimtTile;              // [8] factors of the sums so far
  const TreeLens ln = tree_lens(t, b);
  const int slot0 = b * p.n_split * (int)gridDim.y;
  if (s == 0 && rb == 0 && threadIdx.x == 0) {
    p.split[b] = TreeSplit{slot0, ln.d > 0 ? p.n_split : 0, (int)gridDim.y, ln.bad ? 1 : 0};
    if (ln.bad) input_error(t.err, 0xB01);
  }
  const int64_t rows = (int64_t)ln.d * t.H, r0 = (int64_t)rb * kTreeSimtRows, r = r0 + warp;
  if (r0 >= rows) return;
  tree_stage_q<T>(t, p.q_c, p.q_r, b, r0, rows, q);
  const unsigned long long word = r < rows ? tree_word(t, b, (int)(r / t.H)) : 0ull;
  const int total = ln.n + ln.d;
  int per = (total + p.n_split - 1) / p.n_split;
  per = (per + kTreeSimtTile - 1) / kTreeSimtTile * kTreeSimtTile;
  const int lo = (int)min((int64_t)total, (int64_t)s * per), hi = min(total, lo + per);
  float M = -INFINITY, Z = 0.f;
  float acc[kTreeSimtMaxDims][kTreeSimtRows];
#pragma unroll
  for (int k = 0; k < kTreeSimtMaxDims; ++k)
#pragma unroll
    for (int w = 0; w < kTreeSimtRows; ++w) acc[k][w] = 0.f;
  for (int t0 = lo; t0 < hi; t0 += kTreeSimtTile) {
    __syncthreads();
    tree_stage_tile<T>(t, b, t0, hi, tile, 0xB02);
    __syncthreads();
    const int pos = t0 + lane;
    float x = -INFINITY;
    if (r < rows && pos < hi && tree_sees(ln, word, pos))
      x = kTreeLog2e * tree_dot(q + (size_t)warp * d, tile + (size_t)lane * stride, d);
    float top = x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    top = fmaxf(M, top);
    const bool live = r < rows && pos < hi && tree_sees(ln, word, pos);
    const float e = live ? exp2f(x - top) : 0.f;
    const float f = tree_scale(M, top);
    M = top;
    float z = e;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    Z = Z * f + z;
    // a token that the row does not see is marked by a negative weight and left out below
    pw[warp * kTreeSimtTile + lane] = live ? e : -1.f;
    if (lane == 0) fac[warp] = f;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kTreeSimtRows; ++w) {
      const float fw = fac[w];
#pragma unroll
      for (int k = 0; k < kTreeSimtMaxDims; ++k) acc[k][w] *= fw;
    }
    for (int j = 0; j < kTreeSimtTile && t0 + j < hi; ++j) {
      float v[kTreeSimtMaxDims];
#pragma unroll
      for (int k = 0; k < kTreeSimtMaxDims; ++k) {
        const int dim = threadIdx.x + k * kTreeSimtThreads;
        v[k] = dim < t.d_c ? tile[(size_t)j * stride + dim] : 0.f;
      }
#pragma unroll
      for (int w = 0; w < kTreeSimtRows; ++w) {
        const float e8 = pw[w * kTreeSimtTile + j];
        if (!(e8 < 0.f)) {
#pragma unroll
          for (int k = 0; k < kTreeSimtMaxDims; ++k) acc[k][w] = fmaf(e8, v[k], acc[k][w]);
        }
      }
    }
  }
  if (p.n_split == 1) {
    if (lane == 0) fac[warp] = Z == 0.f ? 0.f : 1.f / Z;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kTreeSimtRows; ++w) {
      if (r0 + w >= rows) break;
      T* out = static_cast<T*>(p.out) + ((int64_t)b * t.T * t.H + r0 + w) * t.d_c;
#pragma unroll
      for (int k = 0; k < kTreeSimtMaxDims; ++k) {
        const int dim = threadIdx.x + k * kTreeSimtThreads;
        if (dim < t.d_c) out[dim] = from_f32<T>(acc[k][w] * fac[w]);
      }
    }
    if (lane == 0 && r < rows && p.lse)
      p.lse[(int64_t)b * t.T * t.H + r] = Z == 0.f ? -INFINITY : kTreeLn2 * (M + log2f(Z));
    return;
  }
  const int64_t i0 = (int64_t)(slot0 + s * (int)gridDim.y + rb) * kTreeSimtRows;
#pragma unroll
  for (int w = 0; w < kTreeSimtRows; ++w) {
    if (r0 + w >= rows) break;
#pragma unroll
    for (int k = 0; k < kTreeSimtMaxDims; ++k) {
      const int dim = threadIdx.x + k * kTreeSimtThreads;
      if (dim < t.d_c) p.part_o[(i0 + w) * t.d_c + dim] = acc[k][w];
    }
  }
  if (lane == 0 && r < rows) {
    p.part_mz[2 * (i0 + warp)] = M;
    p.part_mz[2 * (i0 + warp) + 1] = Z;
  }
}

struct MassParams {
  TreeBatch t;
  const void* q_c;
  const void* q_r;
  const float* lse;             // [B][T][H]
  const float* prev;            // [B][stride]; null: zeros
  float* scores;                // [B][stride]
  int64_t stride;
  float decay;
};

// The row's exponent offset: an infinite lse marks a row that adds nothing.
__device__ __forceinline__ float mass_offset(float lse) { return isinf(lse) ? INFINITY : lse * kTreeLog2e; }

// A position's new sum: cached tokens go on from what they had, drafted ones begin.
__device__ __forceinline__ void mass_store(const MassParams& p, int b, int pos, int n, float add) {
  const int64_t i = (int64_t)b * p.stride + pos;
  float old = 0.f;
  if (pos < n && p.prev && p.decay != 0.f) old = p.decay * p.prev[i];
  p.scores[i] = old + add;
}

// grid (blocks, B): a block takes every gridDim.x-th tile of 32 tokens through all rows.
template <typename T>
__global__ void __launch_bounds__(kTreeSimtThreads) lca_mass_simt_kernel(const MassParams p) {
  extern __shared__ float tree_smem[];
  const TreeBatch& t = p.t;
  const int b = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int d = t.d_c + t.d_r, stride = d + 4;
  float* q = tree_smem;
  float* tile = q + kTreeSimtRows * d;
  float* part = tile + (size_t)kTreeSimtTile * stride;          // [8][32]
  const TreeLens ln = tree_lens(t, b);
  if (ln.bad && blockIdx.x == 0 && threadIdx.x == 0) input_error(t.err, 0xB03);
  const int64_t rows = (int64_t)ln.d * t.H;
  const int total = ln.n + ln.d;
  for (int64_t t0 = (int64_t)blockIdx.x * kTreeSimtTile; t0 < total; t0 += (int64_t)gridDim.x * kTreeSimtTile) {
    __syncthreads();
    tree_stage_tile<T>(t, b, (int)t0, total, tile, 0xB04);
    const int pos = (int)t0 + lane;
    float sum = 0.f;
    for (int64_t r0 = 0; r0 < rows; r0 += kTreeSimtRows) {
      __syncthreads();
      tree_stage_q<T>(t, p.q_c, p.q_r, b, r0, rows, q);
      __syncthreads();
      const int64_t r = r0 + warp;
      if (r >= rows) continue;
      const float off = mass_offset(p.lse[(int64_t)b * t.T * t.H + r]);
      if (off != INFINITY && pos < total && tree_sees(ln, tree_word(t, b, (int)(r / t.H)), pos))
        sum += exp2f(fmaf(tree_dot(q + (size_t)warp * d, tile + (size_t)lane * stride, d), kTreeLog2e, -off));
    }
    part[warp * kTreeSimtTile + lane] = sum;
    __syncthreads();
    if (warp == 0 && pos < total) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kTreeSimtRows; ++w) s += part[w * kTreeSimtTile + lane];
      mass_store(p, b, pos, ln.n, s);
    }
  }
}

}  // namespace lca
