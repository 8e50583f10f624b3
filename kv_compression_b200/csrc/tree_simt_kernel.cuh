// tree_simt_kernel.cuh -- the draft-tree attention and the attention weights on
// CUDA cores, fp32 arithmetic: fp32 caches and the shapes that the tensor-core
// kernels do not take.
//
//   x[r][t] = q_c[r] . c_t + q_r[r] . k_t        r = (node, head), t a token it sees
//   tree    out[r] = sum_t softmax_t(x[r][t]) c_t, lse[r] = log sum_t e^{x[r][t]}
//   mass    s[t] = decay prev[t] + sum_r e^{x[r][t] - lse[r]}
//
// Up to 8 query rows a sequence: a block holds 32 tokens' rows in shared memory
// as fp32, with a warp per row and a lane per token for the products and the
// running maximum and sum, then a thread per latent dim for the sum of values.
// More: blocks of 32 rows x 64 (wide rows: 32) tokens, both in shared memory; a thread
// has 2 rows x 4 (2) tokens of the products, 16-byte reads of both sides (6 for 32
// FMAs), then 4 dims x 2 to 32 rows of the sum of values (3 reads for 32 FMAs at
// d_c = 256).  Bound by shared memory reads (which would allow 80% of the FMA rate
// for the products), and by what its phases leave idle: two or more blocks an SM
// overlap.  Measured (bf16, 256 + 32, three sequences of 30334 tokens): 317 us with 64
// rows each, about a seventh of what 8-row blocks took, and 885 with 192: 0.27 to 0.29
// of the fp32 rate.
// Tokens that a row does not see are left out of every sum (no 0 x value), so
// whatever their rows hold is not felt.
#pragma once
#include "tree_common.cuh"

namespace lca {

constexpr int kTreeSimtRows = 8;       // warps
constexpr int kTreeSimtTile = 32;      // tokens: lanes
constexpr int kTreeSimtThreads = 256;
constexpr int kTreeWideRows = 32;
constexpr int kTreeSimtMaxDims = 4;    // d_c <= 1024: dims of a thread

__host__ __device__ inline size_t tree_simt_smem(int d_c, int d_r) {
  const size_t d = (size_t)d_c + d_r;
  // the tile's rows are 4 floats longer: 16-byte reads of 32 rows then spread over the banks
  return sizeof(float) * (kTreeSimtRows * d + kTreeSimtTile * (d + 4) + kTreeSimtRows * kTreeSimtTile + kTreeSimtRows);
}

// Stage `count` rows of d_c and d_r elements as fp32 rows of d_c + d_r + 4; list[j] is the j-th row's number, -1: zeros.
// Every thread has four 4-element loads under way at a time (a row a warp, one after another, left the memory
// latency in the open: 331 us against 258 for 22 rows over 6 x 37905 tokens of 160 dims).
template <typename T>
__device__ __forceinline__ void tree_stage_rows(const void* c, const void* k, int d_c, int d_r, int count, const int* list, float* dst) {
  const int dq = (d_c + d_r) / 4, cq = d_c / 4, stride = d_c + d_r + 4, total = count * dq;
  constexpr int kAtOnce = 4;
  for (int i0 = threadIdx.x; i0 < total; i0 += kAtOnce * kTreeSimtThreads) {
    float4 v[kAtOnce];
    int at[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int i = i0 + u * kTreeSimtThreads, j = i / dq, e = i - j * dq;
      at[u] = j * stride + 4 * e;
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < total && list[j] >= 0) {
        const int64_t r = list[j];
        v[u] = e < cq ? load4(static_cast<const T*>(c) + r * d_c + 4 * e) : load4(static_cast<const T*>(k) + r * d_r + 4 * (e - cq));
      }
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
      if (i0 + u * kTreeSimtThreads < total) *reinterpret_cast<float4*>(dst + at[u]) = v[u];
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
  int64_t slot_rows;            // rows of both
  TreeSplit* split;
  void* out;
  float* lse;
};

// grid (n_split, ceil(T H / 8), B).
template <typename T>
__global__ void __launch_bounds__(kTreeSimtThreads) lca_tree_simt_kernel(const TreeSimtParams p) {
  extern __shared__ float tree_smem[];
  __shared__ int list[kTreeSimtTile];
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
  const int lo = (int)min((int64_t)total, (int64_t)s * per), hi = (int)min((int64_t)total, (int64_t)lo + per);
  float M = -INFINITY, Z = 0.f;
  float acc[kTreeSimtMaxDims][kTreeSimtRows];
#pragma unroll
  for (int k = 0; k < kTreeSimtMaxDims; ++k)
#pragma unroll
    for (int w = 0; w < kTreeSimtRows; ++w) acc[k][w] = 0.f;
  for (int t0 = lo; t0 < hi; t0 += kTreeSimtTile) {
    __syncthreads();
    if (threadIdx.x < kTreeSimtTile) list[threadIdx.x] = t0 + (int)threadIdx.x < hi ? (int)tree_row(t, b, t0 + threadIdx.x, 0xB02) : -1;
    __syncthreads();
    tree_stage_rows<T>(t.c, t.k, t.d_c, t.d_r, kTreeSimtTile, list, tile);
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
    const float e = live ? exp2f(x - tree_origin(top)) : 0.f;
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
  if (!LCA_CHECK(t.err, i0 + kTreeSimtRows <= p.slot_rows, 0xD53)) return;
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

// ---------------------------------------------------------------- blocks of 32 rows
__host__ __device__ inline size_t tree_wide_smem(int d_c, int d_r, int tokens) {
  const size_t d = (size_t)d_c + d_r + 4;
  return sizeof(float) * ((kTreeWideRows + tokens) * d + (size_t)tokens * (kTreeWideRows + 4) + 2 * kTreeWideRows);
}
// Tokens of a tile: 64 where two blocks then fit an SM.
__host__ __device__ inline int tree_wide_tokens(int d_c, int d_r) { return tree_wide_smem(d_c, d_r, 64) <= 112 * 1024 ? 64 : 32; }

// Products of query rows 2 ty, 2 ty + 1 with tokens tx, tx + 16, ...
template <int J>
__device__ __forceinline__ void tree_products(const float* q, const float* tile, int d, int ty, int tx, float (&acc)[2][J]) {
  const int stride = d + 4;
  const float *q0 = q + (size_t)(2 * ty) * stride, *q1 = q0 + stride, *t0 = tile + (size_t)tx * stride;
#pragma unroll
  for (int j = 0; j < J; ++j) acc[0][j] = acc[1][j] = 0.f;
#pragma unroll 2
  for (int i = 0; i < d; i += 4) {
    const float4 a = *reinterpret_cast<const float4*>(q0 + i), b = *reinterpret_cast<const float4*>(q1 + i);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const float4 v = *reinterpret_cast<const float4*>(t0 + (size_t)(16 * j) * stride + i);
      acc[0][j] = fmaf(a.x, v.x, acc[0][j]); acc[1][j] = fmaf(b.x, v.x, acc[1][j]);
      acc[0][j] = fmaf(a.y, v.y, acc[0][j]); acc[1][j] = fmaf(b.y, v.y, acc[1][j]);
      acc[0][j] = fmaf(a.z, v.z, acc[0][j]); acc[1][j] = fmaf(b.z, v.z, acc[1][j]);
      acc[0][j] = fmaf(a.w, v.w, acc[0][j]); acc[1][j] = fmaf(b.w, v.w, acc[1][j]);
    }
  }
}

// grid (n_split, ceil(T H / 32), B); kRpt: rows of a thread in the sum of values, 32 / (256 / (d_c / 4)) or more.
template <typename T, int kTokens, int kRpt>
__global__ void __launch_bounds__(kTreeSimtThreads) lca_tree_wide_kernel(const TreeSimtParams p) {
  constexpr int J = kTokens / 16, kPs = kTreeWideRows + 4;
  extern __shared__ float tree_smem[];
  __shared__ int list[kTokens];
  const TreeBatch& t = p.t;
  const int b = blockIdx.z, rb = blockIdx.y, s = blockIdx.x, tid = threadIdx.x;
  const int ty = tid >> 4, tx = tid & 15;
  const int d = t.d_c + t.d_r, stride = d + 4;
  float* q = tree_smem;
  float* tile = q + (size_t)kTreeWideRows * stride;
  float* pw = tile + (size_t)kTokens * stride;                  // [token][row] weights; negative: not seen
  float* fac = pw + kTokens * kPs;                              // [32] factors of the sums so far
  const TreeLens ln = tree_lens(t, b);
  const int slot0 = b * p.n_split * (int)gridDim.y;
  if (s == 0 && rb == 0 && tid == 0) {
    p.split[b] = TreeSplit{slot0, ln.d > 0 ? p.n_split : 0, (int)gridDim.y, ln.bad ? 1 : 0};
    if (ln.bad) input_error(t.err, 0xB01);
  }
  const int64_t rows = (int64_t)ln.d * t.H, r0 = (int64_t)rb * kTreeWideRows;
  if (r0 >= rows) return;
  const int64_t q0 = (int64_t)b * t.T * t.H + r0;
  if (tid < kTreeWideRows) list[tid] = r0 + tid < rows ? (int)(q0 + tid) : -1;
  __syncthreads();
  tree_stage_rows<T>(p.q_c, p.q_r, t.d_c, t.d_r, kTreeWideRows, list, q);
  unsigned long long word[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) word[k] = r0 + 2 * ty + k < rows ? tree_word(t, b, (int)((r0 + 2 * ty + k) / t.H)) : 0ull;
  const int total = ln.n + ln.d;
  int per = (total + p.n_split - 1) / p.n_split;
  per = (per + kTokens - 1) / kTokens * kTokens;
  const int lo = (int)min((int64_t)total, (int64_t)s * per), hi = (int)min((int64_t)total, (int64_t)lo + per);
  const int groups = t.d_c / 4, g = tid % groups, rg = tid / groups;    // sum of values: 4 dims x kRpt rows
  const bool act = rg * kRpt < kTreeWideRows;
  float M[2] = {-INFINITY, -INFINITY}, Z[2] = {0.f, 0.f};
  float4 acc[kRpt];
#pragma unroll
  for (int k = 0; k < kRpt; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int t0 = lo; t0 < hi; t0 += kTokens) {
    __syncthreads();
    if (tid < kTokens) list[tid] = t0 + tid < hi ? (int)tree_row(t, b, t0 + tid, 0xB02) : -1;
    __syncthreads();
    tree_stage_rows<T>(t.c, t.k, t.d_c, t.d_r, kTokens, list, tile);
    __syncthreads();
    float x[2][J];
    tree_products<J>(q, tile, d, ty, tx, x);
    const bool special = t0 + kTokens > ln.n || t0 + kTokens > hi;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float top = -INFINITY;
      uint32_t seen = 0;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int pos = t0 + tx + 16 * j;
        const bool sees = !special || (pos < hi && tree_sees(ln, word[k], pos));
        seen |= (uint32_t)sees << j;
        x[k][j] = sees ? x[k][j] * kTreeLog2e : -INFINITY;
        top = fmaxf(top, x[k][j]);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      top = fmaxf(M[k], top);
      const float f = tree_scale(M[k], top);
      M[k] = top;
      const float origin = tree_origin(top);
      float z = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const float e = (seen >> j) & 1u ? exp2f(x[k][j] - origin) : 0.f;
        z += e;
        pw[(tx + 16 * j) * kPs + 2 * ty + k] = (seen >> j) & 1u ? e : -1.f;
      }
      Z[k] = Z[k] * f + z;
      if (tx == 0) fac[2 * ty + k] = f;
    }
    __syncthreads();
    if (act) {
#pragma unroll
      for (int k = 0; k < kRpt; ++k) {
        const float f = fac[rg * kRpt + k];
        acc[k].x *= f; acc[k].y *= f; acc[k].z *= f; acc[k].w *= f;
      }
      const int tokens = min(kTokens, hi - t0);
      const float* vp = tile + 4 * g;
      const float* wp = pw + rg * kRpt;
      auto add = [&](int k, float e, const float4& v) {
        acc[k].x = fmaf(e, v.x, acc[k].x); acc[k].y = fmaf(e, v.y, acc[k].y);
        acc[k].z = fmaf(e, v.z, acc[k].z); acc[k].w = fmaf(e, v.w, acc[k].w);
      };
      if (!special) {
#pragma unroll 2
        for (int j = 0; j < kTokens; ++j) {
          const float4 v = *reinterpret_cast<const float4*>(vp + (size_t)j * stride);
          float e[kRpt];
          if constexpr (kRpt == 2) {
            const float2 u = *reinterpret_cast<const float2*>(wp + j * kPs);
            e[0] = u.x; e[1] = u.y;
          } else {
#pragma unroll
            for (int k = 0; k < kRpt; k += 4) {
              const float4 u = *reinterpret_cast<const float4*>(wp + j * kPs + k);
              e[k] = u.x; e[k + 1] = u.y; e[k + 2] = u.z; e[k + 3] = u.w;
            }
          }
#pragma unroll
          for (int k = 0; k < kRpt; ++k) add(k, e[k], v);
        }
      } else {
        for (int j = 0; j < tokens; ++j) {
          const float4 v = *reinterpret_cast<const float4*>(vp + (size_t)j * stride);
#pragma unroll
          for (int k = 0; k < kRpt; ++k) {
            const float e = wp[j * kPs + k];
            if (!(e < 0.f)) add(k, e, v);
          }
        }
      }
    }
  }
  // a row's Z over its 16 lanes; then the rows' factors or statistics
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) Z[k] += __shfl_xor_sync(0xffffffffu, Z[k], o);
  }
  const int64_t i0 = (int64_t)(slot0 + s * (int)gridDim.y + rb) * kTreeWideRows;
  const bool slot_ok = LCA_CHECK(t.err, p.n_split == 1 || i0 + kTreeWideRows <= p.slot_rows, 0xD54);
  __syncthreads();
  if (tx == 0) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t r = r0 + 2 * ty + k;
      fac[2 * ty + k] = Z[k] == 0.f ? 0.f : 1.f / Z[k];
      if (r >= rows || !slot_ok) continue;
      if (p.n_split > 1) {
        p.part_mz[2 * (i0 + 2 * ty + k)] = M[k];
        p.part_mz[2 * (i0 + 2 * ty + k) + 1] = Z[k];
      } else if (p.lse) {
        p.lse[(int64_t)b * t.T * t.H + r] = Z[k] == 0.f ? -INFINITY : kTreeLn2 * (M[k] + log2f(Z[k]));
      }
    }
  }
  __syncthreads();
  if (!act || !slot_ok) return;
#pragma unroll
  for (int k = 0; k < kRpt; ++k) {
    const int r = rg * kRpt + k;
    if (r0 + r >= rows) break;
    if (p.n_split > 1) {
      store4(p.part_o + (i0 + r) * t.d_c + 4 * g, acc[k]);
    } else {
      const float f = fac[r];
      store4(static_cast<T*>(p.out) + (q0 + r) * t.d_c + 4 * g, make_float4(acc[k].x * f, acc[k].y * f, acc[k].z * f, acc[k].w * f));
    }
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

// -lse of a row; an infinite lse marks a row that adds nothing, and -inf makes it so.  A weight is
// 2^{(x - lse) log2 e}: the difference is taken first, since lse log2 e alone would be rounded by up to
// 1e-6 where lse is above 11, and the weight with it.
__device__ __forceinline__ float mass_offset(float lse) { return isinf(lse) ? -INFINITY : -lse; }

// A position's new sum: cached tokens go on from what they had, drafted ones begin.
__device__ __forceinline__ void mass_store(const MassParams& p, int b, int pos, int n, float add) {
  if (!LCA_CHECK(p.t.err, pos >= 0 && pos < p.t.cap && pos < p.stride && b < p.t.B, 0xD55)) return;
  const int64_t i = (int64_t)b * p.stride + pos;
  float old = 0.f;
  if (pos < n && p.prev && p.decay != 0.f) old = p.decay * p.prev[i];
  p.scores[i] = old + add;
}

// grid (blocks, B): a block takes every gridDim.x-th tile of 32 tokens through all rows.
template <typename T>
__global__ void __launch_bounds__(kTreeSimtThreads) lca_mass_simt_kernel(const MassParams p) {
  extern __shared__ float tree_smem[];
  __shared__ int list[kTreeSimtTile];
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
    if (threadIdx.x < kTreeSimtTile) list[threadIdx.x] = t0 + threadIdx.x < total ? (int)tree_row(t, b, (int)t0 + threadIdx.x, 0xB04) : -1;
    __syncthreads();
    tree_stage_rows<T>(t.c, t.k, t.d_c, t.d_r, kTreeSimtTile, list, tile);
    const int pos = (int)t0 + lane;
    float sum = 0.f;
    for (int64_t r0 = 0; r0 < rows; r0 += kTreeSimtRows) {
      __syncthreads();
      tree_stage_q<T>(t, p.q_c, p.q_r, b, r0, rows, q);
      __syncthreads();
      const int64_t r = r0 + warp;
      if (r >= rows) continue;
      const float off = mass_offset(p.lse[(int64_t)b * t.T * t.H + r]);
      if (off != -INFINITY && pos < total && tree_sees(ln, tree_word(t, b, (int)(r / t.H)), pos))
        sum += exp2f((tree_dot(q + (size_t)warp * d, tile + (size_t)lane * stride, d) + off) * kTreeLog2e);
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

// The same in tiles of kTokens tokens and blocks of 32 rows.
template <typename T, int kTokens>
__global__ void __launch_bounds__(kTreeSimtThreads) lca_mass_wide_kernel(const MassParams p) {
  constexpr int J = kTokens / 16;
  extern __shared__ float tree_smem[];
  __shared__ int list[kTokens];
  const TreeBatch& t = p.t;
  const int b = blockIdx.y, tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int d = t.d_c + t.d_r, stride = d + 4;
  float* q = tree_smem;
  float* tile = q + (size_t)kTreeWideRows * stride;
  float* part = tile + (size_t)kTokens * stride;                // [16][kTokens]
  const TreeLens ln = tree_lens(t, b);
  if (ln.bad && blockIdx.x == 0 && tid == 0) input_error(t.err, 0xB03);
  const int64_t rows = (int64_t)ln.d * t.H, q0 = (int64_t)b * t.T * t.H;
  const int total = ln.n + ln.d;
  for (int64_t t0 = (int64_t)blockIdx.x * kTokens; t0 < total; t0 += (int64_t)gridDim.x * kTokens) {
    __syncthreads();
    if (tid < kTokens) list[tid] = t0 + tid < total ? (int)tree_row(t, b, (int)t0 + tid, 0xB04) : -1;
    __syncthreads();
    tree_stage_rows<T>(t.c, t.k, t.d_c, t.d_r, kTokens, list, tile);
    const bool special = t0 + kTokens > ln.n;
    float sum[J];
#pragma unroll
    for (int j = 0; j < J; ++j) sum[j] = 0.f;
    for (int64_t r0 = 0; r0 < rows; r0 += kTreeWideRows) {
      __syncthreads();
      if (tid < kTreeWideRows) list[tid] = r0 + tid < rows ? (int)(q0 + r0 + tid) : -1;
      __syncthreads();
      tree_stage_rows<T>(p.q_c, p.q_r, t.d_c, t.d_r, kTreeWideRows, list, q);
      __syncthreads();
      float x[2][J];
      tree_products<J>(q, tile, d, ty, tx, x);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int64_t r = r0 + 2 * ty + k;
        if (r >= rows) continue;
        const float off = mass_offset(p.lse[q0 + r]);
        if (off == -INFINITY) continue;
        const unsigned long long word = special ? tree_word(t, b, (int)(r / t.H)) : 0ull;
#pragma unroll
        for (int j = 0; j < J; ++j)
          if (!special || tree_sees(ln, word, (int)t0 + tx + 16 * j)) sum[j] += exp2f((x[k][j] + off) * kTreeLog2e);
      }
    }
#pragma unroll
    for (int j = 0; j < J; ++j) part[ty * kTokens + tx + 16 * j] = sum[j];
    __syncthreads();
    if (tid < kTokens && t0 + tid < total) {
      float a = 0.f;
#pragma unroll
      for (int w = 0; w < 16; ++w) a += part[w * kTokens + tid];
      mass_store(p, b, (int)t0 + tid, ln.n, a);
    }
  }
}

}  // namespace lca
