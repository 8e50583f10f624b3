// tree_capi.cu -- the part of include/lca.h for drafted tokens and eviction:
// tree attention, accumulated attention weights, the choice of the rows to
// keep and their compaction.  As in lca_capi.cu no exception crosses the ABI,
// nothing aborts, and argument errors are reported before anything is launched.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>

#include "evict_kernel.cuh"
#include "lca.h"
#include "mass_tc_kernel.cuh"
#include "plan.cuh"
#include "tree_common.cuh"
#include "tmap.cuh"
#include "tree_simt_kernel.cuh"
#include "tree_tc_kernel.cuh"

namespace {

using lca::TreeBatch;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

constexpr size_t kMaxSmem = 232448 - 1024;     // dynamic, beside what the CUDA-core kernels have besides

// ---------------------------------------------------------------- workspace
// [a record for each sequence][(M, Z) of every slot row][O of every slot row], each part
// 256-byte aligned.
struct Workspace {
  int64_t slot_rows;      // rows of partials
  size_t mz, o, bytes;    // offsets, and the whole
};

// Query rows of a block of the CUDA-core kernels: 32 where there are more than 8 and shared memory holds them
// beside a tile (d_c + d_r up to about 880).
int simt_rows(const lca_plan* p, int T) {
  const bool wide = (int64_t)T * p->H > lca::kTreeSimtRows &&
                    lca::tree_wide_smem(p->d_c, p->d_r, lca::tree_wide_tokens(p->d_c, p->d_r)) <= kMaxSmem;
  return wide ? lca::kTreeWideRows : lca::kTreeSimtRows;
}

// Parts the CUDA-core kernel cuts each sequence into: about four CTAs per SM (two are resident at once) over B and
// the row blocks; one part writes its output itself.  Half as many parts, one wave, are 8% faster for sequences of
// one length and 25% slower for lengths from n / 4 to n, whose longest then sets the time.
int64_t simt_parts(const lca_plan* p, int T) {
  const int64_t units = (int64_t)p->B * ceil_div((int64_t)T * p->H, simt_rows(p, T));
  const int64_t most = std::min<int64_t>(lca::kTreeMaxParts, ceil_div(p->max_L, lca::kTreeSimtTile));
  return std::max<int64_t>(1, std::min<int64_t>(4LL * p->num_sms / units, most));
}

// The tensor-core kernels' shape.
bool tc_ok(const lca_plan* p) { return p->dt == LCA_BF16 && p->d_c == lca::ttc::kDC && p->d_r == lca::ttc::kDR; }

// Query rows of a unit: the least of 16, 32, 64 that holds a sequence's rows, 64 where none does.
int tc_rows(const lca_plan* p, int T) {
  const int64_t r = (int64_t)T * p->H;
  return r <= 16 ? 16 : r <= 32 ? 32 : 64;
}

Workspace workspace_of(const lca_plan* p, int T) {
  Workspace w;
  const int64_t parts = simt_parts(p, T);
  w.slot_rows = parts > 1 ? parts * p->B * round_up((int64_t)T * p->H, simt_rows(p, T)) : 0;
  if (tc_ok(p)) w.slot_rows = std::max<int64_t>(w.slot_rows, (int64_t)lca::kTreeMaxWaves * p->num_sms * tc_rows(p, T));
  static_assert(sizeof(lca::mtc::Split) <= sizeof(lca::TreeSplit), "one record's room");
  w.mz = (size_t)round_up((int64_t)p->B * sizeof(lca::TreeSplit), 256);
  w.o = w.mz + (size_t)round_up(w.slot_rows * 2 * sizeof(float), 256);
  w.bytes = w.o + (size_t)w.slot_rows * p->d_c * sizeof(float);
  return w;
}

// ---------------------------------------------------------------- argument checks
lca_status check_plan(const lca_plan* p) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return LCA_ERR_CUDA;
  return dev == p->device ? LCA_OK : LCA_ERR_PLAN_MISMATCH;
}

// The cache arguments common to the entry points, and their bound on lengths.
lca_status check_cache(const lca_plan* p, const void* c_pool, const void* k_pool, int64_t num_pages, int page_size,
                       const int32_t* block_table, int64_t max_pages, TreeBatch* t) {
  if (!p || !c_pool || !k_pool || num_pages < 1 || page_size < 1 || max_pages < 1) return LCA_ERR_INVALID_ARG;
  if (block_table ? page_size % 64 != 0 : num_pages < p->B) return LCA_ERR_INVALID_ARG;
  if ((uint64_t)num_pages > (uint64_t)INT32_MAX / (uint64_t)page_size) return LCA_ERR_UNSUPPORTED;
  std::memset(t, 0, sizeof(*t));
  t->c = c_pool;
  t->k = k_pool;
  t->num_pages = num_pages;
  t->page_size = page_size;
  t->table = block_table;
  t->max_pages = block_table ? max_pages : 1;
  t->B = p->B;
  t->H = p->H;
  t->d_c = p->d_c;
  t->d_r = p->d_r;
  const int64_t rows = t->max_pages > INT32_MAX / page_size ? INT32_MAX : t->max_pages * page_size;
  t->cap = std::min<int64_t>(std::min<int64_t>(p->max_L, rows), INT32_MAX - 4096);
  t->err = p->err;
  return LCA_OK;
}

lca_status check_batch(const lca_plan* p, int n_draft, const int32_t* seq_lens, const int32_t* draft_lens,
                       const uint64_t* mask, TreeBatch* t) {
  if (!seq_lens || n_draft < 1 || n_draft > lca::kTreeMaxDraft) return LCA_ERR_INVALID_ARG;
  if ((int64_t)p->B * n_draft * p->H > INT32_MAX || p->B > 65535) return LCA_ERR_UNSUPPORTED;
  if (!aligned(seq_lens, 4) || !aligned(draft_lens, 4) || !aligned(mask, 8) || !aligned(t->table, 4))
    return LCA_ERR_ALIGNMENT;
  t->T = n_draft;
  t->seq_lens = seq_lens;
  t->draft_lens = draft_lens;
  t->mask = reinterpret_cast<const unsigned long long*>(mask);
  return LCA_OK;
}

// Let a kernel have up to `most` bytes of shared memory, once per device (so that no call lowers what another
// one, in another thread, is about to launch with).
template <auto kKernel>
bool allow_smem(int device, size_t most) {
  static std::atomic<uint64_t> done{0};
  const uint64_t bit = device >= 0 && device < 64 ? uint64_t(1) << device : 0;
  if (done.load(std::memory_order_acquire) & bit) return true;
  if (cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) != cudaSuccess) return false;
  done.fetch_or(bit, std::memory_order_acq_rel);
  return true;
}

lca_status launched() { return cudaGetLastError() == cudaSuccess ? LCA_OK : LCA_ERR_CUDA; }

// The merge of the parts, a programmatic dependent of the kernel that wrote
// them; four warps share a run of dims where all CTAs are resident at once.
template <typename T, int kSplit>
lca_status launch_merge_split(const lca_plan* p, const lca::TreeMergeParams& mp, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  const int64_t ctas = (int64_t)mp.t.T * mp.t.H * ceil_div(mp.t.d_c, lca::tree_merge_dims(kSplit));
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(ctas, ceil_div(16LL * p->num_sms, mp.t.B)), (unsigned)mp.t.B, 1);
  cfg.blockDim = dim3(lca::kTreeMergeThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, lca::lca_tree_merge_kernel<T, kSplit>, mp) == cudaSuccess ? LCA_OK : LCA_ERR_CUDA;
}

template <typename T>
lca_status launch_merge(const lca_plan* p, const lca::TreeMergeParams& mp, cudaStream_t stream) {
  const int64_t shared = (int64_t)mp.t.B * mp.t.T * mp.t.H * ceil_div(mp.t.d_c, lca::tree_merge_dims(4));
  return shared <= 8LL * p->num_sms ? launch_merge_split<T, 4>(p, mp, stream) : launch_merge_split<T, 1>(p, mp, stream);
}

template <typename T, int kTokens, int kRpt>
lca_status launch_tree_wide(const lca_plan* p, const lca::TreeSimtParams& sp, dim3 grid, cudaStream_t stream) {
  const size_t smem = lca::tree_wide_smem(sp.t.d_c, sp.t.d_r, kTokens);
  if (smem > kMaxSmem) return LCA_ERR_UNSUPPORTED;
  if (!allow_smem<lca::lca_tree_wide_kernel<T, kTokens, kRpt>>(p->device, kMaxSmem)) return LCA_ERR_CUDA;
  lca::lca_tree_wide_kernel<T, kTokens, kRpt><<<grid, lca::kTreeSimtThreads, smem, stream>>>(sp);
  return launched();
}

template <typename T>
lca_status run_tree_simt(const lca_plan* p, const TreeBatch& t, const void* q_c, const void* q_r, void* out,
                         float* lse, uint8_t* ws, const Workspace& w, cudaStream_t stream) {
  lca::TreeSimtParams sp = {};
  sp.t = t;
  sp.q_c = q_c;
  sp.q_r = q_r;
  sp.n_split = (int)simt_parts(p, t.T);
  sp.split = reinterpret_cast<lca::TreeSplit*>(ws);
  sp.part_mz = reinterpret_cast<float*>(ws + w.mz);
  sp.part_o = reinterpret_cast<float*>(ws + w.o);
  sp.slot_rows = w.slot_rows;
  sp.out = out;
  sp.lse = lse;
  const int rows = simt_rows(p, t.T);
  const dim3 grid((unsigned)sp.n_split, (unsigned)ceil_div((int64_t)t.T * t.H, rows), (unsigned)t.B);
  lca_status st;
  if (rows == lca::kTreeSimtRows) {
    const size_t smem = lca::tree_simt_smem(t.d_c, t.d_r);
    if (smem > kMaxSmem) return LCA_ERR_UNSUPPORTED;
    if (!allow_smem<lca::lca_tree_simt_kernel<T>>(p->device, kMaxSmem)) return LCA_ERR_CUDA;
    lca::lca_tree_simt_kernel<T><<<grid, lca::kTreeSimtThreads, smem, stream>>>(sp);
    st = launched();
  } else if (lca::tree_wide_tokens(t.d_c, t.d_r) == 64) {
    st = t.d_c <= 64 ? launch_tree_wide<T, 64, 2>(p, sp, grid, stream) : t.d_c <= 128 ? launch_tree_wide<T, 64, 4>(p, sp, grid, stream)
                                                                                     : launch_tree_wide<T, 64, 8>(p, sp, grid, stream);
  } else {
    st = t.d_c <= 256 ? launch_tree_wide<T, 32, 8>(p, sp, grid, stream) : t.d_c <= 512 ? launch_tree_wide<T, 32, 16>(p, sp, grid, stream)
                                                                                      : launch_tree_wide<T, 32, 32>(p, sp, grid, stream);
  }
  if (st != LCA_OK) return st;
  lca::TreeMergeParams mp = {};
  mp.t = t;
  mp.part_o = sp.part_o;
  mp.part_mz = sp.part_mz;
  mp.split = sp.split;
  mp.slot_rows = w.slot_rows;
  mp.rows_per_block = rows;
  mp.direct = sp.n_split == 1;
  mp.out = out;
  mp.lse = lse;
  return launch_merge<T>(p, mp, stream);
}

template <int N>
lca_status run_tree_tc(const lca_plan* p, const TreeBatch& t, const void* q_c, const void* q_r, void* out, float* lse,
                       uint8_t* ws, const Workspace& w, cudaStream_t stream) {
  namespace ttc = lca::ttc;
  ttc::Params tp;
  std::memset(&tp, 0, sizeof(tp));
  const uint64_t rows = (uint64_t)t.num_pages * (uint64_t)t.page_size, qrows = (uint64_t)t.B * t.T * t.H;
  if (!lca::make_map(&tp.tm_c, t.c, ttc::kDC, rows, 64) || !lca::make_map(&tp.tm_k, t.k, ttc::kDR, rows, 64) ||
      !lca::make_map(&tp.tm_qc, q_c, ttc::kDC, qrows, N) || !lca::make_map(&tp.tm_qr, q_r, ttc::kDR, qrows, N))
    return LCA_ERR_CUDA;
  tp.t = t;
  tp.G = std::min(p->num_ctas > 0 ? p->num_ctas : p->num_sms, lca::kTreeMaxParts / lca::kTreeMaxWaves);
  tp.split = reinterpret_cast<lca::TreeSplit*>(ws);
  tp.part_mz = reinterpret_cast<float*>(ws + w.mz);
  tp.part_o = reinterpret_cast<float*>(ws + w.o);
  tp.slots = w.slot_rows / N;
  tp.out = static_cast<__nv_bfloat16*>(out);
  tp.lse = lse;
  tp.timeout_ns = p->timeout_ns;
  tp.debug_skip_load = p->debug_skip_load;
  if (!allow_smem<ttc::lca_tree_tc_kernel<N>>(p->device, ttc::Layout<N>::kAlloc)) return LCA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)tp.G, 1, 1);
  cfg.blockDim = dim3(ttc::Layout<N>::kThreads, 1, 1);
  cfg.dynamicSmemBytes = ttc::Layout<N>::kAlloc;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, ttc::lca_tree_tc_kernel<N>, tp) != cudaSuccess) return LCA_ERR_CUDA;
  lca::TreeMergeParams mp = {};
  mp.t = t;
  mp.part_o = tp.part_o;
  mp.part_mz = tp.part_mz;
  mp.split = tp.split;
  mp.slot_rows = w.slot_rows;
  mp.rows_per_block = N;
  mp.direct = true;
  mp.out = out;
  mp.lse = lse;
  return launch_merge<__nv_bfloat16>(p, mp, stream);
}

template <typename T>
lca_status run_mass_simt(const lca_plan* p, const lca::MassParams& mp, cudaStream_t stream) {
  const int tokens = lca::tree_wide_tokens(mp.t.d_c, mp.t.d_r);
  const bool narrow = simt_rows(p, mp.t.T) == lca::kTreeSimtRows;
  const size_t smem = narrow ? lca::tree_simt_smem(mp.t.d_c, mp.t.d_r) : lca::tree_wide_smem(mp.t.d_c, mp.t.d_r, tokens);
  if (smem > kMaxSmem) return LCA_ERR_UNSUPPORTED;
  const int64_t tiles = ceil_div(mp.t.cap, narrow ? lca::kTreeSimtTile : tokens);
  const dim3 grid((unsigned)std::min<int64_t>(tiles, std::max<int64_t>(1, 8LL * p->num_sms / p->B)), (unsigned)p->B);
  if (narrow) {
    if (!allow_smem<lca::lca_mass_simt_kernel<T>>(p->device, kMaxSmem)) return LCA_ERR_CUDA;
    lca::lca_mass_simt_kernel<T><<<grid, lca::kTreeSimtThreads, smem, stream>>>(mp);
  } else if (tokens == 64) {
    if (!allow_smem<lca::lca_mass_wide_kernel<T, 64>>(p->device, kMaxSmem)) return LCA_ERR_CUDA;
    lca::lca_mass_wide_kernel<T, 64><<<grid, lca::kTreeSimtThreads, smem, stream>>>(mp);
  } else {
    if (!allow_smem<lca::lca_mass_wide_kernel<T, 32>>(p->device, kMaxSmem)) return LCA_ERR_CUDA;
    lca::lca_mass_wide_kernel<T, 32><<<grid, lca::kTreeSimtThreads, smem, stream>>>(mp);
  }
  return launched();
}

// Up to 128 rows a sequence the queries stay in shared memory, in blocks of N;
// with more they stream past each tile of the cache.
template <int N, bool kStream>
lca_status run_mass_tc(const lca_plan* p, const lca::MassParams& m, uint8_t* ws, const Workspace& w,
                       cudaStream_t stream) {
  namespace mtc = lca::mtc;
  const TreeBatch& t = m.t;
  mtc::Params mp;
  std::memset(&mp, 0, sizeof(mp));
  const uint64_t rows = (uint64_t)t.num_pages * (uint64_t)t.page_size, qrows = (uint64_t)t.B * t.T * t.H;
  if (!lca::make_map(&mp.tm_c, t.c, lca::ttc::kDC, rows, 64) || !lca::make_map(&mp.tm_k, t.k, lca::ttc::kDR, rows, 64) ||
      !lca::make_map(&mp.tm_qc, m.q_c, lca::ttc::kDC, qrows, N) || !lca::make_map(&mp.tm_qr, m.q_r, lca::ttc::kDR, qrows, N))
    return LCA_ERR_CUDA;
  mp.m = m;
  mp.G = p->num_ctas > 0 ? p->num_ctas : p->num_sms;
  mp.split = reinterpret_cast<mtc::Split*>(ws);
  mp.part = reinterpret_cast<float*>(ws + w.o);
  mp.timeout_ns = p->timeout_ns;
  mp.debug_skip_load = p->debug_skip_load;
  if (!allow_smem<mtc::lca_mass_tc_kernel<N, kStream>>(p->device, mtc::Layout<N, kStream>::kAlloc)) return LCA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)mp.G, 1, 1);
  cfg.blockDim = dim3(mtc::kThreads, 1, 1);
  cfg.dynamicSmemBytes = mtc::Layout<N, kStream>::kAlloc;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, mtc::lca_mass_tc_kernel<N, kStream>, mp) != cudaSuccess) return LCA_ERR_CUDA;
  if (!kStream) return LCA_OK;                       // one row block: every tile is one CTA's
  mtc::FinishParams fp = {};
  fp.m = m;
  fp.G = mp.G;
  fp.part = mp.part;
  fp.split = mp.split;
  const int64_t tiles = ceil_div(t.cap, lca::kTreeTile);
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(tiles, std::max<int64_t>(1, 4LL * p->num_sms / t.B)), (unsigned)t.B, 1);
  cfg.blockDim = dim3(lca::kTreeTile, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, mtc::lca_mass_finish_kernel, fp) == cudaSuccess ? LCA_OK : LCA_ERR_CUDA;
}

}  // namespace

extern "C" {

int64_t lca_tree_workspace(const lca_plan* p, int n_draft) {
  if (!p || n_draft < 1 || n_draft > lca::kTreeMaxDraft) return -1;
  // The CUDA-core kernels want less with more drafted tokens where those make row blocks enough: whoever asks for
  // the largest tree has room for every smaller one.
  size_t most = 0;
  for (int T = 1; T <= n_draft; ++T) most = std::max(most, workspace_of(p, T).bytes);
  return (int64_t)most;
}

lca_status lca_tree_decode(lca_plan* p, const void* q_c, const void* q_r, int n_draft, const void* c_pool,
                           const void* k_pool, int64_t num_pages, int page_size, const int32_t* block_table,
                           int64_t max_pages, const int32_t* seq_lens, const int32_t* draft_lens,
                           const uint64_t* mask, void* out, float* lse, void* workspace, int64_t workspace_bytes,
                           void* stream) {
  TreeBatch t;
  lca_status st = check_cache(p, c_pool, k_pool, num_pages, page_size, block_table, max_pages, &t);
  if (st != LCA_OK) return st;
  if (!q_c || !q_r || !out || !workspace) return LCA_ERR_INVALID_ARG;
  if ((st = check_batch(p, n_draft, seq_lens, draft_lens, mask, &t)) != LCA_OK) return st;
  const Workspace w = workspace_of(p, n_draft);
  if (workspace_bytes < (int64_t)w.bytes) return LCA_ERR_INVALID_ARG;
  if (!aligned(q_c, 16) || !aligned(q_r, 16) || !aligned(c_pool, 16) || !aligned(k_pool, 16) || !aligned(out, 16) ||
      !aligned(lse, 4) || !aligned(workspace, 256))
    return LCA_ERR_ALIGNMENT;
  if ((st = check_plan(p)) != LCA_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int pref = p->force_simt ? 1 : p->kernel_pref;      // 1 CUDA-core, 2 tcgen05
  if (pref > 2 || (pref == 2 && !tc_ok(p))) return LCA_ERR_UNSUPPORTED;
  if (tc_ok(p) && pref != 1) {
    switch (tc_rows(p, n_draft)) {
      case 16: return run_tree_tc<16>(p, t, q_c, q_r, out, lse, ws, w, s);
      case 32: return run_tree_tc<32>(p, t, q_c, q_r, out, lse, ws, w, s);
      default: return run_tree_tc<64>(p, t, q_c, q_r, out, lse, ws, w, s);
    }
  }
  if (p->dt == LCA_F32) return run_tree_simt<float>(p, t, q_c, q_r, out, lse, ws, w, s);
  return run_tree_simt<__nv_bfloat16>(p, t, q_c, q_r, out, lse, ws, w, s);
}

lca_status lca_attn_mass(lca_plan* p, const void* q_c, const void* q_r, int n_draft, const void* c_pool,
                         const void* k_pool, int64_t num_pages, int page_size, const int32_t* block_table,
                         int64_t max_pages, const int32_t* seq_lens, const int32_t* draft_lens, const uint64_t* mask,
                         const float* lse, const float* prev, float decay, float* scores, int64_t score_stride,
                         void* workspace, int64_t workspace_bytes, void* stream) {
  lca::MassParams mp = {};
  lca_status st = check_cache(p, c_pool, k_pool, num_pages, page_size, block_table, max_pages, &mp.t);
  if (st != LCA_OK) return st;
  if (!q_c || !q_r || !lse || !scores || !workspace || score_stride < 1) return LCA_ERR_INVALID_ARG;
  if ((st = check_batch(p, n_draft, seq_lens, draft_lens, mask, &mp.t)) != LCA_OK) return st;
  const Workspace w = workspace_of(p, n_draft);
  if (workspace_bytes < (int64_t)w.bytes) return LCA_ERR_INVALID_ARG;
  if (!aligned(q_c, 16) || !aligned(q_r, 16) || !aligned(c_pool, 16) || !aligned(k_pool, 16) || !aligned(lse, 4) ||
      !aligned(prev, 4) || !aligned(scores, 4) || !aligned(workspace, 256))
    return LCA_ERR_ALIGNMENT;
  if ((st = check_plan(p)) != LCA_OK) return st;
  mp.t.cap = std::min(mp.t.cap, score_stride);
  mp.q_c = q_c;
  mp.q_r = q_r;
  mp.lse = lse;
  mp.prev = prev;
  mp.scores = scores;
  mp.stride = score_stride;
  mp.decay = decay;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int pref = p->force_simt ? 1 : p->kernel_pref;
  if (pref > 2 || (pref == 2 && !tc_ok(p))) return LCA_ERR_UNSUPPORTED;
  if (tc_ok(p) && pref != 1) {
    const int64_t r = (int64_t)n_draft * p->H;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    if (r <= 16) return run_mass_tc<16, false>(p, mp, ws, w, s);
    if (r <= 32) return run_mass_tc<32, false>(p, mp, ws, w, s);
    if (r <= 64) return run_mass_tc<64, false>(p, mp, ws, w, s);
    if (r <= 128) return run_mass_tc<128, false>(p, mp, ws, w, s);
    return run_mass_tc<128, true>(p, mp, ws, w, s);
  }
  return p->dt == LCA_F32 ? run_mass_simt<float>(p, mp, s) : run_mass_simt<__nv_bfloat16>(p, mp, s);
}

lca_status lca_evict_select(lca_plan* p, const float* scores, int64_t score_stride, const int32_t* seq_lens,
                            int64_t n_sink, int64_t n_recent, int64_t budget, int32_t* kept, int32_t* kept_lens,
                            void* stream) {
  if (!p || !scores || !seq_lens || !kept || !kept_lens || score_stride < 1 || n_sink < 0 || n_recent < 0 ||
      budget < 1 || budget > INT32_MAX || n_sink > budget || n_recent > budget - n_sink)
    return LCA_ERR_INVALID_ARG;
  if (!aligned(scores, 4) || !aligned(seq_lens, 4) || !aligned(kept, 4) || !aligned(kept_lens, 4))
    return LCA_ERR_ALIGNMENT;
  const lca_status st = check_plan(p);
  if (st != LCA_OK) return st;
  lca::SelectParams sp = {};
  sp.scores = scores;
  sp.stride = score_stride;
  sp.seq_lens = seq_lens;
  sp.B = p->B;
  sp.cap = std::min<int64_t>(std::min<int64_t>(p->max_L, score_stride), 1 << 30);
  sp.n_sink = (int)n_sink;
  sp.n_recent = (int)n_recent;
  sp.budget = (int)budget;
  sp.kept = kept;
  sp.kept_lens = kept_lens;
  sp.err = p->err;
  // One CTA for up to 4096 rows, twice as many for twice the rows, up to a cluster of 8.  Measured with 1 / 2 / 4 / 8
  // CTAs, 8 sequences, a quarter kept (us): 4096 rows 11.5 / 10.8 / 10.1 / 10.6, 8192 14.6 / 12.3 / 11.3 / 11.3, 16384
  // 19.8 / 15.1 / 12.6 / 12.2, 32768 31 / 20 / 15.1 / 13.2, 131072 304 / 115 / 36 / 25.  The rule does not look at B:
  // where all CTAs are not resident at once fewer are faster (32 x 32768: 37 with 8, 16 with 4; 128 x 8192: 23 with
  // 2, 15 with 1).
  sp.ctas = 1;
  while (sp.ctas < lca::kSelectMaxCtas && sp.cap > 4096LL * sp.ctas) sp.ctas *= 2;
  if (p->B > INT32_MAX / lca::kSelectMaxCtas) return LCA_ERR_UNSUPPORTED;
  const size_t smem = lca::select_smem(lca::select_each(sp.cap, sp.ctas));
  if (!allow_smem<lca::lca_select_kernel>(p->device, lca::select_smem(lca::kSelectKeep))) return LCA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p->B * sp.ctas), 1, 1);
  cfg.blockDim = dim3(lca::kSelectThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)sp.ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, lca::lca_select_kernel, sp) == cudaSuccess ? LCA_OK : LCA_ERR_CUDA;
}

lca_status lca_cache_compact(lca_plan* p, void* c_pool, void* k_pool, int64_t num_pages, int page_size,
                             const int32_t* block_table, int64_t max_pages, const int32_t* src, int64_t src_stride,
                             const int32_t* n_src, const int32_t* dst0, float* scores, int64_t score_stride,
                             void* stream) {
  lca::CompactParams cp = {};
  lca_status st = check_cache(p, c_pool, k_pool, num_pages, page_size, block_table, max_pages, &cp.t);
  if (st != LCA_OK) return st;
  if (!src || !n_src || src_stride < 1 || src_stride > INT32_MAX || (scores && score_stride < 1)) return LCA_ERR_INVALID_ARG;
  if (p->B > 65535) return LCA_ERR_UNSUPPORTED;
  if (!aligned(c_pool, 16) || !aligned(k_pool, 16) || !aligned(block_table, 4) || !aligned(src, 4) ||
      !aligned(n_src, 4) || !aligned(dst0, 4) || !aligned(scores, 4))
    return LCA_ERR_ALIGNMENT;
  if ((st = check_plan(p)) != LCA_OK) return st;
  if (scores) cp.t.cap = std::min(cp.t.cap, score_stride);
  cp.elem = p->dt == LCA_F32 ? 4 : 2;
  cp.src = src;
  cp.src_stride = src_stride;
  cp.n_src = n_src;
  cp.dst0 = dst0;
  cp.scores = scores;
  cp.score_stride = score_stride;
  int l = 1;
  while (l < 31 && (1LL << l) < page_size) ++l;
  cp.page_mul = (uint32_t)((uint64_t(1) << (31 + l)) / (uint64_t)page_size + 1);
  cp.page_shift = l - 1;
  // Narrow strips while that makes no second block for an SM; wide ones, in blocks of 512 threads, while all of
  // those are resident; else of 256.
  const int64_t row_c = (int64_t)p->d_c * cp.elem / 16, row_k = (int64_t)p->d_r * cp.elem / 16;     // in 16 bytes
  auto strips = [&](int strip) {
    cp.strips_c = (int)ceil_div(row_c, strip);
    cp.strips_k = (int)ceil_div(row_k, strip);
    return (int64_t)(cp.strips_c + cp.strips_k + (scores ? 1 : 0)) * p->B <= p->num_sms;
  };
  const bool narrow = strips(lca::kCompactNarrow);
  const bool few = narrow || strips(lca::kCompactWide);
  const dim3 grid((unsigned)(cp.strips_c + cp.strips_k + (scores ? 1 : 0)), (unsigned)p->B);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (narrow) lca::lca_compact_kernel<lca::kCompactNarrow, 512><<<grid, 512, 0, s>>>(cp);
  else if (few) lca::lca_compact_kernel<lca::kCompactWide, 512><<<grid, 512, 0, s>>>(cp);
  else lca::lca_compact_kernel<lca::kCompactWide, 256><<<grid, 256, 0, s>>>(cp);
  return launched();
}

}  // extern "C"
