// tree_tc_kernel.cuh -- draft-tree attention over the latent cache with tcgen05
// tensor cores (bf16, d_c = 512, d_r = 64).
//
// One unit of work is a block of N query rows (node, head) of a sequence and a
// run of 128-token tiles (tree_schedule.cuh).  Per tile
//   S^T[128 tokens x N rows] = [C | K]_tile . [q_c | q_r]^T     36 MMAs, M = 128, K = 16
//   P^T = 2^{S^T log2 e - M}                                    softmax warps, a token a thread
//   O^T[512 x N] += C_tile^T . P^T                              32 MMAs, in TMEM
// Tokens are the M side of both products, so the same shared-memory tile is
// the A operand twice: K-major for S, MN-major (its transpose) for O.  A token
// is one thread's: its running sums stay in that thread until the unit ends.
//
// Why this orientation and N = 64.  An M = 128 MMA of K = 16 takes max(44.7,
// 32 + N / 4 cycles for its operands' shared-memory reads) (measured: N = 16, 32:
// 44.7; 64: 48; 128: 64), so N = 64 gives 3264 cycles for 64 x 128 x 1088 MACs
// (67% of the peak of 64 cycles at N = 128).  With rows on the M side a CTA
// would need 128 rows x 512 dims of fp32 for O, all of TMEM, or a cluster that
// exchanges S or P for every tile; O^T of 64 rows takes 256 columns and no
// exchange.
//
// Shared memory: for N = 64 four 32 KB slots hold one tile's C (a slot: 128
// dims), 16 KB its K, and Q the rest, so a tile is resident once and the next
// one streams into the slots as O's MMAs release them, slot by slot; P takes
// K's place, which is read by then.  N <= 32 has a fifth slot and P its own.
//
// The reference M of a row rises only when a logit exceeds it by more than 2^8
// (then Z and O^T are scaled).  Whether one does is not agreed on beforehand: a
// barrier of the softmax warps cost about 500 cycles a tile.  A thread that
// meets such a logit says so beside its arrival; the MMA issuer, which waits for
// all arrivals anyway, then hands the tile back instead of going on to O, and
// the softmax warps raise M and form P again.  (A unit's first tile always
// raises M and does so at once.)  A tile's weights join Z when the next event
// shows that it was not handed back.
//
// Tokens a row does not see get weight 0; because 0 x NaN is not 0, rows of
// the tile that hold no token are zeroed in shared memory, and a drafted row
// whose C holds an infinity or NaN is zeroed too and makes the sums of the rows
// that see it NaN.  K is in the logits alone, which are selected and not
// multiplied, so an infinite key needs no more.
//
// Roles: warp 0 finds the units and loads, warp 1 issues the MMAs, the other 8 (N = 64: 16) do the
// softmax: a warp has 32 tokens (a TMEM lane quarter) and 8 or 16 of the rows.  Every wait
// is bounded: when one runs out the CTA records it, lets its copies and MMAs
// land, frees TMEM and exits.
#pragma once
#include <cuda.h>

#include "checks.cuh"
#include "ptx.cuh"
#include "tree_common.cuh"
#include "tree_events.cuh"
#include "tree_schedule.cuh"

namespace lca {
namespace ttc {

constexpr int kDC = 512, kDR = 64;
constexpr int kChunk = 128 * 128;           // [128 tokens][64 bf16], 128-byte swizzle
constexpr int kSlot = 2 * kChunk;           // 128 latent dims of a tile
constexpr int kMaxSlots = 5;
// The tensor core cuts off where it adds.  Over a logit's 36 additions the partial sums lead up to the logit x on
// average in equal steps, so what is cut off grows with x: measured -4.3e-7 x for random keys, -6.4e-7 x for keys
// along the query, with half that beside it.  3 units of 2^-23 make up for most of the first (error of a logit of
// 2.4: 1.2e-6 before, 0.7e-6 after), in factors that are applied anyway.  A logit that is formed exactly pays for
// it: 3.6e-7 x too much.
constexpr float kLogitScale = 1.f + 3.f / 8388608.f;
constexpr float kLog2eS = (float)(1.4426950408889634 * (1.0 + 3.0 / 8388608.0));
constexpr int kSeqs = 896;                  // sequences whose work is kept in shared memory
// M of a row with "no token yet", and its least: finite, so that differences of it are, and such that a weight
// 2^{x log2 e - M}, whose M is the rounded product, stays in range where x is the maximum (off by up to 2^4 here).
// With -1e30 rows whose first tile held nothing but logits of -5e14 gave NaN.
constexpr float kEmpty = -134217728.f;
constexpr float kRaise = 8.f;
constexpr int kErrTimeout = 1;
constexpr int kProbes = 64;
constexpr uint32_t kColO = 0, kColS = 256, kTmemCols = 512;

template <int N>
struct Layout {
  static constexpr bool kAlias = N == 64;              // P in K's place
  static constexpr int kSoftmaxWarps = N == 64 ? 16 : 8;
  static constexpr int kThreads = 32 * (2 + kSoftmaxWarps);
  static constexpr int kSlots = N == 64 ? 4 : 5;
  static constexpr int kQChunk = N * 128;
  static constexpr int kOffK = kSlots * kSlot;
  static constexpr int kOffQ = kOffK + kChunk;
  static constexpr int kOffP = kAlias ? kOffK : kOffQ + 9 * kQChunk;
  static constexpr int kOffWord = kOffQ + 9 * kQChunk + (kAlias ? 0 : 128 * N * 2);   // mask words of the rows
  static constexpr int kOffRed = kOffWord + 16 * N;    // [2][N], used in turn; float [2][4][N], used in turn
  static constexpr int kOffM = kOffRed + 32 * N;       // float2 [N]: the rows' (M, Z)
  static constexpr int kOffBar = kOffM + 8 * N;
  static constexpr int kBars = 2 * kMaxSlots + 11;
  static constexpr int kOffMisc = kOffBar + 8 * kBars; // TMEM address, abort, S of k waves; nodes with a broken row;
  static constexpr int kOffUnit = kOffMisc + 48;       // the event whose tile has to come back, the event it did
  static constexpr int kOffSeq = kOffUnit + 64;        // Unit [2], used in turn
  static constexpr int kBytes = kOffSeq + 4 * kSeqs;   // u32 [kSeqs]: sequences' tiles and drafted tokens
  static constexpr int kAlloc = kBytes + 1024;         // slack for the 1 KB alignment
  static_assert(kAlloc <= 232448, "shared memory of one CTA");
};

struct Params {
  CUtensorMap tm_c, tm_k;       // pools, box [64 rows][64]
  CUtensorMap tm_qc, tm_qr;     // queries as [B T H rows][..], box [N rows][64]
  TreeBatch t;
  int G;                        // CTAs
  float* part_o;                // [slots][N][512]
  float* part_mz;               // [slots][N][2]
  TreeSplit* split;
  int64_t slots;
  __nv_bfloat16* out;
  float* lse;
  uint64_t timeout_ns;
  int debug_skip_load;
};

// A unit as the loading warp, which finds it, writes it down for the others.
struct Unit {
  TreeUnit un;
  int n, d;                     // its sequence's lengths
};

struct Wait {
  volatile int* abort;
  int* err;
  uint64_t timeout_ns;
};

__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, const Wait& w, int where, bool honour) {
  const uint64_t t0 = ptx::globaltimer_ns();
  for (uint32_t spin = 1;; ++spin) {
    if (ptx::mbar_try_wait_sleep(bar, parity, 100)) return true;
    if (honour && *w.abort) return false;
    if ((spin & 7u) == 0 && ptx::globaltimer_ns() - t0 > w.timeout_ns) {
      *w.abort = 1;
      if (atomicOr(w.err, kErrTimeout) == 0) atomicExch(w.err + 1, where);
      return false;
    }
  }
}
// A bounded wait of one thread; `warp_wait` the same for a whole warp, which leaves it together.  Plain probes
// first: one with a suspend-time hint may wake late, and these hand-offs set the pace.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, const Wait& w, int where, bool honour = true) {
#pragma unroll 1
  for (int i = 0; i < kProbes; ++i)
    if (ptx::mbar_try_wait(bar, parity)) return true;
  return wait_slow(bar, parity, w, where, honour);
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const Wait& w, int where) {
  return __all_sync(0xffffffffu, wait(bar, parity, w, where));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <int C>
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&v)[C]) {
  if constexpr (C == 32) ptx::tmem_ld32(addr, v);
  else if constexpr (C == 16) ptx::tmem_ld16(addr, v);
  else ptx::tmem_ld8(addr, v);
}
// Reduces C values of each lane over the warp's 32 lanes, halving what is held with every exchange (C - 1
// exchanges instead of 5 C): the return value is column lane / (32 / C)'s result.
template <int C, class Op>
__device__ __forceinline__ float fold(const float (&v)[C], int lane, Op op) {
  float h[C / 2];
  const bool up = lane & 16;
#pragma unroll
  for (int i = 0; i < C / 2; ++i)
    h[i] = op(up ? v[i + C / 2] : v[i], __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + C / 2], 16));
  int off = 8;
#pragma unroll
  for (int n = C / 4; n > 0; n /= 2, off /= 2) {
    const bool u = lane & off;
#pragma unroll
    for (int i = 0; i < C / 4; ++i)
      if (i < n) h[i] = op(u ? h[i + n] : h[i], __shfl_xor_sync(0xffffffffu, u ? h[i] : h[i + n], off));
  }
#pragma unroll
  for (; off > 0; off /= 2) h[0] = op(h[0], __shfl_xor_sync(0xffffffffu, h[0], off));
  return h[0];
}

// True if one of the 8 bf16 in `u` is an infinity or NaN.
__device__ __forceinline__ bool any_nonfinite(uint4 u) {
  auto bad = [](uint32_t x) { return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u; };
  return bad(u.x) || bad(u.y) || bad(u.z) || bad(u.w);
}

template <int N>
__global__ void __launch_bounds__(Layout<N>::kThreads, 1) lca_tree_tc_kernel(const __grid_constant__ Params p) {
  using L = Layout<N>;
  constexpr int kSlots = L::kSlots;
  constexpr int kKAt = L::kAlias ? 4 : 1;   // K is taken before this column slot of the tile (last where P waits for it)
  constexpr int kSoftmaxWarps = L::kSoftmaxWarps;
  constexpr int C = 4 * N / kSoftmaxWarps;  // rows of a softmax thread
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t *full = bars, *empty = bars + kMaxSlots, *k_full = bars + 2 * kMaxSlots, *k_empty = k_full + 1,
           *q_full = k_full + 2, *q_empty = k_full + 3, *drain = k_full + 4,
           *event = k_full + 5,       // [2]: for the softmax: S of a tile is there, a tile comes back, O is complete
           *p_full = k_full + 7, *meet = k_full + 8,
           *told = k_full + 9;        // [2]: a unit is written down
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffMisc + 4);
  int* s_least = reinterpret_cast<int*>(smem + L::kOffMisc + 8);       // [kTreeMaxWaves]
  unsigned long long* broken = reinterpret_cast<unsigned long long*>(smem + L::kOffMisc + 24);
  volatile int* too_high = reinterpret_cast<volatile int*>(smem + L::kOffMisc + 32);
  volatile int* come_back = too_high + 1;
  Unit* units = reinterpret_cast<Unit*>(smem + L::kOffUnit);
  static_assert(sizeof(Unit) == 32, "room for two");
  const TreeBatch& t = p.t;
  const Wait wt = {abort_flag, t.err, p.timeout_ns};
  const WarpLanes lanes;

  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      ptx::mbar_init(full + i, 1);
      ptx::mbar_init(empty + i, 1);
    }
    ptx::mbar_init(k_full, 1);
    ptx::mbar_init(k_empty, 1);
    ptx::mbar_init(q_full, 1);
    ptx::mbar_init(q_empty, 1);
    for (int i = 0; i < kTreeEventBars; ++i) ptx::mbar_init(event + i, 1);
    ptx::mbar_init(p_full, kSoftmaxWarps);
    ptx::mbar_init(meet, kSoftmaxWarps);
    ptx::mbar_init(drain, 1);
    ptx::mbar_init(told, 1);
    ptx::mbar_init(told + 1, 1);
    *abort_flag = 0;
    *broken = 0ull;
    *too_high = *come_back = -1;
    ptx::fence_mbarrier_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_slot, kTmemCols);
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

  // ---- the cut: one warp per number of waves.  Up to 32 sequences a lane keeps its own one's work; with more the
  // first 896 ones' is kept in shared memory, 25 bits of tiles and 7 of drafted tokens.
  const bool few = t.B <= 32;
  TreeWork own = {0, 0};
  TreeLens own_len = {0, 0, false};
  if (few && lane < t.B) {
    own_len = tree_lens(t, lane);
    own = tree_work(own_len.n, own_len.d, t.H, N);
  }
  auto lens_of = [&](int b) {                  // for a whole warp
    if (!few) return tree_lens(t, b);
    return TreeLens{__shfl_sync(0xffffffffu, own_len.n, b), __shfl_sync(0xffffffffu, own_len.d, b), false};
  };
  uint32_t* kept = reinterpret_cast<uint32_t*>(smem + L::kOffSeq);
  if (!few) {
    for (int b = tid; b < min(t.B, kSeqs); b += L::kThreads) {
      const TreeLens l = tree_lens(t, b);
      kept[b] = (uint32_t)tree_work(l.n, l.d, t.H, N).tiles << 7 | (uint32_t)l.d;
    }
    __syncthreads();
  }
  auto seq = [&](int b) {
    if (few) return own;                       // asked for b = lane only
    if (b < kSeqs) return TreeWork{(int)((kept[b] & 127u) * (uint32_t)t.H + N - 1) / N, (int)(kept[b] >> 7)};
    const TreeLens l = tree_lens(t, b);
    return tree_work(l.n, l.d, t.H, N);
  };
  int most = 1;
  for (int b = lane; b < t.B; b += 32) most = max(most, seq(b).tiles);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  if (warp >= 2 && warp < 2 + kTreeMaxWaves) {
    const int k = warp - 1;
    const int S = few ? tree_least_few(lanes, own, t.B, most, (int64_t)k * p.G) : tree_least(lanes, seq, t.B, most, (int64_t)k * p.G);
    if (lane == 0) s_least[k - 1] = S;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int S = most;
  int64_t best = INT64_MAX;
#pragma unroll
  for (int k = 1; k <= kTreeMaxWaves; ++k) {
    const int64_t c = tree_cost(k, s_least[k - 1], most);
    if (c < best) {
      best = c;
      S = s_least[k - 1];
    }
  }

  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    // Converged, with one elected lane, like the MMA warp; a tile's rows are looked up a tile ahead.
    int nk = 0, nq = 0, slot = 0, use = 0;     // K tiles, query blocks; next slot, and how often each was filled
    int sent = 0;                              // slots that were ever filled (for the last waits)
    bool ok = true, skip = p.debug_skip_load != 0;
    int nu = 0;
    TreeCursor<int> at_unit;
    for (int64_t u = blockIdx.x; ok && u < INT32_MAX; u += p.G, ++nu) {
      const TreeUnit un = tree_unit<int>(lanes, seq, t.B, S, (int)u, at_unit);
      // Written down for the other warps: the softmax warps have no registers for the search (V2 trees 442 -> 464 us
      // with one), and in the MMA warp it held up the next S (3400 cycles with 740 sequences).  The entry was the
      // one of two units ago, which all have read: the last unit's S is complete, and its first was issued after the
      // P of the unit before it.
      auto tell = [&](const TreeLens& of) {
        if (lane == 0) {
          units[nu & 1] = Unit{un, of.n, of.d};
          ptx::mbar_arrive(told + (nu & 1));
        }
        __syncwarp();
      };
      if (un.b < 0) {
        if (nu < 2 || warp_wait(q_empty, (nq - 1) & 1, wt, 0xC10)) tell(TreeLens{0, 0, false});
        break;
      }
      const TreeLens l = lens_of(un.b);
      const int total = l.n + l.d;
      // a tile's two halves of 64 rows; a second half without tokens is loaded from the first half's rows, and
      // zeroed later
      auto rows_of = [&](int tile, int& r0, int& r1) {
        const int pos = tile * kTreeTile;
        r0 = (int)tree_row(t, un.b, pos, 0xB05);
        r1 = pos + 64 < total ? (int)tree_row(t, un.b, pos + 64, 0xB05) : r0;
      };
      int r0, r1, n0 = 0, n1 = 0;
      rows_of(un.t0, r0, r1);
      const int qrow = (int)((int64_t)un.b * t.T * t.H + (int64_t)un.rb * N);
      if (nq > 0) ok = warp_wait(q_empty, (nq - 1) & 1, wt, 0xC10);
      if (!ok) break;
      tell(l);
      if (ptx::elect_one()) {
        ptx::mbar_arrive_expect_tx(q_full, 9 * L::kQChunk);
#pragma unroll
        for (int c = 0; c < 8; ++c) ptx::tma_load_2d(smem + L::kOffQ + c * L::kQChunk, &p.tm_qc, 64 * c, qrow, q_full);
        ptx::tma_load_2d(smem + L::kOffQ + 8 * L::kQChunk, &p.tm_qr, 0, qrow, q_full);
      }
      __syncwarp();
      ++nq;
      for (int tile = un.t0; tile < un.t1 && ok; ++tile) {
        if (tile + 1 < un.t1) {
          rows_of(tile + 1, n0, n1);
          // Where several row blocks read the tile, the first brings the next one into L2, or the wait for
          // memory would hold up all of them (V2-Lite trees 166 -> 156 us); where there is one, the slots
          // in flight cover that wait and the prefetches only add to the traffic (148 sequences 438 -> 455).
          if (un.rb == 0 && l.d * t.H > N && ptx::elect_one()) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              ptx::tma_prefetch_l2_2d(&p.tm_c, 64 * c, n0);
              ptx::tma_prefetch_l2_2d(&p.tm_c, 64 * c, n1);
            }
            ptx::tma_prefetch_l2_2d(&p.tm_k, 0, n0);
            ptx::tma_prefetch_l2_2d(&p.tm_k, 0, n1);
          }
          __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < 5; ++i) {
          if (i == kKAt) {
            if (nk > 0) ok = warp_wait(k_empty, (nk - 1) & 1, wt, 0xC11);
            if (!ok) break;
            if (ptx::elect_one()) {
              ptx::mbar_arrive_expect_tx(k_full, kChunk);
              ptx::tma_load_2d(smem + L::kOffK, &p.tm_k, 0, r0, k_full);
              ptx::tma_load_2d(smem + L::kOffK + kChunk / 2, &p.tm_k, 0, r1, k_full);
            }
            __syncwarp();
            ++nk;
            continue;
          }
          const int m = i < kKAt ? i : i - 1;
          const int at = kSlots == 4 ? m : slot;
          if (!LCA_CHECK(t.err, at >= 0 && at < kSlots, 0xD42)) ok = false;
          if (use > 0 && ok) ok = warp_wait(empty + at, (use - 1) & 1, wt, 0xC12);
          if (!ok) break;
          if (!skip && ptx::elect_one()) {
            ptx::mbar_arrive_expect_tx(full + at, kSlot);
            uint8_t* dst = smem + at * kSlot;
#pragma unroll
            for (int ch = 0; ch < 2; ++ch) {
              ptx::tma_load_2d(dst + ch * kChunk, &p.tm_c, 128 * m + 64 * ch, r0, full + at);
              ptx::tma_load_2d(dst + ch * kChunk + kChunk / 2, &p.tm_c, 128 * m + 64 * ch, r1, full + at);
            }
          }
          __syncwarp();
          if (!skip && use == 0) sent |= 1 << at;
          skip = false;
          if (++slot == kSlots) {
            slot = 0;
            ++use;
          }
        }
        r0 = n0;
        r1 = n1;
      }
    }
    // every copy lands before the CTA may exit: the last phase of each slot
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const int fills = use + (i < slot ? 1 : 0);
      if (fills > 1 || (fills == 1 && ((sent >> i) & 1))) wait(full + i, (fills - 1) & 1, wt, 0xC1F, false);
    }
    if (nk > 0) wait(k_full, (nk - 1) & 1, wt, 0xC1F, false);
    if (nq > 0) wait(q_full, (nq - 1) & 1, wt, 0xC1F, false);
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMAs
    constexpr uint32_t kIdS = ptx::idesc_bf16_f32(128, N, 0, 0);     // both K-major
    constexpr uint32_t kIdO = ptx::idesc_bf16_f32(128, N, 1, 1);     // both MN-major
    const uint64_t d_c = ptx::smem_desc(ptx::smem_u32(smem), 16, 1024, ptx::kSwizzle128B);
    const uint64_t d_k = ptx::smem_desc(ptx::smem_u32(smem + L::kOffK), 16, 1024, ptx::kSwizzle128B);
    const uint64_t d_q = ptx::smem_desc(ptx::smem_u32(smem + L::kOffQ), 16, 1024, ptx::kSwizzle128B);
    const uint64_t d_ct = ptx::smem_desc(ptx::smem_u32(smem), kChunk, 1024, ptx::kSwizzle128B);
    const uint64_t d_p = ptx::smem_desc(ptx::smem_u32(smem + L::kOffP), 128, 2048, ptx::kSwizzleNone);
    // The whole warp runs this, and one elected lane issues: the operands' descriptors then
    // stay in uniform registers (an MMA every 53 cycles; 77 from a branch that one lane takes).
    // The next load's barrier is probed before the MMAs of the load at hand and looked at
    // after them: a probe takes longer than the MMAs in flight cover.
    int it = 0, nq = 0, s0 = 0, ph = 0, ev = 0, np = 0;   // tiles, query blocks; slot of the tile's first load and the
    bool ok = true, ready = false;                         // parity of its phase; events, arrivals of P
    auto load_bar = [&](int i, int& parity) -> uint64_t* {   // load i of the tile at hand: K, or a column slot
      if (i == kKAt) {
        parity = it & 1;
        return k_full;
      }
      int slot = (kSlots == 4 ? 0 : s0) + (i < kKAt ? i : i - 1);
      parity = ph;
      if (slot >= kSlots) {
        slot -= kSlots;
        parity ^= 1;
      }
      return full + slot;
    };
    while (ok) {
      if (!warp_wait(told + (nq & 1), (nq >> 1) & 1, wt, 0xC21)) break;
      const TreeUnit un = units[nq & 1].un;
      if (un.b < 0) break;
      ok = warp_wait(q_full, nq & 1, wt, 0xC20);
      ++nq;
      for (int tile = un.t0; tile < un.t1 && ok; ++tile) {
#pragma unroll
        for (int i = 0; i < 5; ++i) {
          int parity;
          uint64_t* bar = load_bar(i, parity);
          if (!__all_sync(0xffffffffu, ready)) ok = warp_wait(bar, parity, wt, 0xC22) && ok;
          ptx::tc_fence_after();
          ready = false;
          if (i < 4) {
            uint64_t* ahead = load_bar(i + 1, parity);
            ready = ptx::mbar_test_wait(ahead, parity);
          }
          if (!ok) break;
          if (ptx::elect_one()) {
            if (i == kKAt) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                ptx::mma_bf16_ss(tmem + kColS, d_k + (uint64_t)((32 * k) >> 4),
                                 d_q + (uint64_t)((8 * L::kQChunk + 32 * k) >> 4), kIdS, (i | k) != 0);
              if (!L::kAlias) ptx::mma_commit(k_empty);
            } else {
              const int m = i < kKAt ? i : i - 1;
              const uint64_t a = d_c + (uint64_t)(((bar - full) * kSlot) >> 4);
#pragma unroll
              for (int ch = 0; ch < 2; ++ch)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  ptx::mma_bf16_ss(tmem + kColS, a + (uint64_t)((ch * kChunk + 32 * k) >> 4),
                                   d_q + (uint64_t)(((2 * m + ch) * L::kQChunk + 32 * k) >> 4), kIdS, (i | ch | k) != 0);
            }
            if (i == 4) {
              ptx::mma_commit(event + tree_event_bar(ev));
              if (tile + 1 == un.t1) ptx::mma_commit(q_empty);
            }
          }
          __syncwarp();
        }
        if (!ok) break;
        ok = warp_wait(p_full, np++ & 1, wt, 0xC23);
        if (ok && __shfl_sync(0xffffffffu, *too_high, 0) == ev) {
          ++ev;
          if (lane == 0) {
            *come_back = ev;
            ptx::mbar_arrive(event + tree_event_bar(ev));
          }
          __syncwarp();
          ok = warp_wait(p_full, np++ & 1, wt, 0xC24);
        }
        ++ev;
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t first = tile > un.t0 ? 1u : 0u;
        const int here = kSlots == 4 ? 0 : s0;
        s0 += 4;                            // the next tile's first load
        if (s0 >= kSlots) {
          s0 -= kSlots;
          ph ^= 1;
        }
        ++it;
        if (ptx::elect_one()) {
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            int slot = here + m;
            if (slot >= kSlots) slot -= kSlots;
            const uint64_t a = d_ct + (uint64_t)((slot * kSlot) >> 4);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              ptx::mma_bf16_ss(tmem + kColO + N * m, a + (uint64_t)((2048 * k) >> 4), d_p + (uint64_t)((256 * k) >> 4),
                               kIdO, k > 0 ? 1u : first);
            ptx::mma_commit(empty + slot);
          }
          if (L::kAlias) ptx::mma_commit(k_empty);
          if (tile + 1 == un.t1) ptx::mma_commit(event + tree_event_bar(ev));
        }
        __syncwarp();
        {
          int parity;
          uint64_t* ahead = load_bar(0, parity);
          ready = ptx::mbar_test_wait(ahead, parity);
        }
        if (tile + 1 == un.t1) ++ev;
      }
    }
    if (ptx::elect_one()) ptx::mma_commit(drain);   // and every MMA
    wait(drain, 0, wt, 0xC2F, false);
  } else {
    // ---------------------------------------------------------------- softmax
    const int sw = warp - 2;
    const int quarter = warp & 3, part = sw >> 2;     // TMEM lanes 32 quarter .., rows C part ..
    const int tok = 32 * quarter + lane;              // this thread's token of a tile
    const int sid = tid - 64;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * quarter) << 16) + C * part;
    float* reds = reinterpret_cast<float*>(smem + L::kOffRed);
    int red_turn = 0;
    float2* row_mz = reinterpret_cast<float2*>(smem + L::kOffM);
    uint8_t* pt = smem + L::kOffP + (C / 8) * part * 2048 + tok * 16;
    int s0 = 0, ph = 0;         // slot of the tile's first load and the parity of its phase
    int ev = 0, met = 0;        // events seen; meetings of the softmax warps
    bool ok = true;
    // A barrier of the softmax warps whose wait is bounded: a warp that leaves on an error leaves none behind.
    auto meeting = [&] {
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(meet);
      ok = warp_wait(meet, met++ & 1, wt, 0xC33) && ok;
      return ok;
    };
    // the sequences' records for the merge, by the first CTA
    if (blockIdx.x == 0 && sw == kSoftmaxWarps - 1) {
      int64_t base = 0;
      for (int b0 = 0; b0 < t.B; b0 += 32) {
        const int b = b0 + lane;
        TreeWork k = {0, 0};
        bool bad = false;
        if (b < t.B) {
          k = seq(b);
          bad = tree_lens(t, b).bad;
        }
        const int parts = (k.tiles + S - 1) / S;
        const int64_t mine = (int64_t)k.rb * parts, incl = base + lanes.scan(mine);
        if (b < t.B) p.split[b] = TreeSplit{(int)(incl - mine), parts, k.rb, bad ? 1 : 0};
        if (bad) input_error(t.err, 0xB01);
        base = lanes.get(incl, 31);
      }
    }
    int nu = 0;
    for (int64_t u = blockIdx.x; ok; u += p.G, ++nu) {
      if (!warp_wait(told + (nu & 1), (nu >> 1) & 1, wt, 0xC34)) break;
      const TreeUnit un = units[nu & 1].un;
      if (un.b < 0) break;
      const TreeLens l = TreeLens{units[nu & 1].n, units[nu & 1].d, false};
      const int total = l.n + l.d;
      const int rows = min(N, l.d * t.H - un.rb * N);
      unsigned long long* words = reinterpret_cast<unsigned long long*>(smem + L::kOffWord) + N * (nu & 1);
      if (sid < N) words[sid] = sid < rows ? tree_word(t, un.b, (un.rb * N + sid) / t.H) : 0ull;
      if (!meeting()) break;                           // (and the last unit's sums are read)
      float nM[C], Z[C], x[C];    // -M in units of log2; x: the weights not yet in Z
#pragma unroll
      for (int c = 0; c < C; ++c) {
        nM[c] = -kEmpty;
        Z[c] = x[c] = 0.f;
      }
      // one event after another: S of the next tile, the tile at hand once more, or the end
      bool special = false;
      for (int tile = un.t0 - 1;;) {
        const bool live = warp_wait(event + tree_event_bar(ev), tree_event_parity(ev), wt, 0xC30);
        ptx::tc_fence_after();
        const bool again = *come_back == ev;
        if (!again) {
#pragma unroll
          for (int c = 0; c < C; c += 2)
            ptx::f32x2_split(ptx::add_f32x2(ptx::f32x2(Z[c], Z[c + 1]), ptx::f32x2(x[c], x[c + 1])), Z[c], Z[c + 1]);
          if (tile >= un.t0) {
            s0 += 4;
            if (s0 >= kSlots) {
              s0 -= kSlots;
              ph ^= 1;
            }
          }
          ++tile;
        }
        ok = live;
        if (!ok || tile == un.t1) break;
        const int pos0 = tile * kTreeTile;
        tmem_load<C>(lane_base + kColS, x);
        special = pos0 + kTreeTile > l.n;                      // drafted tokens, or the end, in this tile
        const bool raise = again || tile == un.t0;
        uint32_t hurt = 0;                                     // rows that see this thread's broken token
        if (special) {
          // zero what is no token, and drafted rows that hold an infinity or NaN
          auto slot_of = [&](int m) { return s0 + m < kSlots ? s0 + m : s0 + m - kSlots; };
          auto phase_of = [&](int m) { return (uint32_t)(s0 + m < kSlots ? ph : ph ^ 1); };
          bool there = true;                                   // S is complete, so the rows are; this makes them seen
#pragma unroll
          for (int m = 0; m < 4; ++m) there = ptx::mbar_test_wait(full + slot_of(m), phase_of(m)) && there;
          if (!__all_sync(0xffffffffu, there))
            for (int m = 0; m < 4; ++m) ok = warp_wait(full + slot_of(m), phase_of(m), wt, 0xC31) && ok;
          uint8_t* chunk[2];                                   // 8 chunks of 128 bytes a row, 16 a lane
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int ch = 4 * h + (lane >> 3);
            chunk[h] = smem + slot_of(ch >> 1) * kSlot + (ch & 1) * kChunk + (lane & 7) * 16;
          }
          for (int r = sw; r < kTreeTile; r += kSoftmaxWarps) {
            const int pos = pos0 + r;
            if (pos < l.n) continue;
            uint4* at[2];
            bool bad = false;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              at[h] = reinterpret_cast<uint4*>(chunk[h] + r * 128);
              if (!LCA_CHECK(t.err, chunk[h] >= smem && chunk[h] + r * 128 + 16 <= smem + kSlots * kSlot, 0xD43))
                at[h] = reinterpret_cast<uint4*>(smem);
              bad = bad || any_nonfinite(*at[h]);
            }
            bad = __any_sync(0xffffffffu, bad);
            if (bad || pos >= total) {
              *at[0] = make_uint4(0, 0, 0, 0);
              *at[1] = make_uint4(0, 0, 0, 0);
            }
            if (bad && pos < total && lane == 0) atomicOr(broken, 1ull << (pos - l.n));
          }
          if (!meeting()) break;
        }
        ptx::tmem_wait_ld();
        if (special) {
          const int node = pos0 + tok - l.n;
          if (node >= 0) {
            const bool in = node < l.d;
            const bool bk = in && ((*broken >> node) & 1ull);
#pragma unroll
            for (int c = 0; c < C; ++c) {
              const bool sees = in && ((words[C * part + c] >> node) & 1ull);
              if (sees && bk) hurt |= 1u << c;
              if (!sees || bk) x[c] = -INFINITY;
            }
          }
        }
        if (raise) {
          // M becomes the largest logit so far, row by row
          float* red = reds + 4 * N * (red_turn++ & 1);
          const float m0 = fold<C>(x, lane, [](float a, float b) { return fmaxf(a, b); });
          if (lane % (32 / C) == 0) red[quarter * N + C * part + lane / (32 / C)] = m0 * kLog2eS;
          if (!meeting()) break;
#pragma unroll
          for (int c0 = 0; c0 < C; c0 += 8) {
            float f[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const int r = C * part + c0 + c;
              const float m = fmaxf(fmaxf(fmaxf(red[r], red[N + r]), fmaxf(red[2 * N + r], red[3 * N + r])), -nM[c0 + c]);
              f[c] = ex2(-nM[c0 + c] - m);
              Z[c0 + c] *= f[c];
              nM[c0 + c] = -m;
            }
            if (tile > un.t0) {
#pragma unroll 1
              for (int m = 0; m < 4; ++m) {
                float o[8];
                ptx::tmem_ld8(lane_base + kColO + N * m + c0, o);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 8; ++c) o[c] *= f[c];
                ptx::tmem_st8(lane_base + kColO + N * m + c0, o);
              }
            }
          }
          ptx::tmem_wait_st();
        }
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < C; c += 2) {
          ptx::f32x2_split(ptx::fma_f32x2(ptx::f32x2(x[c], x[c + 1]), ptx::f32x2(kLog2eS, kLog2eS), ptx::f32x2(nM[c], nM[c + 1])),
                           x[c], x[c + 1]);
          top = fmaxf(top, fmaxf(x[c], x[c + 1]));
        }
        if (top > kRaise && !raise) *too_high = ev;
#pragma unroll
        for (int c = 0; c < C; ++c) x[c] = ex2(x[c]);
#pragma unroll
        for (int c = 0; c < C; c += 8)
          *reinterpret_cast<uint4*>(pt + (c / 8) * 2048) = make_uint4(pack2(x[c], x[c + 1]), pack2(x[c + 2], x[c + 3]),
                                                                    pack2(x[c + 4], x[c + 5]), pack2(x[c + 6], x[c + 7]));
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(p_full);
        ++ev;
        if (hurt) {
#pragma unroll
          for (int c = 0; c < C; ++c)
            if ((hurt >> c) & 1u) x[c] = __int_as_float(0x7fc00000);
        }
      }
      if (!ok) break;
      ++ev;
      // ---- the unit's sums
      float* red = reds + 4 * N * (red_turn++ & 1);
      const float z0 = fold<C>(Z, lane, [](float a, float b) { return a + b; });
      if (lane % (32 / C) == 0) red[quarter * N + C * part + lane / (32 / C)] = z0;
      if (quarter == 0) {
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (lane == c) row_mz[C * part + c].x = -nM[c];
      }
      if (sid == 0) *broken = 0ull;
      if (!meeting()) break;
      const bool whole = un.parts == 1;
      const int64_t row0 = (int64_t)un.b * t.T * t.H + (int64_t)un.rb * N;
      if (sid < N) {
        const float z = (red[sid] + red[N + sid]) + (red[2 * N + sid] + red[3 * N + sid]), m = row_mz[sid].x;
        row_mz[sid].y = z == 0.f ? 0.f : 1.f / z;
        if (sid < rows) {
          if (!whole) {
            if (LCA_CHECK(t.err, u < p.slots, 0xD40)) *reinterpret_cast<float2*>(p.part_mz + 2 * (u * N + sid)) = make_float2(m, z);
          } else if (p.lse) {
            p.lse[row0 + sid] = z == 0.f ? -INFINITY : kTreeLn2 * (m + log2f(z));
          }
        }
      }
      if (!meeting()) break;
      // O^T: a thread has one dim and C rows of each block of 128 dims
      const bool out_ok = LCA_CHECK(t.err, row0 + rows <= (int64_t)t.B * t.T * t.H, 0xD44);
      const int mine = out_ok ? min(C, rows - C * part) : 0;   // rows of this thread
      if (whole) {
        __nv_bfloat16* dst = p.out + (row0 + C * part) * kDC + tok;
        const float2* mz = row_mz + C * part;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          float o[C];
          tmem_load<C>(lane_base + kColO + N * m, o);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < C; ++c)
            if (c < mine) dst[c * kDC + 128 * m] = __float2bfloat16_rn(o[c] * mz[c].y);
        }
      } else if (LCA_CHECK(t.err, u < p.slots, 0xD41)) {
        float* dst = p.part_o + (u * N + C * part) * kDC + tok;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          float o[C];
          tmem_load<C>(lane_base + kColO + N * m, o);
          ptx::tmem_wait_ld();
          if (mine == C) {
#pragma unroll
            for (int c = 0; c < C; ++c) dst[c * kDC + 128 * m] = o[c];
          } else {
#pragma unroll
            for (int c = 0; c < C; ++c)
              if (c < mine) dst[c * kDC + 128 * m] = o[c];
          }
        }
      }
      ptx::tc_fence_before();
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc(tmem, kTmemCols);
}

}  // namespace ttc
}  // namespace lca
