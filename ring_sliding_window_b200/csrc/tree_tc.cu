// Attention of drafted tokens over the cache on the 5th-generation tensor
// cores (bf16, d = 64 or 128).
//
// For draft i of a sequence, over the entries j that it may see (the cache's
// prompt and ring slots, and the drafts above it in the tree),
//   o_i = sum_j 2^(x_ij) v_j / sum_j 2^(x_ij),   x_ij = scale log2(e) q_i.k_j - m_i,
// in one pass over K and V.  T drafts do 4 T d operations on the 4 d bytes of
// an entry, so up to T = 128 the tensor cores (about 250 operations a byte)
// could wait for HBM: the kernel's job is to keep the copies coming and
// everything else behind them.  Up to 64 drafts it does on long prompts (1.2 to
// 1.35 times the time of the bytes at 8 x 8,256 and 4 x 16,384 or 32,640 tokens).
//
// The 128-key tiles of all rings (a ring's drafts first, then its cache) are
// cut into one range of about equal cost per CTA, one CTA an SM; a ring in several
// pieces leaves partials that tree_combine_kernel merges.  Inside a CTA:
//   producer warp   K and V tiles by TMA (128-byte swizzle) into two rings of
//                   slots, and the N query rows of each piece;
//   MMA warp        an elected lane: S^T = K Q^T (128 keys x N drafts) into one of
//                   two TMEM buffers, a tile ahead of O^T += V^T P;
//   softmax warps   thread r of four warps owns key r of the tile (TMEM lane r)
//                   and 16 drafts (32 for N = 64): 4, 8 or 8 warps;
//   4 side warps    what would hold the softmax up where pieces begin and end:
//                   the scan of V (below), RoPE, and the results of a piece,
//                   while the next one already fills the other O.
// With the keys on the lanes the work of a tile grows with the drafts (N = 16,
// 32 or 64), and all lanes take part however few they are.  What a softmax needs
// across the lanes is kept off the ordinary tile: the subtracted m_i only moves
// when a score exceeds it by more than 2^16, which one barrier with an OR finds
// out, and the sums over the keys stay per lane until a piece ends.
//
// More than 64 drafts are two columns of the grid with N = 64: half the SMs
// each, over the same tiles at the same time, so HBM is read about once.  (One
// CTA with N = 128 has no registers and shared memory left to keep the tensor
// cores busy: 140 us against 111 for 128 drafts over 4 x 16,384 tokens.)  What
// bounds them is the work on a tile: 70 tiles an SM, about 1.4 us each, and both
// columns take every tile, which an SM's share of HBM brings in 1.5 us (the bytes
// alone: 52 us).
//
// P goes to the MMA as a bf16 pair hi + lo, next to one another along N, so one
// product gives O_hi | O_lo (relative error of a weight 2^-14 at most; bf16 alone
// would add its 2^-9 to an output that is rounded to bf16 once).  Both are cut off,
// never rounded up, and the sum takes the uncut weights, so outputs lie about
// 1e-5 of themselves too close to 0, a hundredth of their rounding.  O_hi is finite
// wherever the exact sum is, and alone decides what is not: O_lo of an infinite
// value is 0 x inf = NaN.
//
// A masked score becomes -inf, so its weight is 0, but 0 x inf is NaN inside
// an MMA.  In the tiles that hold masked entries (the drafts, and the tiles
// with ring slots) the side warps therefore take non-finite values out of V's
// shared-memory copy, and add them to the results of the drafts that see them.
//
// A wait that runs out leaves the softmax warps going through all their tiles
// without waiting (their barriers need every warp), and the side warps; the others stop.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>

#include "internal.h"
#include "ptx.cuh"
#include "tcgen05.cuh"
#include "tmap.h"
#include "tree.cuh"

namespace rswa {
namespace {

constexpr int kTile = kTreeTcTile;          // keys per tile
constexpr int kHalfBytes = kTile * 64 * 2;  // one 64-column swizzled block: 16 KB
// Log2 units.  Weights of up to 2^16 are no less precise: FP32 sums and bf16 pairs
// keep their relative error, and what underflows lies 2^-126 below the weight 1.
constexpr float kGrowth = 16.0f;
constexpr float kLog2e = 1.4426950408889634f;

template <int D, int N>
struct Shape {
  static constexpr int NC = N == 64 ? 32 : 16; // drafts of a softmax thread
  static constexpr int kGroups = N / NC;       // of 4 softmax warps
  static constexpr int kSoftWarps = 4 * kGroups;
  static constexpr int kThreads = (kSoftWarps + 6) * 32;
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kHalves * kHalfBytes;
  static constexpr int kPBytes = N <= 32 ? kHalfBytes : N / 32 * kHalfBytes;
  // K and V tiles in flight, P and Q buffers: what 227 KB hold.  At N = 32 a third
  // V tile is worth more than a second P and Q (1,088-token prompts of 32 users: 58
  // against 69 us); at N = 64 a second P more than a second Q.
  static constexpr int kK = (N <= 32 ? 3 : 2) * (D == 64 ? 2 : 1);
  static constexpr int kV = (N == 32 ? 3 : 2) * (D == 64 ? 2 : 1);
  static constexpr int kPBufs = N == 32 ? 1 : 2;
  static constexpr int kQBufs = N == 16 ? 2 : 1;
  // S0, S1 (N each), O0, O1 (N hi and N lo each)
  static constexpr uint32_t kTmemCols = N == 64 ? 512 : N == 32 ? 256 : 128;
  static constexpr uint32_t kColO = 2 * N;
};

template <int D, int N>
struct __align__(1024) TreeSmem {
  using S = Shape<D, N>;
  uint8_t k[S::kK][S::kTileBytes];
  uint8_t v[S::kV][S::kTileBytes];
  uint8_t p[S::kPBufs][S::kPBytes];
  uint8_t q[S::kQBufs][S::kHalves * N * 128];
  float neg_m[N];      // -m of every draft
  float alpha[N];      // factors of a growth
  int top[N];          // largest scores of a tile, as ordered_int (INT_MIN between growths)
  float sums[2][4][N]; // a finished piece's sums over each warp's keys
  float m[2][N];       // and its m
  float inv[N];        // side warps: 1 / sum
  __align__(4) uint8_t depth[N];
  uint64_t q_full[S::kQBufs], q_free[S::kQBufs];
  uint64_t k_full[S::kK], k_empty[S::kK];
  uint64_t v_full[S::kV], v_empty[S::kV];
  uint64_t v_ask[S::kV], v_fit[S::kV];  // a masked tile's V is on its way; it is scanned
  uint64_t s_full[2];  // S of a tile finished
  // P of a tile written (one arrival a softmax warp).  Two, since the softmax may
  // finish a second tile while the MMA warp still waits for the first one's V: S
  // of a third tile is only issued after that PV.
  uint64_t p_full[2];
  // O += P V of a tile finished.  Waited for with one tile outstanding at most
  // (S of a tile in hand says that the PV of the tile before the last is done).
  uint64_t pv_done;
  uint64_t o_done[2], o_free[2];  // a piece's last PV finished; its results taken
  uint64_t l_done[2];  // sums and m of a piece written
  // RoPE: a piece's queries and drafted keys turned.  One for each Q buffer: the side
  // warps may turn the next piece's before the MMA warp has looked at this one's, but
  // come back to a buffer only after q_free, which follows that look.
  uint64_t turned[S::kQBufs];
  uint64_t mma_done;
  uint32_t tmem_base;
  int dead;
};

struct TreeTcArgs {
  DeviceView v;
  TreeView tv;
  const __nv_bfloat16 *vd, *vc;  // the values, for the ones that are not finite
  __nv_bfloat16 *out;
  int box_rows;  // of the drafts' tiles
};

__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, int *err,
                                         volatile int *dead) {
  if (*dead) return false;
  if (mbar_wait_bounded(bar, parity, err, RSWA_DEVERR_TIMEOUT)) return true;
  *dead = 1;
  return false;
}

// One piece's tiles: the drafts' (if it has it), then cache tiles [c0, c1).
struct PieceTiles {
  int drafts, c0, n;
  __device__ __forceinline__ PieceTiles(const DecodePiece &pc, const RingView &r) {
    drafts = pc.key_begin == 0 ? 1 : 0;
    c0 = max(pc.key_begin - 1 + drafts, r.lo / kTile);
    const int c1 = min(pc.key_end - 1, (r.held + kTile - 1) / kTile);
    n = drafts + max(0, c1 - c0);
  }
  // tile j is the drafts', or begins at this slot
  __device__ __forceinline__ bool is_drafts(int j) const { return drafts && j == 0; }
  __device__ __forceinline__ int slot(int j) const { return (c0 + j - drafts) * kTile; }
  // whether some draft may not see some row of tile j
  __device__ __forceinline__ bool masked(int j, const RingView &r) const {
    return is_drafts(j) || r.swa || slot(j) + kTile > r.plen;
  }
};

__device__ __forceinline__ uint32_t word_of(const uint4 &u, int i) {
  return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
}

// Byte offset of 16-byte chunk c of row r in a swizzled tile of 64-column
// blocks of `block` bytes.
__device__ __forceinline__ uint32_t chunk_at(int r, int c, uint32_t block) {
  return (uint32_t)(c >> 3) * block + (uint32_t)r * 128u + ((uint32_t)((c & 7) ^ (r & 7)) << 4);
}

// Turn row r of a swizzled tile by its (cos, sin) table (rotate-half RoPE).
template <int D>
__device__ __forceinline__ void turn_row(uint8_t *tile, int r, uint32_t block, const float2 *cs) {
#pragma unroll 1
  for (int c = 0; c < D / 16; ++c) {
    uint4 *p0 = reinterpret_cast<uint4 *>(tile + chunk_at(r, c, block));
    uint4 *p1 = reinterpret_cast<uint4 *>(tile + chunk_at(r, c + D / 16, block));
    float x[8], y[8];
    Chunk<__nv_bfloat16>::widen(*p0, x);
    Chunk<__nv_bfloat16>::widen(*p1, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 w = cs[c * 8 + e];
      const float a = x[e], b = y[e];
      x[e] = a * w.x - b * w.y;
      y[e] = b * w.x + a * w.y;
    }
    *p0 = Chunk<__nv_bfloat16>::narrow(x);
    *p1 = Chunk<__nv_bfloat16>::narrow(y);
  }
}

// S^T = K Q^T (128 keys x N drafts).
template <int D, int N>
__device__ __forceinline__ void issue_qk(uint32_t elected, uint32_t d_tmem, uint32_t q_addr, uint32_t k_addr) {
  constexpr uint32_t idesc = tc::idesc_bf16_f32(kTile, N, false, false);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
    tc::mma_ss_elected(elected, d_tmem,
               tc::sw128_desc(k_addr + (uint32_t)(kk >> 2) * kHalfBytes + (uint32_t)(kk & 3) * 32,
                              16, 1024),
               tc::sw128_desc(q_addr + (uint32_t)(kk >> 2) * (N * 128) + (uint32_t)(kk & 3) * 32,
                              16, 1024),
               idesc, kk > 0);
}

// O^T += V^T P (D elements x (N hi, N lo) drafts, K = 128 keys).
template <int D, int N>
__device__ __forceinline__ void issue_pv(uint32_t elected, uint32_t o_tmem, uint32_t p_addr, uint32_t v_addr,
                                         bool accumulate) {
  constexpr uint32_t idesc = tc::idesc_bf16_f32(D, 2 * N, true, true);
#pragma unroll
  for (int kk = 0; kk < kTile / 16; ++kk)
    tc::mma_ss_elected(elected, o_tmem, tc::sw128_desc(v_addr + (uint32_t)kk * 2048, kHalfBytes, 1024),
               tc::sw128_desc(p_addr + (uint32_t)kk * 2048, kHalfBytes, 1024), idesc,
               accumulate || kk > 0);
}

// Bit 15 / 31: the low / high bf16 of a pair is not finite (its exponent's ones
// carry over).
__device__ __forceinline__ uint32_t not_finite(uint32_t x) {
  return ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}
// A pair with 0 where it is not finite.
__device__ __forceinline__ uint32_t finite_part(uint32_t x) {
  const uint32_t t = not_finite(x);
  return x & ~((t & 0x8000u ? 0xffffu : 0u) | (t & 0x80000000u ? 0xffff0000u : 0u));
}

// NC (16 or 32) consecutive TMEM columns of this thread's lane.
template <int NC>
__device__ __forceinline__ void load_cols(uint32_t taddr, float *x) {
  if constexpr (NC == 16)
    tc::ld16(taddr, reinterpret_cast<uint32_t *>(x));
  else
    tc::ld32(taddr, reinterpret_cast<uint32_t *>(x));
  tc::wait_ld();
}
template <int NC>
__device__ __forceinline__ void store_cols(uint32_t taddr, const float *x) {
  if constexpr (NC == 16)
    tc::st16(taddr, reinterpret_cast<const uint32_t *>(x));
  else
    tc::st32(taddr, reinterpret_cast<const uint32_t *>(x));
}

// The order of floats as integers (its own inverse).
__device__ __forceinline__ int ordered_int(int x) { return x >= 0 ? x : x ^ 0x7fffffff; }

// Reduction of NC values over the 32 lanes, each lane ending with the result
// of one of them in x[0]: half the values cross at every step.
// Lane l holds column NC l / 32.
template <int NC, typename Op>
__device__ __forceinline__ void reduce_lanes(float *x, int lane, Op op) {
  int width = NC;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    if (width > 1) {
      const int half = width / 2;
      const bool upper = (lane & off) != 0;
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) {
        if (i >= half) break;
        const float send = upper ? x[i] : x[i + half];
        const float keep = upper ? x[i + half] : x[i];
        x[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, off));
      }
      width = half;
    } else {
      x[0] = op(x[0], __shfl_xor_sync(0xffffffffu, x[0], off));
    }
  }
}

template <int D, int N>
__global__ void __launch_bounds__(Shape<D, N>::kThreads, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kd,
                   const __grid_constant__ CUtensorMap tm_vd, const __grid_constant__ CUtensorMap tm_kc,
                   const __grid_constant__ CUtensorMap tm_vc, const TreeTcArgs a) {
  using S = Shape<D, N>;
  constexpr int NK = S::kK, NV = S::kV, NQ = S::kQBufs, NC = S::NC, kHalves = S::kHalves;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // dynamic shared memory is only 16-byte aligned: round up to 1024 for the swizzle atoms
  TreeSmem<D, N> &sm = *reinterpret_cast<TreeSmem<D, N> *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const DeviceView &v = a.v;
  const TreeView &tv = a.tv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kSide = S::kSoftWarps, kProducer = kSide + 4, kMma = kProducer + 1;
  const int row0 = (int)blockIdx.y * N;  // this CTA's first draft
  const int p_begin = tv.cta_piece[blockIdx.x], p_end = tv.cta_piece[blockIdx.x + 1];

  if (threadIdx.x == 0) {
    for (int s = 0; s < NQ; ++s) {
      mbar_init(&sm.q_full[s], 1);
      mbar_init(&sm.q_free[s], 1);
      mbar_init(&sm.turned[s], 4);
    }
    for (int s = 0; s < NK; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.k_empty[s], 1);
    }
    for (int s = 0; s < NV; ++s) {
      mbar_init(&sm.v_full[s], 1);
      mbar_init(&sm.v_empty[s], 1);
      mbar_init(&sm.v_ask[s], 1);
      mbar_init(&sm.v_fit[s], 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.s_full[s], 1);
      mbar_init(&sm.p_full[s], S::kSoftWarps);
      mbar_init(&sm.o_done[s], 1);
      mbar_init(&sm.o_free[s], 4);
      mbar_init(&sm.l_done[s], S::kSoftWarps);
    }
    mbar_init(&sm.pv_done, 1);
    mbar_init(&sm.mma_done, 1);
    sm.dead = 0;
    fence_mbar_init();
  }
  // the plan and the maps are the tree's own; the first tiles' way to L2, and that
  // of the counters, can begin while the kernel before this one still runs (a hint
  // returns nothing)
  const DecodePiece first_piece = tv.pieces[p_begin];
  if (warp == kProducer && lane == 0) {
    const DecodePiece &pc = first_piece;
    prefetch_l2(tv.n + pc.b);
    prefetch_l2(v.t + pc.b);
    tc::prefetch_tmap(&tm_q);
    tc::prefetch_tmap(&tm_kd);
    tc::prefetch_tmap(&tm_vd);
    tc::prefetch_tmap(&tm_kc);
    tc::prefetch_tmap(&tm_vc);
    const int first = max(0, pc.key_begin - 1);
    for (int t = first; t < min(pc.key_end - 1, first + NV); ++t)
      for (int x = 0; x < kHalves; ++x) {
        tc::tma_prefetch_2d(&tm_kc, 64 * x, (int)(pc.row0 + (int64_t)t * kTile));
        tc::tma_prefetch_2d(&tm_vc, 64 * x, (int)(pc.row0 + (int64_t)t * kTile));
      }
  }
  if (warp == kMma) {
    tc::tmem_alloc(&sm.tmem_base, S::kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = sm.tmem_base;
  volatile int *dead = &sm.dead;
  grid_dependency_wait();
  allow_dependents();

  if (warp == kProducer) {
    // -------------------------------------------------------------- producer
    // test-only fault injection: no loads at all, so every wait runs out
    const bool drop = (*v.fault & RSWA_FAULT_DROP_DECODE_COPIES) != 0;
    if (lane == 0 && !drop) {
      constexpr uint32_t kQBytes = (uint32_t)N * 128u * kHalves;
      const uint32_t draft_bytes = (uint32_t)a.box_rows * 128u * kHalves;
      int it = 0, active = 0;
      bool ok = true;
      for (int p = p_begin; ok && p < p_end; ++p) {
        const DecodePiece pc = p == p_begin ? first_piece : tv.pieces[p];
        if (tv.n[pc.b] <= row0) continue;
        const RingView ring = ring_view(v, pc.b, pc.plen);
        const PieceTiles pt(pc, ring);
        if (pt.n == 0) continue;
        const int qs = active % NQ;
        if (!(ok = wait_bar(&sm.q_free[qs], ((active / NQ) & 1) ^ 1, v.err, dead))) break;
        const int xh = pc.h * D, y_draft = pc.b * tv.T;
        mbar_arrive_expect_tx(&sm.q_full[qs], kQBytes);
        for (int x = 0; x < kHalves; ++x)
          tc::tma_load_2d(sm.q[qs] + x * (N * 128), &tm_q, xh + 64 * x, y_draft + row0,
                          &sm.q_full[qs]);
        ++active;
        for (int j = 0; j < pt.n; ++j, ++it) {
          const bool drafts = pt.is_drafts(j);
          const int ks = it % NK, vs = it % NV;
          const uint32_t bytes = drafts ? draft_bytes : (uint32_t)S::kTileBytes;
          const int x0 = drafts ? xh : 0;
          const int y0 = drafts ? y_draft : (int)(pc.row0 + pt.slot(j));
          if (!(ok = wait_bar(&sm.k_empty[ks], ((it / NK) & 1) ^ 1, v.err, dead))) break;
          mbar_arrive_expect_tx(&sm.k_full[ks], bytes);
          for (int x = 0; x < kHalves; ++x)
            tc::tma_load_2d(sm.k[ks] + x * kHalfBytes, drafts ? &tm_kd : &tm_kc, x0 + 64 * x, y0,
                            &sm.k_full[ks]);
          if (!(ok = wait_bar(&sm.v_empty[vs], ((it / NV) & 1) ^ 1, v.err, dead))) {
            mbar_wait_bounded(&sm.k_full[ks], (it / NK) & 1, v.err, RSWA_DEVERR_TIMEOUT);
            break;
          }
          mbar_arrive_expect_tx(&sm.v_full[vs], bytes);
          for (int x = 0; x < kHalves; ++x)
            tc::tma_load_2d(sm.v[vs] + x * kHalfBytes, drafts ? &tm_vd : &tm_vc, x0 + 64 * x, y0,
                            &sm.v_full[vs]);
          if (pt.masked(j, ring)) mbar_arrive(&sm.v_ask[vs]);
        }
      }
      // every load issued has landed before the CTA may exit (bounded): phase of
      // the last use of slot s among n uses of a ring of slots
      auto drain = [&](uint64_t *bar, int slots, int n) {
        for (int s = 0; s < slots && s < n; ++s)
          mbar_wait_bounded(&bar[s], ((n - 1 - s) / slots) & 1, v.err, RSWA_DEVERR_TIMEOUT);
      };
      drain(sm.q_full, NQ, active);
      drain(sm.k_full, NK, it);
      drain(sm.v_full, NV, it);
    }
  } else if (warp == kMma) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t el = tc::elect_one();
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      return __all_sync(0xffffffffu, wait_bar(bar, parity, v.err, dead)) != 0;
    };
    int it = 0, active = 0;
    uint32_t fit = 0;  // bit s: parity of V slot s's next v_fit
    bool ok = true;
    // O += P V of tile i, the first of its piece or not, into O buffer o
    auto pv = [&](int i, bool first, bool masked, int o) {
      const int s = i % NV;
      if (!wait(&sm.v_full[s], (i / NV) & 1)) return false;
      if (masked) {
        if (!wait(&sm.v_fit[s], (fit >> s) & 1u)) return false;
        fit ^= 1u << s;
      }
      if (!wait(&sm.p_full[i & 1], (i >> 1) & 1)) return false;
      tc::fence_after_sync();
      issue_pv<D, N>(el, tbase + S::kColO + (uint32_t)o * (2 * N), smem_u32(sm.p[i % S::kPBufs]),
                     smem_u32(sm.v[s]), !first);
      tc::commit_elected(el, &sm.v_empty[s]);
      tc::commit_elected(el, &sm.pv_done);
      return true;
    };
    for (int p = p_begin; ok && p < p_end; ++p) {
      const DecodePiece pc = p == p_begin ? first_piece : tv.pieces[p];
      if (tv.n[pc.b] <= row0) continue;
      const RingView ring = ring_view(v, pc.b, pc.plen);
      const PieceTiles pt(pc, ring);
      if (pt.n == 0) continue;
      const int qs = active % NQ;
      if (!(ok = wait(&sm.q_full[qs], (active / NQ) & 1))) break;
      if (v.rope && !(ok = wait(&sm.turned[qs], (active / NQ) & 1))) break;
      const int o = active & 1;
      for (int j = 0; ok && j < pt.n; ++j, ++it) {
        const int s = it % NK;
        if (!(ok = wait(&sm.k_full[s], (it / NK) & 1))) break;
        tc::fence_after_sync();
        // overwrites S of tile it - 2, which the softmax had read before its PV
        issue_qk<D, N>(el, tbase + (uint32_t)(it & 1) * N, smem_u32(sm.q[qs]), smem_u32(sm.k[s]));
        tc::commit_elected(el, &sm.s_full[it & 1]);
        tc::commit_elected(el, &sm.k_empty[s]);
        if (j == pt.n - 1) tc::commit_elected(el, &sm.q_free[qs]);
        if (j == 1 &&  // the results of the piece before the last are out of this O
            !(ok = wait(&sm.o_free[o], ((active >> 1) & 1) ^ 1)))
          break;
        if (j > 0 && !(ok = pv(it - 1, j == 1, pt.masked(j - 1, ring), o))) break;
      }
      if (ok && pt.n == 1) ok = wait(&sm.o_free[o], ((active >> 1) & 1) ^ 1);
      if (ok && (ok = pv(it - 1, pt.n == 1, pt.masked(pt.n - 1, ring), o)))
        tc::commit_elected(el, &sm.o_done[o]);
      ++active;
    }
    tc::commit_elected(el, &sm.mma_done);
    mbar_wait_bounded(&sm.mma_done, 0, v.err, RSWA_DEVERR_TIMEOUT);
    __syncwarp();
  } else if (warp >= kSide) {
    // ------------------------------------------------------------ side warps
    constexpr int kSideBar = 1 + S::kGroups;
    const int tid = (int)threadIdx.x - kSide * 32;  // 0..127: a row of a tile, a TMEM lane
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    // element of the output on this lane (64 rows of an MMA take 16 lanes a warp)
    const int elem = D == 128 ? tid : (warp & 3) * 16 + (lane & 15);
    const bool has_elem = D == 128 || lane < 16;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      wait_bar(bar, parity, v.err, dead);
      __syncwarp();
    };
    int it = 0, active = 0;
    uint32_t ask = 0;         // bit s: parity of V slot s's next v_ask
    int last = -1;            // the piece whose results are due
    bool last_mend = false;   // a value that is not finite was taken out of its V
    // The results of piece `last`: final where it is the ring's only one, else a partial.
    auto finish = [&]() {
      const DecodePiece pc = tv.pieces[last];
      const int o = (active - 1) & 1;
      const uint32_t parity = (uint32_t)((active - 1) >> 1) & 1u;
      const int n = min(tv.n[pc.b] - row0, N);
      const int64_t draft0 = (int64_t)pc.b * tv.T + row0;
      const uint32_t t_hi = tbase + lane_off + S::kColO + (uint32_t)o * (2 * N), t_lo = t_hi + N;
      wait(&sm.l_done[o], parity);
      if (tid < N) {
        const float l = (sm.sums[o][0][tid] + sm.sums[o][1][tid]) +
                        (sm.sums[o][2][tid] + sm.sums[o][3][tid]);
        sm.inv[tid] = 1.f / l;
        if (pc.count > 1 && tid < n) {
          const float m = sm.m[o][tid];
          tv.part_ml[(int64_t)last * tv.T + row0 + tid] =
              make_float2(m == -FLT_MAX ? -INFINITY : m, l);
        }
      }
      __syncwarp();
      wait(&sm.o_done[o], parity);
      tc::fence_after_sync();
      if (last_mend) {
        // what the scan took out, to the drafts that see it
        const RingView ring = ring_view(v, pc.b, pc.plen);
        const PieceTiles pt(pc, ring);
#pragma unroll 1
        for (int j = 0; j < pt.n; ++j) {
          if (!pt.masked(j, ring)) continue;
          const bool drafts = pt.is_drafts(j);
          const int held = min(kTile, drafts ? row0 + n : ring.held - pt.slot(j));
#pragma unroll 1
          for (int r = 0; r < held; ++r) {
            const float y = __bfloat162float(
                drafts ? a.vd[((draft0 - row0 + r) * v.H + pc.h) * D + elem]
                       : a.vc[(pc.row0 + pt.slot(j) + r) * (int64_t)D + elem]);
            if (!__any_sync(0xffffffffu, !isfinite(y))) continue;
            const uint4 below = drafts ? tv.below[draft0 - row0 + r] : make_uint4(0u, 0u, 0u, 0u);
            const int age = drafts ? 0 : slot_age(ring, pt.slot(j) + r);
#pragma unroll 1
            for (int c = 0; c < n; ++c) {
              const int i = row0 + c;
              const bool seen = drafts ? ((word_of(below, i >> 5) >> (i & 31)) & 1u) != 0u
                                       : age <= v.W - 1 - tv.depth[draft0 + c];
              if (!seen) continue;
              uint32_t u;
              tc::ld1(t_hi + (uint32_t)c, &u);
              tc::wait_ld();
              if (!isfinite(y)) u = __float_as_uint(__uint_as_float(u) + y);
              tc::st1(t_hi + (uint32_t)c, u);
              tc::wait_st();
            }
          }
        }
      }
      named_bar_sync(kSideBar, 128);  // sm.inv is written
      const bool whole = pc.count == 1;
      const int64_t step = whole ? (int64_t)v.H * D : D;  // elements from draft to draft
      __nv_bfloat16 *dst = a.out + (draft0 * v.H + pc.h) * D + elem;
      float *part = tv.part_o + ((int64_t)last * tv.T + row0) * D + elem;
#pragma unroll 1
      for (int c0 = 0; c0 < n; c0 += 8) {
        float x[8], x_lo[8];
        tc::ld8(t_hi + (uint32_t)c0, reinterpret_cast<uint32_t *>(x));
        tc::ld8(t_lo + (uint32_t)c0, reinterpret_cast<uint32_t *>(x_lo));
        tc::wait_ld();
#pragma unroll
        for (int c = 0; c < 8; ++c) x[c] += isfinite(x[c]) ? x_lo[c] : 0.f;
        const int left = has_elem ? n - c0 : 0;
        if (whole) {
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (c < left) dst[c * step] = __float2bfloat16_rn(x[c] * sm.inv[c0 + c]);
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (c < left) part[c * step] = x[c];
        }
        dst += 8 * step;
        part += 8 * step;
        __syncwarp();
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.o_free[o]);
      named_bar_sync(kSideBar, 128);  // sm.inv is read
      last = -1;
    };
    for (int p = p_begin; p < p_end; ++p) {
      const DecodePiece pc = p == p_begin ? first_piece : tv.pieces[p];
      const int n = tv.n[pc.b];
      if (n <= row0) continue;
      const RingView ring = ring_view(v, pc.b, pc.plen);
      const PieceTiles pt(pc, ring);
      const int64_t draft0 = (int64_t)pc.b * tv.T;
      if (pt.n == 0) {  // nothing to see in this piece
        if (pc.count > 1 && tid < N && row0 + tid < n)
          tv.part_ml[(int64_t)p * tv.T + row0 + tid] = make_float2(-INFINITY, 0.f);
        continue;
      }
      if (v.rope) {
        const int qs = active % NQ;
        wait(&sm.q_full[qs], (active / NQ) & 1);
        if (tid < N && row0 + tid < n)
          turn_row<D>(sm.q[qs], tid, N * 128, tv.cs + (draft0 + row0 + tid) * (D / 2));
        if (pt.drafts) {
          wait(&sm.k_full[it % NK], (it / NK) & 1);
          if (tid < n)
            turn_row<D>(sm.k[it % NK], tid, kHalfBytes, tv.cs + (draft0 + tid) * (D / 2));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.turned[qs]);
      }
      bool mend = false;
      for (int j = 0; j < pt.n; ++j, ++it) {
        if (pt.masked(j, ring)) {
          // V's rows that hold no entry become 0, and so do values that are not finite
          const int held = pt.is_drafts(j) ? n : ring.held - pt.slot(j);
          bool bad = false;
          const int vs = it % NV;
          // the load is under way, so v_full's phase before this one is over; and
          // none comes after it before v_fit
          wait(&sm.v_ask[vs], (ask >> vs) & 1u);
          ask ^= 1u << vs;
          wait(&sm.v_full[vs], (it / NV) & 1);
          uint8_t *vt = sm.v[vs];
          constexpr int kScan = 8;  // 16-byte chunks of a row looked at together
          for (int c0 = 0; c0 < D / 8; c0 += kScan) {
            uint4 u[kScan];
            uint32_t t = 0;
#pragma unroll
            for (int c = 0; c < kScan; ++c)
              u[c] = *reinterpret_cast<const uint4 *>(vt + chunk_at(tid, c0 + c, kHalfBytes));
#pragma unroll
            for (int c = 0; c < kScan; ++c)
              t |= not_finite(u[c].x) | not_finite(u[c].y) | not_finite(u[c].z) | not_finite(u[c].w);
            if (tid < held && !t) continue;
            bad |= tid < held;
#pragma unroll
            for (int c = 0; c < kScan; ++c)
              *reinterpret_cast<uint4 *>(vt + chunk_at(tid, c0 + c, kHalfBytes)) =
                  tid < held ? make_uint4(finite_part(u[c].x), finite_part(u[c].y),
                                          finite_part(u[c].z), finite_part(u[c].w))
                             : make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.v_fit[vs]);
          mend |= bar_red_or(kSideBar, 128, bad);
        }
        if (j == 0 && last >= 0) finish();
      }
      last = p;
      last_mend = mend;
      ++active;
    }
    if (last >= 0) finish();
  } else {
    // --------------------------------------------------------------- softmax
    const int group = warp >> 2;
    const int key = (int)threadIdx.x & 127;     // key row of the tile, and TMEM lane
    const int col0 = group * NC;                // first column of this thread
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const int bar_group = 1 + group;            // the group's hardware barrier
    const float sl2 = v.scale * kLog2e;
    const uint64_t sl2x2 = tc::f2_pack(sl2, sl2), minus1 = tc::f2_pack(-1.f, -1.f);
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      wait_bar(bar, parity, v.err, dead);
      __syncwarp();
    };
    int it = 0, active = 0;
    for (int p = p_begin; p < p_end; ++p) {
      const DecodePiece pc = p == p_begin ? first_piece : tv.pieces[p];
      const int n_all = tv.n[pc.b], n = min(n_all - row0, N);
      if (n <= 0) continue;
      const RingView ring = ring_view(v, pc.b, pc.plen);
      const PieceTiles pt(pc, ring);
      if (pt.n == 0) continue;
      const int64_t draft0 = (int64_t)pc.b * tv.T;
      const int o = active & 1;
      const uint32_t t_hi =
          tbase + lane_off + S::kColO + (uint32_t)o * (2 * N) + (uint32_t)col0;
      const uint32_t t_lo = t_hi + N;
      named_bar_sync(bar_group, 128);  // the previous piece's m is read
      // m starts below every score; a column that holds no draft never grows
      if (key < NC) {
        const int c = col0 + key;
        sm.neg_m[c] = c < n ? FLT_MAX : -FLT_MAX;
        sm.top[c] = INT_MIN;
        sm.depth[c] = (uint8_t)(c < n ? tv.depth[draft0 + row0 + c] : 0);
      }
      __syncwarp();
      named_bar_sync(bar_group, 128);
      uint64_t l2[NC / 2];  // sums of weights over this lane's keys
#pragma unroll
      for (int c = 0; c < NC / 2; ++c) l2[c] = 0;

      for (int j = 0; j < pt.n; ++j, ++it) {
        const bool masked = pt.masked(j, ring);
        const uint32_t t_s = tbase + lane_off + (uint32_t)(it & 1) * N + (uint32_t)col0;
        uint32_t sees = 0xffffffffu;  // bit c: draft row0 + col0 + c sees this key
        if (masked) {
          if (pt.is_drafts(j)) {
            sees = key < n_all ? word_of(tv.below[draft0 + key], (row0 + col0) >> 5) >> (col0 & 31)
                               : 0u;
          } else {
            const int age = slot_age(ring, pt.slot(j) + key);
            const int deepest = age == INT_MIN ? INT_MAX : age == INT_MAX ? -1 : v.W - 1 - age;
            if (deepest >= RSWA_TREE_MAX || deepest < 0) {
              sees = deepest < 0 ? 0u : 0xffffffffu;
            } else {
              // four depths at a time: a byte of ones where the draft sees the key,
              // of which byte i gives bit i
              sees = 0;
#pragma unroll
              for (int c = 0; c < NC; c += 4) {
                const uint32_t d4 = *reinterpret_cast<const uint32_t *>(&sm.depth[col0 + c]);
                const uint32_t le = __vcmpleu4(d4, (uint32_t)deepest * 0x01010101u);
                sees |= (((le & 0x08040201u) * 0x01010101u) >> 24) << c;
              }
            }
          }
        }
        wait(&sm.s_full[it & 1], (it >> 1) & 1);
        tc::fence_after_sync();
        float x[NC];
        // pass 0: the scores less m; where one exceeds it by more than kGrowth (as
        // in every first tile), pass 2 moves m and pass 3 is pass 0 again
#pragma unroll 1
        for (int pass = j == 0 ? 2 : 0;; ++pass) {
          load_cols<NC>(t_s, x);
          if (masked) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
              if (!((sees >> c) & 1u)) x[c] = -INFINITY;
          }
          if (pass == 2) {
            // the largest score of every draft in the tile; m moves to it where
            // it exceeds m by more than kGrowth, for each draft by its own scores
            if (j > 0) wait(&sm.pv_done, (it - 1) & 1);  // O is free
            tc::fence_after_sync();
            reduce_lanes<NC>(x, lane, [](float a, float b) { return fmaxf(a, b); });
            atomicMax(&sm.top[col0 + lane * NC / 32], ordered_int(__float_as_int(x[0])));
            named_bar_sync(bar_group, 128);
            if (key < NC) {
              const float mx = __int_as_float(ordered_int(sm.top[col0 + key]));
              sm.top[col0 + key] = INT_MIN;
              const float neg = sm.neg_m[col0 + key];
              const bool grew = fmaf(mx, sl2, neg) > kGrowth;
              const float m_new = mx * sl2;
              sm.alpha[col0 + key] = grew ? tc::ex2(-neg - m_new) : 1.f;
              if (grew) sm.neg_m[col0 + key] = -m_new;
            }
            __syncwarp();
            named_bar_sync(bar_group, 128);
#pragma unroll
            for (int c = 0; c < NC / 2; ++c)
              l2[c] = tc::fmul2(l2[c], *reinterpret_cast<const uint64_t *>(&sm.alpha[col0 + 2 * c]));
            if (j > 0) {
#pragma unroll 1
              for (int part = 0; part < 2; ++part) {
                const uint32_t t_o = part ? t_lo : t_hi;
                load_cols<NC>(t_o, x);
#pragma unroll
                for (int c = 0; c < NC; ++c) x[c] *= sm.alpha[col0 + c];
                store_cols<NC>(t_o, x);
              }
              tc::wait_st();
            }
            continue;
          }
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < NC; c += 4) {
            const ulonglong2 neg = *reinterpret_cast<const ulonglong2 *>(&sm.neg_m[col0 + c]);
            const uint64_t a0 = tc::ffma2(tc::f2_pack(x[c], x[c + 1]), sl2x2, neg.x);
            const uint64_t a1 = tc::ffma2(tc::f2_pack(x[c + 2], x[c + 3]), sl2x2, neg.y);
            x[c] = tc::f2_lo(a0);
            x[c + 1] = tc::f2_hi(a0);
            x[c + 2] = tc::f2_lo(a1);
            x[c + 3] = tc::f2_hi(a1);
            top = tc::fmax3(tc::fmax3(top, x[c], x[c + 1]), x[c + 2], x[c + 3]);
          }
          if (pass == 3 || !bar_red_or(bar_group, 128, top > kGrowth)) break;
          pass = 1;
        }
        // P: 2^x as hi + lo, both cut off (never rounded up), 8 drafts a chunk
        if (S::kPBufs == 1 && it > 0) wait(&sm.pv_done, (it - 1) & 1);
        uint8_t *pt_row = sm.p[it % S::kPBufs];
#pragma unroll
        for (int c = 0; c < NC; c += 8) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p0 = tc::ex2(x[c + 2 * e]), p1 = tc::ex2(x[c + 2 * e + 1]);
            const uint64_t pp = tc::f2_pack(p0, p1);
            l2[c / 2 + e] = tc::fadd2(l2[c / 2 + e], pp);
            hi[e] = __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);
            const uint64_t cut = tc::f2_pack(__uint_as_float(__float_as_uint(p0) & 0xffff0000u),
                                             __uint_as_float(__float_as_uint(p1) & 0xffff0000u));
            const uint64_t rest = tc::ffma2(cut, minus1, pp);  // exact
            lo[e] = __byte_perm(__float_as_uint(tc::f2_lo(rest)), __float_as_uint(tc::f2_hi(rest)),
                                0x7632);
          }
          *reinterpret_cast<uint4 *>(pt_row + chunk_at(key, (col0 + c) / 8, kHalfBytes)) =
              make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4 *>(pt_row + chunk_at(key, (N + col0 + c) / 8, kHalfBytes)) =
              make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        fence_proxy_async_smem();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[it & 1]);
      }
      // sums and m to the side warps
      float sum[NC];
#pragma unroll
      for (int c = 0; c < NC / 2; ++c) {
        sum[2 * c] = tc::f2_lo(l2[c]);
        sum[2 * c + 1] = tc::f2_hi(l2[c]);
      }
      reduce_lanes<NC>(sum, lane, [](float a, float b) { return a + b; });
      wait(&sm.o_free[o], ((active >> 1) & 1) ^ 1);  // those of two pieces ago are read
      sm.sums[o][warp & 3][col0 + lane * NC / 32] = sum[0];
      if (key < NC) sm.m[o][col0 + key] = -sm.neg_m[col0 + key];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.l_done[o]);
      ++active;
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kMma) tc::tmem_dealloc(tbase, S::kTmemCols);
}

template <int D, int N>
cudaError_t launch_t(const DeviceView &v, const TreeView &tv, const CUtensorMap &tkc,
                     const CUtensorMap &tvc, const void *q, const void *kd, const void *vd,
                     const void *vc, void *out, cudaStream_t s) {
  const int smem = (int)sizeof(TreeSmem<D, N>) + 1024;
  static_assert(sizeof(TreeSmem<D, N>) + 1024 <= 232448, "227 KB of shared memory a CTA");
  static bool attr_set[64] = {};  // per device
  const int dev = current_device();
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(tree_tc_kernel<D, N>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  const int64_t rows = (int64_t)v.B * tv.T, elems = (int64_t)v.H * D;
  const int box_rows = (tv.T + 7) / 8 * 8;  // whole 8-row swizzle atoms
  CUtensorMap tq, tk, tvv;
  if (!make_tmap_rows(&tq, q, rows, elems, N) || !make_tmap_rows(&tk, kd, rows, elems, box_rows) ||
      !make_tmap_rows(&tvv, vd, rows, elems, box_rows))
    return cudaErrorInvalidValue;
  const TreeTcArgs args{v, tv, (const __nv_bfloat16 *)vd, (const __nv_bfloat16 *)vc,
                        (__nv_bfloat16 *)out, box_rows};
  return launch_overlapped(tree_tc_kernel<D, N>, dim3((unsigned)tv.grid, (unsigned)((tv.T + N - 1) / N)),
                           dim3(Shape<D, N>::kThreads), (size_t)smem, s, tq, tk, tvv, tkc, tvc, args);
}

template <int D>
cudaError_t launch_d(const DeviceView &v, const TreeView &tv, const CUtensorMap &tkc,
                     const CUtensorMap &tvc, const void *q, const void *kd, const void *vd,
                     const void *vc, void *out, cudaStream_t s) {
  if (tv.T <= 16) return launch_t<D, 16>(v, tv, tkc, tvc, q, kd, vd, vc, out, s);
  if (tv.T <= 32) return launch_t<D, 32>(v, tv, tkc, tvc, q, kd, vd, vc, out, s);
  return launch_t<D, 64>(v, tv, tkc, tvc, q, kd, vd, vc, out, s);
}

}  // namespace

bool tree_tc_maps(const DeviceView &v, const void *kc, const void *vc, int64_t cache_rows,
                  CUtensorMap *tkc, CUtensorMap *tvc) {
  return cache_rows >= 1 && cache_rows < (int64_t(1) << 31) &&
         make_tmap_rows(tkc, kc, cache_rows, v.D, kTile) &&
         make_tmap_rows(tvc, vc, cache_rows, v.D, kTile);
}

cudaError_t launch_tree_tc(const DeviceView &v, const TreeView &tv, const CUtensorMap &tkc,
                           const CUtensorMap &tvc, const void *q, const void *kd, const void *vd,
                           const void *vc, void *out, cudaStream_t s) {
  return v.D == 128 ? launch_d<128>(v, tv, tkc, tvc, q, kd, vd, vc, out, s)
                    : launch_d<64>(v, tv, tkc, tvc, q, kd, vd, vc, out, s);
}

}  // namespace rswa
