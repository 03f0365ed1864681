// Attention of drafted tokens over the cache on the 5th-generation tensor
// cores (bf16, d = 64 or 128).
//
// For draft i of a sequence, over the entries j that it may see (the cache's
// prompt and ring slots, and the drafts above it in the tree),
//   o_i = sum_j 2^(s_ij - m_i) v_j / sum_j 2^(s_ij - m_i),
//   s_ij = scale log2(e) q_i.k_j,
// in one pass over K and V.  T drafts do 4 T d operations on the 4 d bytes of
// an entry, so up to T = 128 the tensor cores (about 250 operations a byte)
// wait for HBM: the kernel's job is to keep the copies coming.
//
// The 128-key tiles of all rings (a ring's drafts first, then its cache) are
// cut into one equal range per CTA, one CTA an SM; a ring in several pieces
// leaves partials that tree_combine_kernel merges.  Inside a CTA:
//   producer warp   K and V tiles by TMA (128-byte swizzle) into two rings of
//                   kStages slots, and the T query rows of each piece;
//   MMA warp        one thread: S = Q K^T into one of two TMEM buffers, a tile
//                   ahead of O += P V (P from TMEM);
//   softmax warps   ceil(T / 32): thread r owns query row r (TMEM lane r) and
//                   runs the online softmax in the log2 domain.  O is rescaled
//                   only when a running maximum grows by more than 2^8.
// The query tile is padded to the 128 rows of the MMA: rows past T hold what
// they hold, and no other row can see it.  P goes to the MMA as a bf16 pair
// hi + lo (relative error 2^-17; bf16 alone would add its 2^-9 to an output
// that is rounded to bf16 once): one more PV product, which the copies hide.
//
// A masked score becomes -inf, so its weight is 0, but 0 x inf is NaN inside
// an MMA.  In the tiles that hold masked entries (the drafts, and the tiles
// with ring slots) the softmax threads therefore take non-finite values out of
// V's shared-memory copy, and add them to the rows that do see them, by hand.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "internal.h"
#include "ptx.cuh"
#include "tcgen05.cuh"
#include "tmap.h"
#include "tree.cuh"

namespace rswa {
namespace {

constexpr int kTile = kTreeTcTile;           // keys per tile, and the MMA's query rows
constexpr int kHalfBytes = kTile * 64 * 2;   // one 64-column swizzled half: 16 KB
constexpr uint32_t kTmemCols = 512;          // S0, S1 (128 each), O (D)
constexpr uint32_t kColO = 256;
constexpr float kRescaleThreshold = 8.0f;    // log2 units
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxThreads = 192;

template <int D>
struct __align__(1024) TreeSmem {
  static constexpr int kTileBytes = D / 64 * kHalfBytes;
  static constexpr int kStages = D == 128 ? 3 : 6;  // 192 KB of K and V in flight
  uint8_t q[kTileBytes];
  uint8_t k[kStages][kTileBytes];
  uint8_t v[kStages][kTileBytes];
  uint64_t q_full, q_free;
  uint64_t k_full[kStages], k_empty[kStages];
  uint64_t v_full[kStages], v_empty[kStages];
  uint64_t s_full[2];  // S of a tile finished
  // P of a tile written, V's copy fit to use (one arrival a softmax warp).  Two,
  // since the softmax may finish a second tile while the MMA warp still waits for
  // the first one's V: S of a third tile is only issued after that PV.
  uint64_t p_full[2];
  // O += P V of a tile finished.  Waited for with one tile outstanding at most
  // (S of a tile in hand says that the PV of the tile before the last is done).
  uint64_t pv_done;
  uint64_t o_done;     // a piece's last PV finished
  uint64_t turned;     // RoPE: a piece's queries and drafted keys turned
  uint64_t soft;       // the softmax warps, one another
  uint64_t mma_done;
  uint32_t bad[4];     // rows of the V tile that held a non-finite value
  uint32_t tmem_base;
  int dead;
};

struct TreeTcArgs {
  DeviceView v;
  TreeView tv;
  const __nv_bfloat16 *vd, *vc;  // the values, for the ones that are not finite
  __nv_bfloat16 *out;
  int box_rows;  // rows of the query and draft boxes
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
};

// Byte offset of 16-byte chunk c of row r in a swizzled tile.
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return (uint32_t)(c >> 3) * kHalfBytes + (uint32_t)r * 128u +
         ((uint32_t)((c & 7) ^ (r & 7)) << 4);
}

// Turn row r of a swizzled tile by its (cos, sin) table (rotate-half RoPE).
template <int D>
__device__ __forceinline__ void turn_row(uint8_t *tile, int r, const float2 *cs) {
  for (int c = 0; c < D / 16; ++c) {
    uint4 *p0 = reinterpret_cast<uint4 *>(tile + chunk_at(r, c));
    uint4 *p1 = reinterpret_cast<uint4 *>(tile + chunk_at(r, c + D / 16));
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

// S = Q K^T (M = N = 128).
template <int D>
__device__ __forceinline__ void issue_qk(uint32_t d_tmem, uint32_t q_addr, uint32_t k_addr) {
  constexpr uint32_t idesc = tc::idesc_bf16_f32(kTile, kTile, false, false);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = (uint32_t)(kk >> 2) * kHalfBytes + (uint32_t)(kk & 3) * 32;
    tc::mma_ss(d_tmem, tc::sw128_desc(q_addr + off, 16, 1024),
               tc::sw128_desc(k_addr + off, 16, 1024), idesc, kk > 0);
  }
}

// O += (P_hi + P_lo) V (M = 128 rows, N = D, twice K = 128 keys).
template <int D>
__device__ __forceinline__ void issue_pv(uint32_t o_tmem, uint32_t p_tmem, uint32_t v_addr) {
  constexpr uint32_t idesc = tc::idesc_bf16_f32(kTile, D, false, true);
#pragma unroll
  for (int part = 0; part < 2; ++part)
#pragma unroll
    for (int kk = 0; kk < kTile / 16; ++kk)
      tc::mma_ts(o_tmem, p_tmem + (uint32_t)(part * 64 + kk * 8),
                 tc::sw128_desc(v_addr + (uint32_t)kk * 2048, kHalfBytes, 1024), idesc, 1u);
}

__device__ __forceinline__ bool finite_bf16(uint32_t x) { return (x & 0x7f80u) != 0x7f80u; }

template <int D>
__global__ void __launch_bounds__(kMaxThreads, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kd,
                   const __grid_constant__ CUtensorMap tm_vd, const __grid_constant__ CUtensorMap tm_kc,
                   const __grid_constant__ CUtensorMap tm_vc, const TreeTcArgs a) {
  using Smem = TreeSmem<D>;
  constexpr int NST = Smem::kStages;
  constexpr int kHalves = D / 64;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // dynamic shared memory is only 16-byte aligned: round up to 1024 for the swizzle atoms
  Smem &sm = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                       ~uintptr_t(1023));
  const DeviceView &v = a.v;
  const TreeView &tv = a.tv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_soft = (int)(blockDim.x >> 5) - 2;  // softmax warps
  const int producer_warp = n_soft, mma_warp = n_soft + 1;
  const int p_begin = tv.cta_piece[blockIdx.x], p_end = tv.cta_piece[blockIdx.x + 1];

  if (threadIdx.x == 0) {
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_free, 1);
    for (int s = 0; s < NST; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.k_empty[s], 1);
      mbar_init(&sm.v_full[s], 1);
      mbar_init(&sm.v_empty[s], 1);
    }
    mbar_init(&sm.s_full[0], 1);
    mbar_init(&sm.s_full[1], 1);
    mbar_init(&sm.p_full[0], (uint32_t)n_soft);
    mbar_init(&sm.p_full[1], (uint32_t)n_soft);
    mbar_init(&sm.pv_done, 1);
    mbar_init(&sm.o_done, 1);
    mbar_init(&sm.turned, (uint32_t)n_soft);
    mbar_init(&sm.soft, (uint32_t)n_soft);
    mbar_init(&sm.mma_done, 1);
    sm.dead = 0;
    fence_mbar_init();
  }
  if (warp == mma_warp) {
    tc::tmem_alloc(&sm.tmem_base, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = sm.tmem_base;
  volatile int *dead = &sm.dead;

  if (warp == producer_warp) {
    // -------------------------------------------------------------- producer
    // test-only fault injection: no loads at all, so every wait runs out
    const bool drop = (*v.fault & RSWA_FAULT_DROP_DECODE_COPIES) != 0;
    if (lane == 0 && !drop) {
      tc::prefetch_tmap(&tm_q);
      tc::prefetch_tmap(&tm_kc);
      tc::prefetch_tmap(&tm_vc);
      const uint32_t box_bytes = (uint32_t)a.box_rows * 128u * kHalves;
      int it = 0, active = 0;
      bool ok = true;
      for (int p = p_begin; ok && p < p_end; ++p) {
        const DecodePiece pc = tv.pieces[p];
        if (tv.n[pc.b] == 0) continue;
        const PieceTiles pt(pc, ring_view(v, pc.b, pc.plen));
        if (pt.n == 0) continue;
        if (!(ok = wait_bar(&sm.q_free, (active & 1) ^ 1, v.err, dead))) break;
        const int xh = pc.h * D, y_draft = pc.b * tv.T;
        mbar_arrive_expect_tx(&sm.q_full, box_bytes);
        for (int x = 0; x < kHalves; ++x)
          tc::tma_load_2d(sm.q + x * kHalfBytes, &tm_q, xh + 64 * x, y_draft, &sm.q_full);
        ++active;
        for (int j = 0; j < pt.n; ++j, ++it) {
          const bool drafts = pt.drafts && j == 0;
          const int s = it % NST;
          const uint32_t parity = ((it / NST) & 1) ^ 1;
          const uint32_t bytes = drafts ? box_bytes : (uint32_t)Smem::kTileBytes;
          const int x0 = drafts ? xh : 0;
          const int y0 = drafts ? y_draft : (int)(pc.row0 + (int64_t)(pt.c0 + j - pt.drafts) * kTile);
          if (!(ok = wait_bar(&sm.k_empty[s], parity, v.err, dead))) break;
          mbar_arrive_expect_tx(&sm.k_full[s], bytes);
          for (int x = 0; x < kHalves; ++x)
            tc::tma_load_2d(sm.k[s] + x * kHalfBytes, drafts ? &tm_kd : &tm_kc, x0 + 64 * x, y0,
                            &sm.k_full[s]);
          if (!(ok = wait_bar(&sm.v_empty[s], parity, v.err, dead))) {
            mbar_wait_bounded(&sm.k_full[s], (it / NST) & 1, v.err, RSWA_DEVERR_TIMEOUT);
            break;
          }
          mbar_arrive_expect_tx(&sm.v_full[s], bytes);
          for (int x = 0; x < kHalves; ++x)
            tc::tma_load_2d(sm.v[s] + x * kHalfBytes, drafts ? &tm_vd : &tm_vc, x0 + 64 * x, y0,
                            &sm.v_full[s]);
        }
      }
      // every load issued has landed before the CTA may exit (bounded)
      if (active > 0)
        mbar_wait_bounded(&sm.q_full, (active - 1) & 1, v.err, RSWA_DEVERR_TIMEOUT);
      for (int s = 0; s < NST && s < it; ++s) {
        const int last = s + ((it - 1 - s) / NST) * NST;
        mbar_wait_bounded(&sm.k_full[s], (last / NST) & 1, v.err, RSWA_DEVERR_TIMEOUT);
        mbar_wait_bounded(&sm.v_full[s], (last / NST) & 1, v.err, RSWA_DEVERR_TIMEOUT);
      }
    }
  } else if (warp == mma_warp) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t q_addr = smem_u32(sm.q);
      int it = 0, active = 0;
      bool ok = true;
      auto pv = [&](int i) {  // O += P V of tile i
        const int s = i % NST;
        if (!wait_bar(&sm.v_full[s], (i / NST) & 1, v.err, dead)) return false;
        if (!wait_bar(&sm.p_full[i & 1], (i >> 1) & 1, v.err, dead)) return false;
        tc::fence_after_sync();
        issue_pv<D>(tbase + kColO, tbase + (uint32_t)(i & 1) * kTile, smem_u32(sm.v[s]));
        tc::commit(&sm.v_empty[s]);
        tc::commit(&sm.pv_done);
        return true;
      };
      for (int p = p_begin; ok && p < p_end; ++p) {
        const DecodePiece pc = tv.pieces[p];
        if (tv.n[pc.b] == 0) continue;
        const PieceTiles pt(pc, ring_view(v, pc.b, pc.plen));
        if (pt.n == 0) continue;
        if (!(ok = wait_bar(&sm.q_full, active & 1, v.err, dead))) break;
        if (v.rope && !(ok = wait_bar(&sm.turned, active & 1, v.err, dead))) break;
        ++active;
        for (int j = 0; ok && j < pt.n; ++j, ++it) {
          const int s = it % NST;
          if (!(ok = wait_bar(&sm.k_full[s], (it / NST) & 1, v.err, dead))) break;
          tc::fence_after_sync();
          // overwrites P of tile it - 2, whose PV was issued before
          issue_qk<D>(tbase + (uint32_t)(it & 1) * kTile, q_addr, smem_u32(sm.k[s]));
          tc::commit(&sm.s_full[it & 1]);
          tc::commit(&sm.k_empty[s]);
          if (j == pt.n - 1) tc::commit(&sm.q_free);
          if (j > 0) ok = pv(it - 1);
        }
        if (ok && (ok = pv(it - 1))) tc::commit(&sm.o_done);
      }
      tc::commit(&sm.mma_done);
      mbar_wait_bounded(&sm.mma_done, 0, v.err, RSWA_DEVERR_TIMEOUT);
    }
  } else {
    // --------------------------------------------------------------- softmax
    const int row = (int)threadIdx.x;  // query row and TMEM lane
    const int n_threads = n_soft * 32;
    uint32_t met = 0;  // parity of the next meeting of the softmax warps
    // a barrier of the softmax warps; false once a wait has run out anywhere
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.soft);
      const bool all = __all_sync(0xffffffffu, wait_bar(&sm.soft, met, v.err, dead));
      met ^= 1u;
      return all;
    };
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    const uint32_t t_o = tbase + lane_off + kColO;
    const float sl2 = v.scale * kLog2e;
    int it = 0, active = 0;
    bool ok = true;
    for (int p = p_begin; ok && p < p_end; ++p) {
      const DecodePiece pc = tv.pieces[p];
      const int n = tv.n[pc.b];
      if (n == 0) continue;
      const RingView ring = ring_view(v, pc.b, pc.plen);
      const PieceTiles pt(pc, ring);
      const int64_t draft0 = (int64_t)pc.b * tv.T;
      if (pt.n == 0) {  // nothing to see in this piece
        if (pc.count > 1 && row < n)
          tv.part_ml[(int64_t)p * tv.T + row] = make_float2(-INFINITY, 0.f);
        continue;
      }
      const int64_t my = draft0 + min(row, n - 1);
      const int limit = v.W - 1 - tv.depth[my];
      const uint4 ab = tv.above[my];
      const uint32_t above[4] = {ab.x, ab.y, ab.z, ab.w};
      if (v.rope) {
        ok = wait_bar(&sm.q_full, active & 1, v.err, dead);
        if (ok && row < n) turn_row<D>(sm.q, row, tv.cs + my * (D / 2));
        if (ok && pt.drafts) {
          ok = wait_bar(&sm.k_full[it % NST], (it / NST) & 1, v.err, dead);
          if (ok && row < n) turn_row<D>(sm.k[it % NST], row, tv.cs + my * (D / 2));
        }
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.turned);
      }
      ++active;
      {
        // O = 0 (every PV of the piece accumulates)
        uint32_t zero[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) zero[c] = 0u;
#pragma unroll
        for (int c4 = 0; c4 < D / 32; ++c4) tc::st32(t_o + 32 * c4, zero);
      }
      float m_run = -INFINITY, l_run = 0.f;
      for (int j = 0; j < pt.n; ++j, ++it) {
        const bool drafts = pt.drafts && j == 0;
        const int k0 = drafts ? 0 : (pt.c0 + j - pt.drafts) * kTile;  // first draft / slot
        const bool masked = drafts || ring.swa || k0 + kTile > ring.plen;
        const uint32_t t_s = tbase + lane_off + (uint32_t)(it & 1) * kTile;
        ok = __all_sync(0xffffffffu, wait_bar(&sm.s_full[it & 1], (it >> 1) & 1, v.err, dead));
        if (!ok) break;
        tc::fence_after_sync();
        float s[kTile];
#pragma unroll
        for (int c = 0; c < kTile; c += 32) tc::ld32(t_s + c, reinterpret_cast<uint32_t *>(s) + c);
        tc::wait_ld();
        // whether this row sees column c of the tile
        auto sees = [&](int c) {
          if (drafts) return ((above[c >> 5] >> (c & 31)) & 1u) != 0u;
          const int age = slot_age(ring, k0 + c);
          return age <= limit;
        };
        if (masked) {
          if (drafts) {
#pragma unroll
            for (int c = 0; c < kTile; ++c)
              if (!((above[c >> 5] >> (c & 31)) & 1u)) s[c] = -INFINITY;
          } else {
#pragma unroll
            for (int c = 0; c < kTile; ++c)
              if (slot_age(ring, k0 + c) > limit) s[c] = -INFINITY;
          }
        }
        // row max as an 8-way tree
        float mx8[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) mx8[i] = s[i];
#pragma unroll
        for (int c = 8; c < kTile; c += 2)
          mx8[(c >> 1) & 7] = tc::fmax3(mx8[(c >> 1) & 7], s[c], s[c + 1]);
        float mx = tc::fmax3(tc::fmax3(mx8[0], mx8[1], mx8[2]), tc::fmax3(mx8[3], mx8[4], mx8[5]),
                             fmaxf(mx8[6], mx8[7]));
        mx *= sl2;
        const float m_new = fmaxf(m_run, mx);
        const bool first = j == 0;
        // each row by its own scores: another row's change nothing of its result
        const bool grew = !first && row < n && m_new > m_run + kRescaleThreshold;
        const bool rescale = __any_sync(0xffffffffu, grew);
        const float m_use = first || grew ? m_new : m_run;
        const float alpha = grew ? tc::ex2(m_run - m_new) : 1.f;
        // a row that has seen nothing yet has m = -inf: its p are 2^-inf = 0
        const float m_sub = m_use == -INFINITY ? 0.f : m_use;
        const uint64_t sl2x2 = tc::f2_pack(sl2, sl2), negm2 = tc::f2_pack(-m_sub, -m_sub);
        uint64_t rs4[4];  // row sum as 4 packed pairs of partial sums
#pragma unroll
        for (int i = 0; i < 4; ++i) rs4[i] = 0;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t hi[32], lo[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const uint64_t xx = tc::ffma2(tc::f2_pack(s[64 * half + 2 * c], s[64 * half + 2 * c + 1]),
                                          sl2x2, negm2);
            const float p0 = tc::ex2(tc::f2_lo(xx)), p1 = tc::ex2(tc::f2_hi(xx));
            rs4[c & 3] = tc::fadd2(rs4[c & 3], tc::f2_pack(p0, p1));
            hi[c] = tc::pack_bf16x2(p0, p1);
            lo[c] = tc::pack_bf16x2(p0 - __uint_as_float(hi[c] << 16),
                                    p1 - __uint_as_float(hi[c] & 0xffff0000u));
          }
          tc::st32(t_s + 32 * half, hi);
          tc::st32(t_s + 64 + 32 * half, lo);
        }
        const uint64_t r01 = tc::fadd2(tc::fadd2(rs4[0], rs4[1]), tc::fadd2(rs4[2], rs4[3]));
        l_run = l_run * alpha + tc::f2_lo(r01) + tc::f2_hi(r01);
        m_run = m_use;
        if (rescale) {
          // O may only be touched between PV of the tile before and this tile's
          ok = __all_sync(0xffffffffu, wait_bar(&sm.pv_done, (it - 1) & 1, v.err, dead));
          if (!ok) break;
          tc::fence_after_sync();
#pragma unroll
          for (int c4 = 0; c4 < D / 32; ++c4) {
            float o[32];
            tc::ld32(t_o + 32 * c4, reinterpret_cast<uint32_t *>(o));
            tc::wait_ld();
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] *= alpha;
            tc::st32(t_o + 32 * c4, reinterpret_cast<const uint32_t *>(o));
          }
        }
        if (masked) {
          // V's rows that hold no entry become 0, and so do values that are not finite
          const int held = drafts ? n : ring.held - k0;
          ok = __all_sync(0xffffffffu,
                          wait_bar(&sm.v_full[it % NST], (it / NST) & 1, v.err, dead));
          if (!ok) break;
          uint8_t *vt = sm.v[it % NST];
          if (!(ok = meet())) break;  // sm.bad of the previous masked tile is read
          for (int r = row; r < kTile; r += n_threads) {
            bool bad = false;
#pragma unroll 4
            for (int c = 0; c < D / 8; ++c) {
              uint4 *at = reinterpret_cast<uint4 *>(vt + chunk_at(r, c));
              uint4 u = *at;
              uint32_t w[4] = {u.x, u.y, u.z, u.w};
              bool touched = false;
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const bool f0 = finite_bf16(w[x]), f1 = finite_bf16(w[x] >> 16);
                if (!f0) w[x] &= 0xffff0000u;
                if (!f1) w[x] &= 0x0000ffffu;
                touched |= !f0 || !f1;
              }
              if (r >= held) {
                *at = make_uint4(0u, 0u, 0u, 0u);
              } else if (touched) {
                *at = make_uint4(w[0], w[1], w[2], w[3]);
                bad = true;
              }
            }
            const uint32_t word = __ballot_sync(0xffffffffu, bad);
            if (lane == 0) sm.bad[r >> 5] = word;
          }
          fence_proxy_async_smem();
          if (!(ok = meet())) break;
          if ((sm.bad[0] | sm.bad[1] | sm.bad[2] | sm.bad[3]) != 0u) {
            if (!first) {
              ok = __all_sync(0xffffffffu, wait_bar(&sm.pv_done, (it - 1) & 1, v.err, dead));
              if (!ok) break;
            }
            tc::fence_after_sync();
            for (int r = 0; r < kTile; ++r) {
              if (!((sm.bad[r >> 5] >> (r & 31)) & 1u)) continue;
              const bool seen = row < n && sees(r);
              const __nv_bfloat16 *src = drafts ? a.vd + ((draft0 + r) * v.H + pc.h) * D
                                                : a.vc + (pc.row0 + k0 + r) * (int64_t)D;
              for (int c4 = 0; c4 < D / 32; ++c4) {
                float o[32];
                tc::wait_st();
                tc::ld32(t_o + 32 * c4, reinterpret_cast<uint32_t *>(o));
                tc::wait_ld();
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                  const float x = __bfloat162float(src[32 * c4 + c]);
                  if (seen && !isfinite(x)) o[c] += x;
                }
                tc::st32(t_o + 32 * c4, reinterpret_cast<const uint32_t *>(o));
              }
            }
          }
        }
        tc::wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[it & 1]);
      }
      if (!ok) break;
      // the piece's result: final where it is the ring's only one, else a partial
      ok = __all_sync(0xffffffffu, wait_bar(&sm.o_done, (active - 1) & 1, v.err, dead));
      if (!ok) break;
      tc::fence_after_sync();
      // Tiles without masks keep their non-finite values, and P_hi and P_lo may
      // turn an infinity into NaN (inf - inf, 0 inf): sum those values by hand.
      const int plain0 = pt.c0 * kTile;
      const int plain1 =
          ring.swa ? plain0 : (pt.c0 + min(pt.n - pt.drafts, ring.plen / kTile - pt.c0)) * kTile;
      bool stray = false;
#pragma unroll
      for (int c4 = 0; c4 < D / 32; ++c4) {
        float o[32];
        tc::ld32(t_o + 32 * c4, reinterpret_cast<uint32_t *>(o));
        tc::wait_ld();
#pragma unroll
        for (int c = 0; c < 32; ++c) stray |= o[c] != o[c];
      }
      // a row whose scores hold a NaN is NaN
      const bool mend = row < n && l_run == l_run;
      if (plain1 > plain0 && __any_sync(0xffffffffu, stray && mend)) {
        const __nv_bfloat16 *src = a.vc + (pc.row0 + plain0) * (int64_t)D;
#pragma unroll 1
        for (int c = 0; c < D; ++c) {
          uint32_t u;
          tc::ld1(t_o + c, &u);
          tc::wait_ld();
          const float x = __uint_as_float(u);
          if (!__any_sync(0xffffffffu, mend && x != x)) continue;
          float sum = 0.f;
          for (int r = lane; r < plain1 - plain0; r += 32) {
            const float y = __bfloat162float(src[(int64_t)r * D + c]);
            if (!isfinite(y)) sum += y;
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          if (mend && x != x && !isfinite(sum)) u = __float_as_uint(sum);
          tc::st1(t_o + c, u);
        }
        tc::wait_st();
      }
      const bool final_row = pc.count == 1;
      if (!final_row && row < n) tv.part_ml[(int64_t)p * tv.T + row] = make_float2(m_run, l_run);
      float *po = tv.part_o + ((int64_t)p * tv.T + row) * D;
      __nv_bfloat16 *dst = a.out + ((draft0 + row) * v.H + pc.h) * D;
#pragma unroll
      for (int c4 = 0; c4 < D / 32; ++c4) {
        float o[32];
        tc::ld32(t_o + 32 * c4, reinterpret_cast<uint32_t *>(o));
        tc::wait_ld();
        if (row >= n) continue;
        if (final_row) {
          uint4 *d4 = reinterpret_cast<uint4 *>(dst + 32 * c4);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = o[8 * c + e] / l_run;
            d4[c] = Chunk<__nv_bfloat16>::narrow(x);
          }
        } else {
          float4 *d4 = reinterpret_cast<float4 *>(po + 32 * c4);
#pragma unroll
          for (int c = 0; c < 8; ++c)
            d4[c] = make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
        }
      }
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == mma_warp) tc::tmem_dealloc(tbase, kTmemCols);
}

template <int D>
cudaError_t launch_t(const DeviceView &v, const TreeView &tv, const CUtensorMap &tkc,
                     const CUtensorMap &tvc, const void *q, const void *kd, const void *vd,
                     const void *vc, void *out, cudaStream_t s) {
  const int smem = (int)sizeof(TreeSmem<D>) + 1024;
  static bool attr_set[64] = {};  // per device
  const int dev = current_device();
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(tree_tc_kernel<D>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  const int box_rows = (tv.T + 7) / 8 * 8;  // whole 8-row swizzle atoms
  const int64_t rows = (int64_t)v.B * tv.T, elems = (int64_t)v.H * D;
  CUtensorMap tq, tk, tvv;
  if (!make_tmap_rows(&tq, q, rows, elems, box_rows) ||
      !make_tmap_rows(&tk, kd, rows, elems, box_rows) ||
      !make_tmap_rows(&tvv, vd, rows, elems, box_rows))
    return cudaErrorInvalidValue;
  const TreeTcArgs args{v, tv, (const __nv_bfloat16 *)vd, (const __nv_bfloat16 *)vc,
                        (__nv_bfloat16 *)out, box_rows};
  const int threads = ((tv.T + 31) / 32 + 2) * 32;
  tree_tc_kernel<D><<<tv.grid, threads, smem, s>>>(tq, tk, tvv, tkc, tvc, args);
  return cudaGetLastError();
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
  return v.D == 128 ? launch_t<128>(v, tv, tkc, tvc, q, kd, vd, vc, out, s)
                    : launch_t<64>(v, tv, tkc, tvc, q, kd, vd, vc, out, s);
}

}  // namespace rswa
