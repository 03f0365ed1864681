// Attention of drafted tokens over the cache on CUDA cores (FP32 FMA): the
// fp32 path, whose 1e-5 bound the tensor cores' input types cannot meet.
//
// For draft i of a sequence, over the entries j that it may see (the cache's
// prompt and ring slots, and the drafts above it in the tree),
//   o_i = sum_j 2^(s_ij - m_i) v_j / sum_j 2^(s_ij - m_i),
//   s_ij = scale log2(e) q_i.k_j,
// in one pass over K and V.  The keys of all rings are cut into one range of
// tiles per CTA (the work plan of the tree); a ring in several pieces leaves
// partials that tree_combine_kernel merges.
//
// Up to 32 drafts: tree_rows_kernel, 16 of them a CTA.  A warp takes four drafts,
// their queries and outputs in registers, and four to sixteen keys at a time, d / 16
// lanes a key; bulk copies stream K and V rows into shared memory.  Every 16 bytes
// that leave shared memory meet four drafts, in packed FP32 pairs.  Bound by HBM up
// to 4 drafts (8 x 8,000 tokens, d = 128: 122 us, 84 % of the measured copy rate),
// by the latency of a key's chain (products, shuffles, exponential, products) with
// two warps a scheduler from 8 (4 x 4,096 tokens: 84 us for 16 drafts).
//
// More: tree_simt_kernel, row groups of 64.  A tile is 64 keys: 256 threads form
// a 16 x 16 grid, each with 4 query rows x 4 keys of the scores, then the same
// rows x D / 16 output columns.  Bound by FP32 FMA issue and the barriers between
// its phases.  4 x 4,096 tokens: 181 us for 33 to 64 drafts, where the rows kernel
// takes 157 for 32 and twice that for 64.
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>

#include "internal.h"
#include "ptx.cuh"
#include "tcgen05.cuh"
#include "tree.cuh"

namespace rswa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kKeys = kTreeSimtTile;
constexpr int kThreads = 256;
constexpr int kRowsMax = 32;      // drafts that tree_rows_kernel takes
constexpr int kRowsCta = 16;      // of them a CTA

template <int D>
struct SimtSmem {
  static constexpr int kRows = 64;
  float q[kRows][D + 4];
  // d = 128: one buffer, a tile's K until its scores are done, then its V, so that
  // two CTAs fit an SM (4 x 64 drafts over 4,096 tokens: 235 us became 205 by this
  // step alone, and 181 with those after it)
  static constexpr bool kShared = D == 128;
  float k[kKeys][D + 4];
  float v_own[kShared ? 1 : kKeys][D + 4];
  __device__ float (*v())[D + 4] { return kShared ? k : v_own; }
  float p[kRows][kKeys + 4];
  float alpha[kRows];
  int limit[kRows];     // W - 1 - depth of the row
  uint4 above[kRows];
  int age[kKeys];
};

struct TreeSimtArgs {
  DeviceView v;
  TreeView tv;
  const float *q, *kd, *vd, *kc, *vc;
  float *out;
  int row_base;  // rows kernel: the first draft of its grid's first row
};

template <int N>
struct Count {
  static constexpr int value = N;
};

// Elements 4 c .. 4 c + 3 of both halves of the row at `src` into dst, turned by
// the (cos, sin) table cs (rotate-half RoPE).
template <int D>
__device__ __forceinline__ void load_rotated(const float *src, float *dst, int c,
                                             const float2 *cs) {
  constexpr int N = 4;
  float a[N], b[N];
  Chunk<float>::widen(*reinterpret_cast<const uint4 *>(src + c * N), a);
  Chunk<float>::widen(*reinterpret_cast<const uint4 *>(src + c * N + D / 2), b);
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float2 r = cs[c * N + e];
    const float x = a[e] * r.x - b[e] * r.y, y = b[e] * r.x + a[e] * r.y;
    a[e] = x;
    b[e] = y;
  }
  *reinterpret_cast<float4 *>(dst + c * N) = make_float4(a[0], a[1], a[2], a[3]);
  *reinterpret_cast<float4 *>(dst + c * N + D / 2) = make_float4(b[0], b[1], b[2], b[3]);
}

// Two CTAs an SM: one's loads and softmax behind the other's products.
template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    tree_simt_kernel(const TreeSimtArgs a) {
  using Smem = SimtSmem<D>;
  constexpr int kRows = Smem::kRows;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
  constexpr int kCT = D / 64;           // groups of 4 output columns of a thread
  constexpr int kTPR = kThreads / kRows;  // threads of a row in the softmax
  constexpr int N = 4;  // elements of a 16-byte chunk
  const DeviceView &v = a.v;
  const TreeView &tv = a.tv;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int row0 = (int)blockIdx.y * kRows;
  const int n_draft_tiles = (tv.T + kKeys - 1) / kKeys;
  const float qs = v.scale * kLog2e;
  grid_dependency_wait();
  allow_dependents();

  for (int p = tv.cta_piece[blockIdx.x]; p < tv.cta_piece[blockIdx.x + 1]; ++p) {
    const DecodePiece pc = tv.pieces[p];
    const int n = tv.n[pc.b];
    if (row0 >= n) continue;  // no row of this group to compute
    const RingView ring = ring_view(v, pc.b, pc.plen);
    const int64_t draft0 = (int64_t)pc.b * tv.T;  // first draft's row of [B][T]
    __syncthreads();  // the previous piece is done with shared memory
    if (v.rope) {
      for (int e = tid; e < kRows * (D / 2 / N); e += kThreads) {
        const int r = e / (D / 2 / N), c = e % (D / 2 / N);
        const int64_t i = draft0 + min(row0 + r, n - 1);
        load_rotated<D>(a.q + (i * v.H + pc.h) * D, sm.q[r], c, tv.cs + i * (D / 2));
      }
    } else {
#pragma unroll
      for (int e = 0; e < kRows * (D / N) / kThreads; ++e) {
        const int at = tid + e * kThreads, r = at / (D / N), c = at % (D / N) * N;
        *reinterpret_cast<float4 *>(&sm.q[r][c]) = *reinterpret_cast<const float4 *>(
            a.q + ((draft0 + min(row0 + r, n - 1)) * v.H + pc.h) * D + c);
      }
    }
    for (int r = tid; r < kRows; r += kThreads) {
      const int64_t i = draft0 + min(row0 + r, n - 1);
      sm.limit[r] = v.W - 1 - tv.depth[i];
      sm.above[r] = tv.above[i];
    }
    // with rt rows a thread: no more than the sequence's drafts need
    auto run = [&](auto rt) {
      constexpr int kRT = decltype(rt)::value;
      float m = -INFINITY, l = 0.f;  // of row tid / kTPR
      uint64_t acc[kRT][kCT * 2];  // columns in pairs
#pragma unroll
      for (int i = 0; i < kRT; ++i)
#pragma unroll
        for (int c = 0; c < kCT * 2; ++c) acc[i][c] = 0;

      for (int tl = pc.key_begin; tl < pc.key_end; ++tl) {
        const bool drafts = tl < n_draft_tiles;
        const int k0 = (drafts ? tl : tl - n_draft_tiles) * kKeys;  // first draft / slot
        const int nk = drafts ? min(kKeys, n - k0) : min(kKeys, ring.held - k0);
        if (nk <= 0 || (!drafts && k0 + kKeys <= ring.lo)) continue;  // nothing in it
        __syncthreads();  // the previous tile's products are done
        // K and V: from memory to registers, every load in flight, and from there to
        // shared memory (0 behind the last entry)
        constexpr int kLoads = kKeys * (D / N) / kThreads;
        auto fetch = [&](const float *drafted, const float *cached, float4 *x) {
#pragma unroll
          for (int e = 0; e < kLoads; ++e) {
            const int at = tid + e * kThreads, r = at / (D / N), c = at % (D / N) * N;
            x[e] = r >= nk ? make_float4(0.f, 0.f, 0.f, 0.f)
                           : *reinterpret_cast<const float4 *>(
                                 drafts ? drafted + ((draft0 + k0 + r) * v.H + pc.h) * D + c
                                        : cached + (pc.row0 + k0 + r) * D + c);
          }
        };
        float4 vreg[kLoads];
        bool bad = false;  // a value that is not finite
        auto store_v = [&]() {
#pragma unroll
          for (int e = 0; e < kLoads; ++e) {
            const int at = tid + e * kThreads, r = at / (D / N), c = at % (D / N) * N;
            const float4 x = vreg[e];
            bad |= !isfinite(x.x) || !isfinite(x.y) || !isfinite(x.z) || !isfinite(x.w);
            *reinterpret_cast<float4 *>(&sm.v()[r][c]) = x;
          }
        };
        if constexpr (!Smem::kShared) fetch(a.vd, a.vc, vreg);
        if (drafts && v.rope) {
          for (int e = tid; e < nk * (D / 2 / N); e += kThreads) {
            const int r = e / (D / 2 / N), c = e % (D / 2 / N);
            const int64_t i = draft0 + k0 + r;
            load_rotated<D>(a.kd + (i * v.H + pc.h) * D, sm.k[r], c, tv.cs + i * (D / 2));
          }
        } else {
          float4 kreg[kLoads];
          fetch(a.kd, a.kc, kreg);
#pragma unroll
          for (int e = 0; e < kLoads; ++e) {
            const int at = tid + e * kThreads;
            *reinterpret_cast<float4 *>(&sm.k[at / (D / N)][at % (D / N) * N]) = kreg[e];
          }
        }
        if constexpr (!Smem::kShared) store_v();
        if (!drafts && tid < kKeys) sm.age[tid] = slot_age(ring, k0 + tid);
        __syncthreads();
        // scores of rows ty + 16 i against keys tx + 16 j
        float s[kRT][4];
#pragma unroll
        for (int i = 0; i < kRT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
        auto scores = [&](auto count) {  // of the first 16 J keys
          constexpr int J = decltype(count)::value;
#pragma unroll 4
          for (int c = 0; c < D; c += 4) {
            float4 qv[kRT], kv[J];
#pragma unroll
            for (int i = 0; i < kRT; ++i)
              qv[i] = *reinterpret_cast<const float4 *>(&sm.q[ty + 16 * i][c]);
#pragma unroll
            for (int j = 0; j < J; ++j)
              kv[j] = *reinterpret_cast<const float4 *>(&sm.k[tx + 16 * j][c]);
#pragma unroll
            for (int i = 0; i < kRT; ++i)
#pragma unroll
              for (int j = 0; j < J; ++j) {
                s[i][j] = fmaf(qv[i].x, kv[j].x, s[i][j]);
                s[i][j] = fmaf(qv[i].y, kv[j].y, s[i][j]);
                s[i][j] = fmaf(qv[i].z, kv[j].z, s[i][j]);
                s[i][j] = fmaf(qv[i].w, kv[j].w, s[i][j]);
              }
          }
        };
        if (nk <= 16)
          scores(Count<1>());
        else if (nk <= 32)
          scores(Count<2>());
        else
          scores(Count<4>());
#pragma unroll
        for (int i = 0; i < kRT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) sm.p[ty + 16 * i][tx + 16 * j] = s[i][j] * qs;
        __syncthreads();
        if constexpr (Smem::kShared) fetch(a.vd, a.vc, vreg);  // behind the softmax
        {
          // softmax of row r by kTPR neighbouring threads
          const int r = tid / kTPR, sub = tid % kTPR;
          const int limit = sm.limit[r];
          const uint4 ab = sm.above[r];
          const uint32_t word[4] = {ab.x, ab.y, ab.z, ab.w};
          bool see[kKeys / kTPR];
          float x[kKeys / kTPR], mt = -INFINITY;
#pragma unroll
          for (int j = 0; j < kKeys / kTPR; ++j) {
            const int key = sub + kTPR * j;
            x[j] = sm.p[r][key];
            if (drafts) {
              const int node = k0 + key;
              see[j] = key < nk && ((word[node >> 5 & 3] >> (node & 31)) & 1u);
            } else {
              see[j] = key < nk && sm.age[key] <= limit;
            }
            if (see[j]) mt = fmaxf(mt, x[j]);
          }
#pragma unroll
          for (int o = kTPR / 2; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
          const float m_new = fmaxf(m, mt);
          // a row that has seen nothing yet keeps m = -inf, l = 0
          const float sub_m = m_new == -INFINITY ? 0.f : m_new;
          const float corr = exp2f(m - sub_m);
          float lt = 0.f;
#pragma unroll
          for (int j = 0; j < kKeys / kTPR; ++j) {
            const float w = see[j] ? exp2f(x[j] - sub_m) : 0.f;
            lt += w;
            sm.p[r][sub + kTPR * j] = w;
          }
#pragma unroll
          for (int o = kTPR / 2; o > 0; o >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, o);
          l = l * corr + lt;
          m = m_new;
          if (sub == 0) sm.alpha[r] = corr;
        }
        if constexpr (Smem::kShared) store_v();
        bad = __syncthreads_or(bad) != 0;
#pragma unroll
        for (int i = 0; i < kRT; ++i) {
          const float corr = sm.alpha[ty + 16 * i];
#pragma unroll
          for (int c = 0; c < kCT * 2; ++c) acc[i][c] = tc::fmul2(acc[i][c], tc::f2_pack(corr, corr));
        }
        auto sees = [&](int row, int key) {
          if (!drafts) return key < nk && sm.age[key] <= sm.limit[row];
          const uint4 ab = sm.above[row];
          const int node = k0 + key, w = node >> 5;
          return key < nk &&
                 (((w == 0 ? ab.x : w == 1 ? ab.y : w == 2 ? ab.z : ab.w) >> (node & 31)) & 1u) != 0u;
        };
        auto products = [&](auto check) {
#pragma unroll 2
          for (int j0 = 0; j0 < nk; j0 += 4) {
            float4 w4[kRT];
#pragma unroll
            for (int i = 0; i < kRT; ++i)
              w4[i] = *reinterpret_cast<const float4 *>(&sm.p[ty + 16 * i][j0]);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              ulonglong2 vv[kCT];
#pragma unroll
              for (int c = 0; c < kCT; ++c)
                vv[c] = *reinterpret_cast<const ulonglong2 *>(&sm.v()[j0 + u][tx * 4 + 64 * c]);
#pragma unroll
              for (int i = 0; i < kRT; ++i) {
                const float w = u == 0 ? w4[i].x : u == 1 ? w4[i].y : u == 2 ? w4[i].z : w4[i].w;
                if (!decltype(check)::value || sees(ty + 16 * i, j0 + u)) {
                  const uint64_t w2 = tc::f2_pack(w, w);
#pragma unroll
                  for (int c = 0; c < kCT; ++c) {
                    acc[i][2 * c] = tc::ffma2(w2, vv[c].x, acc[i][2 * c]);
                    acc[i][2 * c + 1] = tc::ffma2(w2, vv[c].y, acc[i][2 * c + 1]);
                  }
                }
              }
            }
          }
        };
        // an unseen entry's weight is 0; where its value would make 0 x inf of that it
        // is left out one by one
        if (!bad)
          products(Count<0>());
        else
          products(Count<1>());
      }

      // the piece's result: final where it is the ring's only one, else a partial
      __syncthreads();
      if (tid % kTPR == 0) {
        const int r = tid / kTPR;
        if (pc.count == 1)
          sm.alpha[r] = l;
        else if (row0 + r < n)
          tv.part_ml[(int64_t)p * tv.T + row0 + r] = make_float2(m, l);
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kRT; ++i) {
        const int r = row0 + ty + 16 * i;
        if (r >= n) continue;
#pragma unroll
        for (int c = 0; c < kCT; ++c) {
          const int e = tx * 4 + 64 * c;
          float4 x = make_float4(tc::f2_lo(acc[i][2 * c]), tc::f2_hi(acc[i][2 * c]),
                                 tc::f2_lo(acc[i][2 * c + 1]), tc::f2_hi(acc[i][2 * c + 1]));
          if (pc.count == 1) {
            const float sum = sm.alpha[ty + 16 * i];
            x = make_float4(x.x / sum, x.y / sum, x.z / sum, x.w / sum);
            *reinterpret_cast<float4 *>(a.out + ((draft0 + r) * v.H + pc.h) * D + e) = x;
          } else {
            *reinterpret_cast<float4 *>(tv.part_o + ((int64_t)p * tv.T + r) * D + e) = x;
          }
        }
      }
    };
    const int rt = (min(kRows, n - row0) + 15) / 16;
    if (rt == 1)
      run(Count<1>());
    else if (rt == 2)
      run(Count<2>());
    else if (rt == 3)
      run(Count<3>());
    else
      run(Count<4>());
  }
}

// ------------------------------------------------------- up to 32 drafts
constexpr int kRowWarps = 8;            // (a ninth, for the copies, would cost 80 registers a thread)
constexpr int kPerWarp = 4;             // drafts of a warp
constexpr float kGrowth = 8.f;          // m moves past a score 2^8 above it

template <int D>
struct __align__(128) RowsSmem {
  static constexpr int kRows = 4096 / D;  // keys of a stage: 16 KB of K, and of V
  static constexpr int kStages = 5;
  float k[kStages][kRows * D], v[kStages][kRows * D];
  float red_o[kRowWarps][kPerWarp][D];
  float red_m[kRowWarps][kPerWarp], red_l[kRowWarps][kPerWarp];
  uint64_t full[kStages], empty[kStages];
};

// G groups of four drafts, 8 / G warps each.
template <int D, int G>
__global__ void __launch_bounds__(kRowWarps * 32, 1)
    tree_rows_kernel(const TreeSimtArgs a) {
  using Smem = RowsSmem<D>;
  constexpr int NST = Smem::kStages, kRows = Smem::kRows;
  constexpr int kWarps = kRowWarps / G;   // of a group
  constexpr int LK = D / 16, KG = 32 / LK;  // lanes of a key, keys of a warp
  constexpr int NP = 8;                   // pairs of a row's elements on a lane (4 chunks)
  constexpr int kPass = kWarps * KG;      // keys that a group takes at a time
  constexpr int KK = kRows >= 2 * kPass ? 2 : 1;  // times one or two a lane group
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
  const DeviceView &v = a.v;
  const TreeView &tv = a.tv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = a.row_base + (int)blockIdx.y * kRowsCta;  // this CTA's first draft
  const int p_begin = tv.cta_piece[blockIdx.x], p_end = tv.cta_piece[blockIdx.x + 1];
  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], kRowWarps);
    }
    fence_mbar_init();
  }
  __syncthreads();
  grid_dependency_wait();
  allow_dependents();
  // a piece's cache slots [k0, k1)
  auto slots = [&](const DecodePiece &pc, const RingView &ring, int &k0, int &k1) {
    k0 = max(max(0, pc.key_begin - 1) * kKeys, ring.lo);
    k1 = max(k0, min((pc.key_end - 1) * kKeys, ring.held));
  };

  // ------------------------------------------------------------------ copies
  // by warp 0, kStages - 1 ahead of the stage in use
  struct {
    int p, k0, k1, it;
    int64_t row0;
    bool on;
  } copy{p_begin, 0, 0, 0, 0, warp == 0};
  // test-only fault injection: no copies at all, so every wait runs out
  if ((*v.fault & RSWA_FAULT_DROP_DECODE_COPIES) != 0) copy.on = false;
  auto copy_next = [&]() {
    while (copy.on && copy.k0 >= copy.k1) {
      if (copy.p == p_end) {
        copy.on = false;
      } else {
        const DecodePiece pc = tv.pieces[copy.p++];
        if (tv.n[pc.b] <= row0) continue;
        slots(pc, ring_view(v, pc.b, pc.plen), copy.k0, copy.k1);
        copy.row0 = pc.row0;
      }
    }
    if (!copy.on) return;
    const int s = copy.it % NST;
    // (a free slot from the second round on: every warp is done with the stage
    // before the one in use, or soon)
    const bool free = mbar_wait_bounded(&sm.empty[s], ((copy.it / NST) & 1) ^ 1, v.err,
                                        RSWA_DEVERR_TIMEOUT);
    if (!__all_sync(0xffffffffu, free)) {
      copy.on = false;
      return;
    }
    if (lane == 0) {
      const uint32_t bytes =
          (uint32_t)min(kRows, copy.k1 - copy.k0) * (uint32_t)(D * sizeof(float));
      mbar_arrive_expect_tx(&sm.full[s], 2 * bytes);
      bulk_g2s(sm.k[s], a.kc + (copy.row0 + copy.k0) * D, bytes, &sm.full[s]);
      bulk_g2s(sm.v[s], a.vc + (copy.row0 + copy.k0) * D, bytes, &sm.full[s]);
    }
    __syncwarp();
    copy.k0 += kRows;
    ++copy.it;
  };
  if (warp == 0)
    for (int s = 0; s < NST - 1; ++s) copy_next();

  // --------------------------------------------------------------- consumers
  const int li = lane % LK, lg = lane / LK;      // lane of a key, key of the warp's
  // 16-byte chunk j of a lane's four.  Two keys of d = 64 share a quarter warp's
  // load: the odd one takes the chunks in another order, so the banks differ.
  auto chunk = [&](int j) { return li + LK * (D == 64 ? j ^ (lg & 1) : j); };
  const int group = warp / kWarps, wg = warp % kWarps;
  const float qs = v.scale * kLog2e;
  int it = 0;
  bool dead = false;
  for (int p = p_begin; p < p_end; ++p) {
    const DecodePiece pc = tv.pieces[p];
    const int n = tv.n[pc.b];
    if (n <= row0) continue;
    const RingView ring = ring_view(v, pc.b, pc.plen);
    const int64_t draft0 = (int64_t)pc.b * tv.T;
    // a lane's part of a row as packed pairs, turned at draft i's position if RoPE is on
    auto load_row = [&](const float *src, int64_t i, bool turn, uint64_t *x) {
      float f[2 * NP];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<float4 *>(f + 4 * j) =
            *reinterpret_cast<const float4 *>(src + chunk(j) * 4);
      if (turn && v.rope) {
        const float2 *cs = tv.cs + i * (D / 2);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 w = cs[chunk(j) * 4 + e];
            const float c0 = f[4 * j + e], c1 = f[4 * (j + 2) + e];
            f[4 * j + e] = c0 * w.x - c1 * w.y;
            f[4 * (j + 2) + e] = c1 * w.x + c0 * w.y;
          }
      }
#pragma unroll
      for (int j = 0; j < NP; ++j) x[j] = tc::f2_pack(f[2 * j], f[2 * j + 1]);
    };
    uint64_t q[kPerWarp][NP], o[kPerWarp][NP];
    float m[kPerWarp], l[kPerWarp];
    int limit[kPerWarp];
#pragma unroll
    for (int r = 0; r < kPerWarp; ++r) {
      const int64_t i = draft0 + min(row0 + group * kPerWarp + r, n - 1);
      load_row(a.q + (i * v.H + pc.h) * D, i, true, q[r]);
      limit[r] = v.W - 1 - tv.depth[i];
      m[r] = -FLT_MAX;
      l[r] = 0.f;
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        q[r][j] = tc::fmul2(q[r][j], tc::f2_pack(qs, qs));
        o[r][j] = 0;
      }
    }
    // a lane's part of the scores of one key, and the sums over a key's lanes
    auto dot = [&](const uint64_t *k, float *x) {
#pragma unroll
      for (int r = 0; r < kPerWarp; ++r) {
        uint64_t s0 = 0, s1 = 0;
#pragma unroll
        for (int j = 0; j < NP; j += 2) {
          s0 = tc::ffma2(q[r][j], k[j], s0);
          s1 = tc::ffma2(q[r][j + 1], k[j + 1], s1);
        }
        s0 = tc::fadd2(s0, s1);
        x[r] = tc::f2_lo(s0) + tc::f2_hi(s0);
      }
    };
    auto add_lanes = [&](auto count, float *x) {
      constexpr int N = decltype(count)::value;
#pragma unroll
      for (int off = 1; off < LK; off <<= 1)
#pragma unroll
        for (int e = 0; e < N * kPerWarp; ++e) x[e] += __shfl_xor_sync(0xffffffffu, x[e], off);
    };
    // x[4 c + r]: scores of N keys a lane group to weights.  seen: bit 4 c + r, draft
    // r sees key c; `all` if every bit of every lane is set
    auto weigh = [&](auto count, float *x, uint32_t seen, bool all) {
      constexpr int N = decltype(count)::value;
      bool grew = false;
#pragma unroll
      for (int e = 0; e < N * kPerWarp; ++e) {
        if (!all && !((seen >> e) & 1u)) x[e] = -INFINITY;
        grew |= x[e] - m[e % kPerWarp] > kGrowth;
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int e = 0; e < N * kPerWarp; ++e) {
          const int r = e % kPerWarp;
          if (x[e] - m[r] > kGrowth) {
            const float f = exp2f(m[r] - x[e]);
            m[r] = x[e];
            l[r] *= f;
#pragma unroll
            for (int j = 0; j < NP; ++j) o[r][j] = tc::fmul2(o[r][j], tc::f2_pack(f, f));
          }
        }
      }
#pragma unroll
      for (int e = 0; e < N * kPerWarp; ++e) {
        x[e] = exp2f(x[e] - m[e % kPerWarp]);
        l[e % kPerWarp] += x[e];
      }
    };
    auto gather = [&](const uint64_t *val, const float *w, uint32_t seen, bool all) {
#pragma unroll
      for (int r = 0; r < kPerWarp; ++r)
        if (all || ((seen >> r) & 1u)) {  // an unseen entry's value never enters, whatever it holds
#pragma unroll
          for (int j = 0; j < NP; ++j) o[r][j] = tc::ffma2(val[j], tc::f2_pack(w[r], w[r]), o[r][j]);
        }
    };
    auto from_smem = [&](const float *row, uint64_t *x) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const ulonglong2 u = *reinterpret_cast<const ulonglong2 *>(row + chunk(j) * 4);
        x[2 * j] = u.x;
        x[2 * j + 1] = u.y;
      }
    };

    if (pc.key_begin == 0) {
      for (int j0 = wg * KG; j0 < n; j0 += kPass) {
        const int key = j0 + lg;
        const int64_t i = draft0 + min(key, n - 1);
        uint32_t seen = 0;
#pragma unroll
        for (int r = 0; r < kPerWarp; ++r)
          if (key < n) {
            const int64_t q_row = draft0 + min(row0 + group * kPerWarp + r, n - 1);
            const uint32_t above = reinterpret_cast<const uint32_t *>(tv.above + q_row)[key >> 5];
            seen |= ((above >> (key & 31)) & 1u) << r;
          }
        uint64_t row[NP];
        float x[kPerWarp];
        load_row(a.kd + (i * v.H + pc.h) * D, i, true, row);
        dot(row, x);
        add_lanes(Count<1>(), x);
        weigh(Count<1>(), x, seen, false);
        load_row(a.vd + (i * v.H + pc.h) * D, i, false, row);
        gather(row, x, seen, false);
      }
    }
    int k0, k1;
    slots(pc, ring, k0, k1);
    for (; k0 < k1; k0 += kRows, ++it) {
      const int s = it % NST, rows = min(kRows, k1 - k0);
      const bool all = !ring.swa && rows == kRows && k0 + kRows <= ring.plen;
      if (!dead && !mbar_wait_bounded(&sm.full[s], (it / NST) & 1, v.err, RSWA_DEVERR_TIMEOUT))
        dead = true;
      dead = __any_sync(0xffffffffu, dead) != 0;
      if (!dead) {
#pragma unroll 1
        for (int r0 = wg * KG; r0 < rows; r0 += KK * kPass) {
          int key[KK];
          uint32_t seen = 0;
          float x[KK * kPerWarp];
#pragma unroll
          for (int c = 0; c < KK; ++c) {
            const int at = r0 + c * kPass + lg;
            key[c] = min(at, rows - 1);
            if (!all) {
              const int age = at < rows ? slot_age(ring, k0 + at) : INT_MAX;
#pragma unroll
              for (int r = 0; r < kPerWarp; ++r)
                seen |= (age <= limit[r] ? 1u : 0u) << (c * kPerWarp + r);
            }
          }
          uint64_t row[KK][NP];
#pragma unroll
          for (int c = 0; c < KK; ++c) from_smem(sm.k[s] + key[c] * D, row[c]);
#pragma unroll
          for (int c = 0; c < KK; ++c) dot(row[c], x + c * kPerWarp);
          add_lanes(Count<KK>(), x);
#pragma unroll
          for (int c = 0; c < KK; ++c) from_smem(sm.v[s] + key[c] * D, row[c]);
          weigh(Count<KK>(), x, seen, all);
#pragma unroll
          for (int c = 0; c < KK; ++c)
            gather(row[c], x + c * kPerWarp, seen >> (c * kPerWarp), all);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[s]);
      if (warp == 0) copy_next();
    }

    // the warp's lane groups, then the group's warps
#pragma unroll
    for (int r = 0; r < kPerWarp; ++r) {
      if (D == 64 && (lg & 1))
#pragma unroll
        for (int j = 0; j < NP; j += 4)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint64_t x = o[r][j + e];
            o[r][j + e] = o[r][j + 2 + e];
            o[r][j + 2 + e] = x;
          }
      float top = m[r];
#pragma unroll
      for (int off = LK; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      const float f = exp2f(m[r] - top);
      float lr = l[r] * f;
#pragma unroll
      for (int off = LK; off < 32; off <<= 1) lr += __shfl_xor_sync(0xffffffffu, lr, off);
      if (lane == 0) {
        sm.red_m[warp][r] = top;
        sm.red_l[warp][r] = lr;
      }
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        float x = tc::f2_lo(o[r][j]) * f, y = tc::f2_hi(o[r][j]) * f;
#pragma unroll
        for (int off = LK; off < 32; off <<= 1) {
          x += __shfl_xor_sync(0xffffffffu, x, off);
          y += __shfl_xor_sync(0xffffffffu, y, off);
        }
        if (lg == 0)
          *reinterpret_cast<float2 *>(&sm.red_o[warp][r][(li + LK * (j >> 1)) * 4 + (j & 1) * 2]) =
              make_float2(x, y);
      }
    }
    __syncwarp();
    named_bar_sync(1, kRowWarps * 32);
    for (int e = (int)threadIdx.x; e < G * kPerWarp * (D / 4); e += kRowWarps * 32) {
      const int i = e / (D / 4), c = e % (D / 4) * 4;
      if (row0 + i >= n) continue;
      const int w0 = i / kPerWarp * kWarps, r = i % kPerWarp;
      float top = -FLT_MAX;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm.red_m[w0 + w][r]);
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2f(sm.red_m[w0 + w][r] - top);
        const float4 x = *reinterpret_cast<const float4 *>(&sm.red_o[w0 + w][r][c]);
        sum = fmaf(f, sm.red_l[w0 + w][r], sum);
        acc.x = fmaf(f, x.x, acc.x);
        acc.y = fmaf(f, x.y, acc.y);
        acc.z = fmaf(f, x.z, acc.z);
        acc.w = fmaf(f, x.w, acc.w);
      }
      if (pc.count == 1) {
        *reinterpret_cast<float4 *>(a.out + ((draft0 + row0 + i) * v.H + pc.h) * D + c) =
            make_float4(acc.x / sum, acc.y / sum, acc.z / sum, acc.w / sum);
      } else {
        *reinterpret_cast<float4 *>(tv.part_o + ((int64_t)p * tv.T + row0 + i) * D + c) = acc;
        if (c == 0)
          tv.part_ml[(int64_t)p * tv.T + row0 + i] =
              make_float2(top == -FLT_MAX ? -INFINITY : top, sum);
      }
    }
    __syncwarp();
    named_bar_sync(1, kRowWarps * 32);  // the partials are read
  }
  // every copy issued has landed before the CTA may exit (bounded)
  for (int s = 0; s < NST && s < copy.it; ++s)
    mbar_wait_bounded(&sm.full[s], ((copy.it - 1 - s) / NST) & 1, v.err, RSWA_DEVERR_TIMEOUT);
}

template <typename Smem, void (*kKernel)(TreeSimtArgs)>
cudaError_t prepare_kernel() {
  static bool attr_set[64] = {};  // per device
  const int dev = current_device();
  if (dev >= 0 && dev < 64 && attr_set[dev]) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(
      kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem));
  if (e == cudaSuccess && dev >= 0 && dev < 64) attr_set[dev] = true;
  return e;
}

template <int D, int G>
cudaError_t launch_rows(const TreeSimtArgs &a, int rows, cudaStream_t s) {
  cudaError_t e = prepare_kernel<RowsSmem<D>, tree_rows_kernel<D, G>>();
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)a.tv.grid, (unsigned)((rows + kRowsCta - 1) / kRowsCta));
  return launch_overlapped(tree_rows_kernel<D, G>, grid, dim3(kRowWarps * 32),
                           sizeof(RowsSmem<D>), s, a);
}

// Whole groups of 64 drafts, and a rest of more than kRowsMax, by the tiled
// kernel; a smaller rest by the rows kernel (65 drafts as 64 + 1, not as 128).
template <int D>
cudaError_t launch_d(TreeSimtArgs a, cudaStream_t s) {
  constexpr int kRows = SimtSmem<D>::kRows;
  const int rest = a.tv.T % kRows;
  const bool split = rest > 0 && rest <= kRowsMax;
  const int groups = a.tv.T / kRows + (rest > 0 && !split ? 1 : 0);
  if (groups > 0) {
    cudaError_t e = prepare_kernel<SimtSmem<D>, tree_simt_kernel<D>>();
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)a.tv.grid, (unsigned)groups);
    e = launch_overlapped(tree_simt_kernel<D>, grid, dim3(kThreads), sizeof(SimtSmem<D>), s, a);
    if (e != cudaSuccess || !split) return e;
  }
  a.row_base = a.tv.T / kRows * kRows;
  if (rest <= 4) return launch_rows<D, 1>(a, rest, s);
  if (rest <= 8) return launch_rows<D, 2>(a, rest, s);
  return launch_rows<D, 4>(a, rest, s);
}

template <int D>
int ctas_d() {
  int n = 0;
  if (prepare_kernel<SimtSmem<D>, tree_simt_kernel<D>>() != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, tree_simt_kernel<D>, kThreads,
                                                    sizeof(SimtSmem<D>)) != cudaSuccess ||
      n < 1)
    return 1;
  return n;
}

}  // namespace

int tree_simt_ctas(int num_sms, int head_dim, int T) {
  // the rows kernel: one CTA an SM, its columns of the grid side by side
  if (T <= kRowsMax) return num_sms / ((T + kRowsCta - 1) / kRowsCta);
  return num_sms * (head_dim == 128 ? ctas_d<128>() : ctas_d<64>());
}

cudaError_t launch_tree_simt(const DeviceView &v, const TreeView &tv, const float *q,
                             const float *kd, const float *vd, const float *kc, const float *vc,
                             float *out, cudaStream_t s) {
  const TreeSimtArgs a{v, tv, q, kd, vd, kc, vc, out, 0};
  return v.D == 128 ? launch_d<128>(a, s) : launch_d<64>(a, s);
}

}  // namespace rswa
