// Attention of drafted tokens over the cache on CUDA cores (FP32 FMA): the
// fp32 path, whose 1e-5 bound the tensor cores' input types cannot meet.
//
// For draft i of a sequence, over the entries j that it may see (the cache's
// prompt and ring slots, and the drafts above it in the tree),
//   o_i = sum_j 2^(s_ij - m_i) v_j / sum_j 2^(s_ij - m_i),
//   s_ij = scale log2(e) q_i.k_j,  m_i = max_j s_ij,
// in one pass over K and V with the running (m, l, o) of the online softmax.
//
// The keys of all rings are cut into one range of tiles per CTA (the work
// plan of the tree), so one K/V byte is read once for all the drafts of a row
// group; a ring in several pieces leaves partials that tree_combine_kernel
// merges.  A tile is 64 keys: 256 threads form a 16 x 16 grid, each with
// kRows / 16 query rows x 4 keys of the scores, then the same rows x D / 16
// output columns.  Groups of 16 rows (fewer than 17 drafts) or 64.  Bound by
// FP32 FMA issue once a row group is full.
#include <cuda_runtime.h>
#include <math.h>

#include "internal.h"
#include "ptx.cuh"
#include "tree.cuh"

namespace rswa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kKeys = kTreeSimtTile;
constexpr int kThreads = 256;
constexpr float kMasked = -1.f;  // marks an unseen pair where a weight (>= 0) would stand

template <int D, int kRows>
struct SimtSmem {
  float q[kRows][D + 4];
  float k[kKeys][D + 4];
  float v[kKeys][D + 4];
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
};

// Elements 4 c .. 4 c + 3 of both halves of the row at `src` into dst, turned by
// the (cos, sin) table cs if there is one (rotate-half RoPE).
template <int D>
__device__ __forceinline__ void load_rotated(const float *src, float *dst, int c,
                                             const float2 *cs) {
  constexpr int N = 4;
  float a[N], b[N];
  Chunk<float>::widen(*reinterpret_cast<const uint4 *>(src + c * N), a);
  Chunk<float>::widen(*reinterpret_cast<const uint4 *>(src + c * N + D / 2), b);
#pragma unroll
  for (int e = 0; e < N; ++e) {
    float x = a[e], y = b[e];
    if (cs) {
      const float2 r = cs[c * N + e];
      x = a[e] * r.x - b[e] * r.y;
      y = b[e] * r.x + a[e] * r.y;
    }
    a[e] = x;
    b[e] = y;
  }
  *reinterpret_cast<float4 *>(dst + c * N) = make_float4(a[0], a[1], a[2], a[3]);
  *reinterpret_cast<float4 *>(dst + c * N + D / 2) = make_float4(b[0], b[1], b[2], b[3]);
}

template <int D, int kRows>
__global__ void __launch_bounds__(kThreads)
    tree_simt_kernel(const TreeSimtArgs a) {
  using Smem = SimtSmem<D, kRows>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
  constexpr int kRT = kRows / 16;       // rows of a thread
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
    for (int e = tid; e < kRows * (D / 2 / N); e += kThreads) {
      const int r = e / (D / 2 / N), c = e % (D / 2 / N);
      const int64_t i = draft0 + min(row0 + r, n - 1);
      load_rotated<D>(a.q + (i * v.H + pc.h) * D, sm.q[r], c,
                         v.rope ? tv.cs + i * (D / 2) : nullptr);
    }
    for (int r = tid; r < kRows; r += kThreads) {
      const int64_t i = draft0 + min(row0 + r, n - 1);
      sm.limit[r] = v.W - 1 - tv.depth[i];
      sm.above[r] = tv.above[i];
    }
    float m = -INFINITY, l = 0.f;  // of row tid / kTPR
    float acc[kRT][kCT * 4];
#pragma unroll
    for (int i = 0; i < kRT; ++i)
#pragma unroll
      for (int c = 0; c < kCT * 4; ++c) acc[i][c] = 0.f;

    for (int tl = pc.key_begin; tl < pc.key_end; ++tl) {
      const bool drafts = tl < n_draft_tiles;
      const int k0 = (drafts ? tl : tl - n_draft_tiles) * kKeys;  // first draft / slot
      const int nk = drafts ? min(kKeys, n - k0) : min(kKeys, ring.held - k0);
      if (nk <= 0 || (!drafts && k0 + kKeys <= ring.lo)) continue;  // nothing in it
      __syncthreads();  // the previous tile's products are done
      for (int e = tid; e < kKeys * (D / 2 / N); e += kThreads) {
        const int r = e / (D / 2 / N), c = e % (D / 2 / N);
        if (r >= nk) continue;  // masked below, its contents unused
        if (drafts) {
          const int64_t i = draft0 + k0 + r;
          const int64_t off = (i * v.H + pc.h) * D;
          load_rotated<D>(a.kd + off, sm.k[r], c,
                             v.rope ? tv.cs + i * (D / 2) : nullptr);
          load_rotated<D>(a.vd + off, sm.v[r], c, nullptr);
        } else {
          const int64_t off = (pc.row0 + k0 + r) * D;
          load_rotated<D>(a.kc + off, sm.k[r], c, nullptr);
          load_rotated<D>(a.vc + off, sm.v[r], c, nullptr);
        }
      }
      if (!drafts && tid < kKeys) sm.age[tid] = slot_age(ring, k0 + tid);
      __syncthreads();
      // scores of rows ty + 16 i against keys tx + 16 j
      float s[kRT][4];
#pragma unroll
      for (int i = 0; i < kRT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
      for (int c = 0; c < D; c += 4) {
        float4 qv[kRT], kv[4];
#pragma unroll
        for (int i = 0; i < kRT; ++i) qv[i] = *reinterpret_cast<const float4 *>(&sm.q[ty + 16 * i][c]);
#pragma unroll
        for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4 *>(&sm.k[tx + 16 * j][c]);
#pragma unroll
        for (int i = 0; i < kRT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[i][j] = fmaf(qv[i].x, kv[j].x, s[i][j]);
            s[i][j] = fmaf(qv[i].y, kv[j].y, s[i][j]);
            s[i][j] = fmaf(qv[i].z, kv[j].z, s[i][j]);
            s[i][j] = fmaf(qv[i].w, kv[j].w, s[i][j]);
          }
      }
#pragma unroll
      for (int i = 0; i < kRT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sm.p[ty + 16 * i][tx + 16 * j] = s[i][j] * qs;
      __syncthreads();
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
          const float w = see[j] ? exp2f(x[j] - sub_m) : kMasked;
          if (see[j]) lt += w;
          sm.p[r][sub + kTPR * j] = w;
        }
#pragma unroll
        for (int o = kTPR / 2; o > 0; o >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, o);
        l = l * corr + lt;
        m = m_new;
        if (sub == 0) sm.alpha[r] = corr;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kRT; ++i) {
        const float corr = sm.alpha[ty + 16 * i];
#pragma unroll
        for (int c = 0; c < kCT * 4; ++c) acc[i][c] *= corr;
      }
#pragma unroll 2
      for (int j0 = 0; j0 < nk; j0 += 4) {  // (rows of V behind the last entry have w < 0)
        float4 w4[kRT];
#pragma unroll
        for (int i = 0; i < kRT; ++i)
          w4[i] = *reinterpret_cast<const float4 *>(&sm.p[ty + 16 * i][j0]);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float4 vv[kCT];
#pragma unroll
          for (int c = 0; c < kCT; ++c)
            vv[c] = *reinterpret_cast<const float4 *>(&sm.v[j0 + u][tx * 4 + 64 * c]);
#pragma unroll
          for (int i = 0; i < kRT; ++i) {
            const float w = u == 0 ? w4[i].x : u == 1 ? w4[i].y : u == 2 ? w4[i].z : w4[i].w;
            if (w >= 0.f || w != w) {  // an unseen entry's value never enters, whatever it holds
#pragma unroll
              for (int c = 0; c < kCT; ++c) {
                acc[i][4 * c] = fmaf(w, vv[c].x, acc[i][4 * c]);
                acc[i][4 * c + 1] = fmaf(w, vv[c].y, acc[i][4 * c + 1]);
                acc[i][4 * c + 2] = fmaf(w, vv[c].z, acc[i][4 * c + 2]);
                acc[i][4 * c + 3] = fmaf(w, vv[c].w, acc[i][4 * c + 3]);
              }
            }
          }
        }
      }
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
        if (pc.count == 1) {
          const float sum = sm.alpha[ty + 16 * i];
          float *dst = a.out + ((draft0 + r) * v.H + pc.h) * D + e;
#pragma unroll
          for (int x = 0; x < 4; ++x) dst[x] = acc[i][4 * c + x] / sum;
        } else {
          *reinterpret_cast<float4 *>(tv.part_o + ((int64_t)p * tv.T + r) * D + e) =
              make_float4(acc[i][4 * c], acc[i][4 * c + 1], acc[i][4 * c + 2], acc[i][4 * c + 3]);
        }
      }
    }
  }
}

template <int D, int kRows>
cudaError_t set_attr() {
  return cudaFuncSetAttribute(tree_simt_kernel<D, kRows>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)sizeof(SimtSmem<D, kRows>));
}

template <int D, int kRows>
cudaError_t launch_t(const TreeSimtArgs &a, cudaStream_t s) {
  cudaError_t e = set_attr<D, kRows>();
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)a.tv.grid, (unsigned)((a.tv.T + kRows - 1) / kRows));
  return launch_overlapped(tree_simt_kernel<D, kRows>, grid, dim3(kThreads),
                           sizeof(SimtSmem<D, kRows>), s, a);
}

template <int D, int kRows>
int ctas_t() {
  int n = 0;
  if (set_attr<D, kRows>() != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, tree_simt_kernel<D, kRows>, kThreads,
                                                    sizeof(SimtSmem<D, kRows>)) != cudaSuccess ||
      n < 1)
    return 1;
  return n;
}

}  // namespace

int tree_simt_ctas_per_sm(int head_dim, int n_rows) {
  const bool small = n_rows <= 16;
  if (head_dim == 128) return small ? ctas_t<128, 16>() : ctas_t<128, 64>();
  return small ? ctas_t<64, 16>() : ctas_t<64, 64>();
}

cudaError_t launch_tree_simt(const DeviceView &v, const TreeView &tv, const float *q,
                             const float *kd, const float *vd, const float *kc, const float *vc,
                             float *out, cudaStream_t s) {
  const TreeSimtArgs a{v, tv, q, kd, vd, kc, vc, out};
  const bool small = tv.T <= 16;
  if (v.D == 128) return small ? launch_t<128, 16>(a, s) : launch_t<128, 64>(a, s);
  return small ? launch_t<64, 16>(a, s) : launch_t<64, 64>(a, s);
}

}  // namespace rswa
