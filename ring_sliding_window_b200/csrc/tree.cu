// Trees of drafted tokens over the ring cache: the host layer, and the small
// kernels around the attention (tree_simt.cu and tree_tc.cu).
//
// A step of speculative decoding drafts up to T tokens a sequence as a tree:
// node i continues node parent[i] (or the committed tokens).  One pass gives
// every node the attention output that ordinary decoding would give it after
// the tokens on its path; the caller picks the longest path that its model
// confirms and commits that path's keys and values to the ring.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <memory>
#include <new>
#include <vector>

#include "internal.h"
#include "ptx.cuh"
#include "tree.cuh"

using namespace rswa;

// The opaque tree of the C interface.
struct rswa_tree {
  rswa_state *state;
  TreeView tv;
  int n_pieces;
  std::vector<CUtensorMap> tm_k, tm_v;  // every layer's caches (bf16)
};

namespace rswa {
namespace {

// ------------------------------------------------------------- tree masks
// One CTA per sequence, one thread per node.  Depths and the sets of nodes
// above each node come from pointer doubling: with up(i) the 2^k-th node above
// i and above(i) the set of the first 2^k, above(i) |= above(up(i)) doubles k;
// seven rounds reach 128, fewer the deepest node.  The sets below a node are the
// transpose.  Latency-bound (a few kilobytes of input).
__global__ void __launch_bounds__(RSWA_TREE_MAX)
    tree_set_kernel(const DeviceView v, const TreeView tv, const int32_t *parent,
                    const int32_t *n_draft) {
  __shared__ uint32_t above[2][RSWA_TREE_MAX][4];
  __shared__ int depth[2][RSWA_TREE_MAX], up[2][RSWA_TREE_MAX];
  const int b = blockIdx.x, i = threadIdx.x;
  const int T = tv.T;
  grid_dependency_wait();
  allow_dependents();
  int n = n_draft ? n_draft[b] : T;
  const bool bad_len = n < 0 || n > T;
  if (bad_len) n = 0;
  int pr = -1;
  if (i < n) pr = parent ? parent[(int64_t)b * T + i] : i - 1;
  const bool bad = i < n && (pr < -1 || pr >= i);
  const bool any_bad = __syncthreads_or(bad) != 0;
  if (any_bad) {
    n = 0;
    pr = -1;
  }
  if (i == 0) {
    if (bad_len) atomicOr(v.err, RSWA_DEVERR_BAD_LENGTH);
    if (any_bad) atomicOr(v.err, RSWA_DEVERR_BAD_TREE);
    tv.n[b] = n;
    tv.accepted[b] = 0;
  }
  for (int w = 0; w < 4; ++w) above[0][i][w] = w == i >> 5 ? 1u << (i & 31) : 0u;
  depth[0][i] = pr >= 0 ? 1 : 0;
  up[0][i] = pr;
  __syncthreads();
  int cur = 0;
#pragma unroll 1
  for (int k = 0; k < 7; ++k) {
    if (!__syncthreads_or(up[cur][i] >= 0)) break;  // every path has reached its top
    const int u = up[cur][i], nx = cur ^ 1;
    const bool some = u >= 0;
    for (int w = 0; w < 4; ++w) above[nx][i][w] = above[cur][i][w] | (some ? above[cur][u][w] : 0u);
    depth[nx][i] = depth[cur][i] + (some ? depth[cur][u] : 0);
    up[nx][i] = some ? up[cur][u] : -1;
    cur = nx;
    __syncthreads();
  }
  const int d = depth[cur][i];
  if (i < n && d >= v.W) {
    // the window ends below the path's first nodes
    for (int j = 0; j < i; ++j)
      if (depth[cur][j] < d - v.W + 1) above[cur][i][j >> 5] &= ~(1u << (j & 31));
  }
  __shared__ uint4 below[RSWA_TREE_MAX];
  {
    // 32 x 32 bits at a time: lane l takes column l of its warp's rows
    const int lane = i & 31;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t x = i < n ? above[cur][i][c] : 0u;
      uint32_t m = 0x0000ffffu;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const uint32_t y = __shfl_xor_sync(0xffffffffu, x, o);
        x = lane & o ? (x & ~m) | ((y >> o) & m) : (x & m) | ((y << o) & ~m);
        m ^= m << (o >> 1);
      }
      reinterpret_cast<uint32_t *>(&below[32 * c + lane])[i >> 5] = x;
    }
  }
  __syncthreads();
  if (i >= T) return;
  const int64_t row = (int64_t)b * T + i;
  tv.parent[row] = pr;
  tv.depth[row] = d;
  tv.below[row] = below[i];
  tv.above[row] = make_uint4(above[cur][i][0], above[cur][i][1], above[cur][i][2], above[cur][i][3]);
}

// ------------------------------------------------------- merge of partials
// out = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p over the pieces p of a
// ring, M = max_p m_p.  One warp per ring and row: lane p holds the (m, l) of
// piece p (32 at a time), then every lane D / 32 elements of the output, with
// eight pieces' loads in flight.  Latency-bound.
constexpr int kMergeWarps = 4;
constexpr int kMergeAhead = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kMergeWarps * 32)
    tree_combine_kernel(const DeviceView v, const TreeView tv, T *out) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t id = (int64_t)blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
  const int64_t bh = id / tv.T;
  const int i = (int)(id % tv.T);
  const bool any = bh < (int64_t)v.B * v.H;
  const int p0 = any ? tv.bh_piece[bh] : 0, p1 = any ? tv.bh_piece[bh + 1] : 0;
  grid_dependency_wait();
  allow_dependents();
  if (p1 - p0 < 2) return;  // its one piece wrote the output
  const int b = (int)(bh / v.H), h = (int)(bh % v.H);
  // one trip to memory: the count, 32 pieces' (m, l) and the first eight pieces' o
  // at once (what the partials of absent rows and unseen pieces hold is not used)
  const int n = tv.n[b];
  const float *o_row = tv.part_o + (int64_t)i * D + lane * E;
  const int64_t o_step = (int64_t)tv.T * D;
  float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int c0 = p0; c0 < p1; c0 += 32) {
    const int cnt = min(32, p1 - c0);
    float2 ml = tv.part_ml[(int64_t)(c0 + min(lane, cnt - 1)) * tv.T + i];
    float o[kMergeAhead][E];
    auto load = [&](int j0) {
#pragma unroll
      for (int u = 0; u < kMergeAhead; ++u) {
        const float *src = o_row + (c0 + min(j0 + u, cnt - 1)) * o_step;
        if constexpr (E == 4)
          *reinterpret_cast<float4 *>(o[u]) = *reinterpret_cast<const float4 *>(src);
        else
          *reinterpret_cast<float2 *>(o[u]) = *reinterpret_cast<const float2 *>(src);
      }
    };
    load(0);
    if (i >= n) return;
    if (lane >= cnt) ml = make_float2(-INFINITY, 0.f);
    // a piece in which the row saw nothing has no o; one of NaN scores has l = NaN
    const bool seen = ml.x != -INFINITY || ml.y != 0.f;
    float top = ml.x;
#pragma unroll
    for (int f = 16; f > 0; f >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, f));
    const float m_new = fmaxf(m, top);
    const float w = !seen ? 0.f : ml.x == m_new ? 1.f : exp2f(ml.x - m_new);
    float lc = seen ? w * ml.y : 0.f;
#pragma unroll
    for (int f = 16; f > 0; f >>= 1) lc += __shfl_xor_sync(0xffffffffu, lc, f);
    const float corr = m == m_new ? 1.f : exp2f(m - m_new);
    l = fmaf(l, corr, lc);
    m = m_new;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= corr;
    const uint32_t use = __ballot_sync(0xffffffffu, seen);
    for (int j0 = 0;;) {
#pragma unroll
      for (int u = 0; u < kMergeAhead; ++u) {
        const float wj = __shfl_sync(0xffffffffu, w, (j0 + u) & 31);
        if ((use >> ((j0 + u) & 31)) & 1u) {
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] = fmaf(wj, o[u][e], acc[e]);
        }
      }
      j0 += kMergeAhead;
      if (j0 >= cnt) break;
      load(j0);
    }
  }
  T *dst = out + (((int64_t)b * tv.T + i) * v.H + h) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) dst[e] = from_float<T>(acc[e] / l);
}

// ------------------------------------------------------------------ commit
// Accepted node path[i] of a sequence becomes generated token t + i: its K
// (turned at its position with RoPE) and V go to ring slot P + (t + i) mod W of
// every layer.  With more than W accepted tokens only the last W are written,
// so no slot is written twice.  A path that is not a chain down from a first
// node leaves the sequence as it was.  Moves 4 n H d elements a sequence and
// layer: bound by launch latency in ordinary use.
constexpr int kLayersPerLaunch = 64;
constexpr int kCommitThreads = 256;

struct CommitArgs {
  DeviceView v;
  TreeView tv;
  const int32_t *path, *path_len;
  int first;  // this launch holds the call's first layers
  const void *kd[kLayersPerLaunch], *vd[kLayersPerLaunch];
  void *kc[kLayersPerLaunch], *vc[kLayersPerLaunch];
};

template <typename T, int D>
__global__ void __launch_bounds__(kCommitThreads)
    tree_commit_kernel(const __grid_constant__ CommitArgs a) {
  constexpr int N = Chunk<T>::N;
  constexpr int kHalf = D / 2 / N;  // 16-byte chunks of half a row
  __shared__ int path[RSWA_TREE_MAX];
  const DeviceView &v = a.v;
  const TreeView &tv = a.tv;
  const int b = blockIdx.x, layer = blockIdx.y;
  grid_dependency_wait();
  int n = a.path_len[b];
  const int drafts = tv.n[b];
  const bool bad_len = n < 0 || n > tv.T;
  if (bad_len) n = 0;
  const int i = threadIdx.x;
  bool bad = false;
  if (i < n) {
    const int32_t *pb = a.path + (int64_t)b * tv.T;
    const int x = pb[i];
    path[i] = x;
    bad = x < 0 || x >= drafts ||
          tv.parent[(int64_t)b * tv.T + x] != (i > 0 ? pb[i - 1] : -1);
  }
  const bool any_bad = __syncthreads_or(bad) != 0;
  if (any_bad) n = 0;
  if (a.first && layer == 0 && blockIdx.z == 0 && i == 0) {
    if (bad_len) atomicOr(v.err, RSWA_DEVERR_BAD_LENGTH);
    if (any_bad) atomicOr(v.err, RSWA_DEVERR_BAD_TREE);
    tv.accepted[b] = n;
  }
  const int skip = n > v.W ? n - v.W : 0;
  const int64_t t = v.t[b];
  const int P = v.plen[b];
  const int64_t crow = (int64_t)v.H * v.slot_base[b];
  const T *kd = (const T *)a.kd[layer], *vd = (const T *)a.vd[layer];
  T *kc = (T *)a.kc[layer], *vc = (T *)a.vc[layer];
  // one item: both halves' 16-byte chunks of one head's K and V of one token
  const int per_token = v.H * kHalf;
  const int items = (n - skip) * per_token;
  for (int e = (int)blockIdx.z * kCommitThreads + i; e < items; e += (int)gridDim.z * kCommitThreads) {
    const int tok = skip + e / per_token, rem = e % per_token;
    const int h = rem / kHalf, c = rem % kHalf;
    const int64_t drow = (int64_t)b * tv.T + path[tok];
    const int64_t src = (drow * v.H + h) * D + c * N;
    const int slot = P + (int)((t + tok) % v.W);
    const int64_t dst = (crow + (int64_t)h * (P + v.W) + slot) * D + c * N;
    uint4 k0 = *reinterpret_cast<const uint4 *>(kd + src);
    uint4 k1 = *reinterpret_cast<const uint4 *>(kd + src + D / 2);
    const uint4 v0 = *reinterpret_cast<const uint4 *>(vd + src);
    const uint4 v1 = *reinterpret_cast<const uint4 *>(vd + src + D / 2);
    if (v.rope) {
      const float2 *cs = tv.cs + drow * (D / 2) + c * N;
      float x[N], y[N];
      Chunk<T>::widen(k0, x);
      Chunk<T>::widen(k1, y);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float2 r = cs[j];
        const float x0 = x[j], y0 = y[j];
        x[j] = x0 * r.x - y0 * r.y;
        y[j] = y0 * r.x + x0 * r.y;
      }
      k0 = Chunk<T>::narrow(x);
      k1 = Chunk<T>::narrow(y);
    }
    *reinterpret_cast<uint4 *>(kc + dst) = k0;
    *reinterpret_cast<uint4 *>(kc + dst + D / 2) = k1;
    *reinterpret_cast<uint4 *>(vc + dst) = v0;
    *reinterpret_cast<uint4 *>(vc + dst + D / 2) = v1;
  }
}

// -------------------------------------------------------------- host layer
bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// The tiles of all rings (each ring's draft tiles, then its cache tiles) cut
// into ranges of about equal cost, one per CTA.  Beginning and ending a piece of
// a ring costs a CTA as much as `piece_cost` tiles, so the pieces count too: the
// cut is the one with the least cost that some CTA has, found by bisection.
struct TreeCut {
  const rswa_state *s;
  int64_t draft_tiles;
  int tile, piece_cost;

  int64_t tiles(int b) const {
    return draft_tiles + (s->plen[(size_t)b] + s->cfg.window + tile - 1) / tile;
  }
  // CTAs that ranges of at most `budget` (> piece_cost) take; on_piece(b, h, t0, t1, cta).
  template <typename F>
  int64_t run(int64_t budget, F on_piece) const {
    int64_t cta = 0, left = budget;
    for (int b = 0; b < s->cfg.batch; ++b) {
      const int64_t n = tiles(b);
      for (int h = 0; h < s->cfg.num_heads; ++h)
        for (int64_t t0 = 0; t0 < n;) {
          if (left <= piece_cost) {
            ++cta;
            left = budget;
          }
          const int64_t t1 = std::min(n, t0 + left - piece_cost);
          on_piece(b, h, t0, t1, cta);
          left -= piece_cost + (t1 - t0);
          t0 = t1;
        }
    }
    return cta + 1;
  }
};

DecodePlan plan_tree(const rswa_state *s, int T, int tile, int ctas, int piece_cost) {
  const int B = s->cfg.batch, H = s->cfg.num_heads, W = s->cfg.window;
  const TreeCut cut{s, (T + tile - 1) / tile, tile, piece_cost};
  int64_t total = 0;
  for (int b = 0; b < B; ++b) total += H * (cut.tiles(b) + piece_cost);
  auto nothing = [](int, int, int64_t, int64_t, int64_t) {};
  int64_t lo = piece_cost + 1, hi = std::max(lo, total);  // hi: one CTA holds all
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (cut.run(mid, nothing) <= ctas)
      hi = mid;
    else
      lo = mid + 1;
  }
  DecodePlan p;
  p.bh_piece.reserve((size_t)B * H + 1);
  int64_t first = 0;
  cut.run(hi, [&](int b, int h, int64_t t0, int64_t t1, int64_t cta) {
    const int64_t P = s->plen[(size_t)b];
    if (t0 == 0) {
      first = (int64_t)p.pieces.size();
      p.bh_piece.push_back((int32_t)first);
    }
    while ((int64_t)p.cta_piece.size() <= cta) p.cta_piece.push_back((int32_t)p.pieces.size());
    DecodePiece pc;
    pc.row0 = (int64_t)H * s->slot_base[(size_t)b] + (int64_t)h * (P + W);
    pc.b = b;
    pc.h = h;
    pc.key_begin = (int32_t)t0;
    pc.key_end = (int32_t)t1;
    pc.plen = (int32_t)P;
    pc.first = (int32_t)first;
    pc.cta = (int32_t)cta;
    p.pieces.push_back(pc);
    if (t1 == cut.tiles(b))
      for (size_t i = (size_t)first; i < p.pieces.size(); ++i)
        p.pieces[i].count = (int32_t)(p.pieces.size() - (size_t)first);
  });
  p.n_pieces = (int)p.pieces.size();
  p.grid = (int)p.cta_piece.size();
  p.cta_piece.push_back(p.n_pieces);
  p.bh_piece.push_back(p.n_pieces);
  return p;
}

DecodePlan plan_for(const rswa_state *s, int T) {
  if (s->cfg.dtype == RSWA_BF16) {
    // the tensor-core kernel: one CTA an SM for every kTreeTcRows drafts
    const int cols = (T + kTreeTcRows - 1) / kTreeTcRows;
    return plan_tree(s, T, kTreeTcTile, std::max(1, s->num_sms / cols), kTreeTcPieceCost);
  }
  return plan_tree(s, T, kTreeSimtTile,
                   std::max(1, tree_simt_ctas(s->num_sms, s->cfg.head_dim, T)), kTreeSimtPieceCost);
}

struct TreeLayout {
  size_t pieces, cta_piece, bh_piece, uploaded, n, accepted, parent, depth, above, below, cs,
      part_ml, part_o, total;
};

TreeLayout layout_tree(const rswa_state *s, int T, const DecodePlan &p) {
  const size_t rows = (size_t)s->cfg.batch * (size_t)T, d = (size_t)s->cfg.head_dim;
  TreeLayout w;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  w.pieces = take(p.pieces.size() * sizeof(DecodePiece));
  w.cta_piece = take(p.cta_piece.size() * sizeof(int32_t));
  w.bh_piece = take(p.bh_piece.size() * sizeof(int32_t));
  // drafts in use and accepted tokens: zero until rswa_tree_set
  w.n = take((size_t)s->cfg.batch * sizeof(int32_t));
  w.accepted = take((size_t)s->cfg.batch * sizeof(int32_t));
  w.uploaded = off;
  w.parent = take(rows * sizeof(int32_t));
  w.depth = take(rows * sizeof(int32_t));
  w.above = take(rows * sizeof(uint4));
  w.below = take(rows * sizeof(uint4));
  w.cs = take(rows * (d / 2) * sizeof(float2));
  w.part_ml = take((size_t)p.n_pieces * (size_t)T * sizeof(float2));
  w.part_o = take((size_t)p.n_pieces * (size_t)T * d * sizeof(float));
  w.total = off;
  return w;
}

bool tree_args_ok(const rswa_state *s, int32_t max_draft) {
  return s && max_draft >= 1 && max_draft <= RSWA_TREE_MAX &&
         (int64_t)s->cfg.batch * max_draft < (int64_t(1) << 31);
}

}  // namespace

cudaError_t launch_tree_set(const DeviceView &v, const TreeView &tv, const int32_t *parent,
                            const int32_t *n_draft, cudaStream_t s) {
  cudaError_t e = launch_overlapped(tree_set_kernel, dim3((unsigned)v.B), dim3(RSWA_TREE_MAX), 0, s,
                                    v, tv, parent, n_draft);
  return e != cudaSuccess ? e : launch_tree_rope(v, tv, s);
}

template <typename T, int D>
static cudaError_t combine_t(const DeviceView &v, const TreeView &tv, void *out, cudaStream_t s) {
  const int64_t rows = (int64_t)v.B * v.H * tv.T;
  return launch_overlapped(tree_combine_kernel<T, D>,
                           dim3((unsigned)((rows + kMergeWarps - 1) / kMergeWarps)),
                           dim3(kMergeWarps * 32), 0, s, v, tv, (T *)out);
}

cudaError_t launch_tree_combine(const DeviceView &v, const TreeView &tv, void *out,
                                cudaStream_t s) {
  if (v.dtype == RSWA_BF16)
    return v.D == 128 ? combine_t<__nv_bfloat16, 128>(v, tv, out, s)
                      : combine_t<__nv_bfloat16, 64>(v, tv, out, s);
  return v.D == 128 ? combine_t<float, 128>(v, tv, out, s) : combine_t<float, 64>(v, tv, out, s);
}

}  // namespace rswa

extern "C" {

size_t rswa_tree_workspace_bytes(const rswa_state *state, int32_t max_draft) {
  if (!tree_args_ok(state, max_draft) || current_device() != state->device) return 0;
  try {
    return layout_tree(state, max_draft, plan_for(state, max_draft)).total;
  } catch (const std::exception &) {
    return 0;
  }
}

rswa_status rswa_tree_create(rswa_state *state, int32_t max_draft, void *workspace,
                             size_t workspace_size, void *stream, rswa_tree **out) {
  if (!out) return RSWA_EINVAL;
  *out = nullptr;
  if (!tree_args_ok(state, max_draft) || !workspace || ((uintptr_t)workspace & 255u) != 0)
    return RSWA_EINVAL;
  if (current_device() != state->device) return RSWA_EINVAL;
  try {
    const DecodePlan p = plan_for(state, max_draft);
    const TreeLayout w = layout_tree(state, max_draft, p);
    if (workspace_size < w.total) return RSWA_ENOMEM;
    std::vector<uint8_t> img(w.uploaded, 0);
    std::copy_n((const uint8_t *)p.pieces.data(), p.pieces.size() * sizeof(DecodePiece),
                img.data() + w.pieces);
    std::copy_n((const uint8_t *)p.cta_piece.data(), p.cta_piece.size() * sizeof(int32_t),
                img.data() + w.cta_piece);
    std::copy_n((const uint8_t *)p.bh_piece.data(), p.bh_piece.size() * sizeof(int32_t),
                img.data() + w.bh_piece);
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = cudaMemcpyAsync(workspace, img.data(), img.size(), cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return from_cuda(e);
    std::unique_ptr<rswa_tree> t(new rswa_tree());
    if (state->cfg.dtype == RSWA_BF16) {
      const size_t L = (size_t)state->cfg.num_layers;
      t->tm_k.resize(L);
      t->tm_v.resize(L);
      for (size_t l = 0; l < L; ++l)
        if (!tree_tc_maps(state->dv, state->k_cache[l], state->v_cache[l],
                          (int64_t)state->cfg.num_heads * state->pool_slots, &t->tm_k[l],
                          &t->tm_v[l]))
          return RSWA_EINVAL;
    }
    uint8_t *base = (uint8_t *)workspace;
    t->state = state;
    t->n_pieces = p.n_pieces;
    TreeView &tv = t->tv;
    tv.T = max_draft;
    tv.grid = p.grid;
    tv.pieces = (const DecodePiece *)(base + w.pieces);
    tv.cta_piece = (const int32_t *)(base + w.cta_piece);
    tv.bh_piece = (const int32_t *)(base + w.bh_piece);
    tv.part_ml = (float2 *)(base + w.part_ml);
    tv.part_o = (float *)(base + w.part_o);
    tv.parent = (int32_t *)(base + w.parent);
    tv.depth = (int32_t *)(base + w.depth);
    tv.above = (uint4 *)(base + w.above);
    tv.below = (uint4 *)(base + w.below);
    tv.n = (int32_t *)(base + w.n);
    tv.accepted = (int32_t *)(base + w.accepted);
    tv.cs = (float2 *)(base + w.cs);
    *out = t.release();
    return RSWA_OK;
  } catch (const std::exception &) {
    return RSWA_ENOMEM;
  }
}

rswa_status rswa_tree_destroy(rswa_tree *tree) {
  if (!tree) return RSWA_EINVAL;
  delete tree;
  return RSWA_OK;
}

rswa_status rswa_tree_set(rswa_tree *tree, const int32_t *parent, const int32_t *n_draft,
                          void *stream) {
  if (!tree || current_device() != tree->state->device) return RSWA_EINVAL;
  return from_cuda(launch_tree_set(tree->state->dv, tree->tv, parent, n_draft, (cudaStream_t)stream));
}

rswa_status rswa_tree_attention(rswa_tree *tree, int32_t layer, const void *q, const void *k_draft,
                                const void *v_draft, void *out, void *stream) {
  if (!tree) return RSWA_EINVAL;
  const rswa_state *s = tree->state;
  if (layer < 0 || layer >= s->cfg.num_layers) return RSWA_EINVAL;
  if (!q || !k_draft || !v_draft || !out) return RSWA_EINVAL;
  if (out == q || out == k_draft || out == v_draft) return RSWA_EINVAL;
  if (!aligned16(q) || !aligned16(k_draft) || !aligned16(v_draft) || !aligned16(out))
    return RSWA_EINVAL;
  if (!s->layer_ready[(size_t)layer]) return RSWA_ESTATE;
  if (current_device() != s->device) return RSWA_EINVAL;
  const cudaStream_t st = (cudaStream_t)stream;
  const size_t l = (size_t)layer;
  cudaError_t e =
      s->cfg.dtype == RSWA_BF16
          ? launch_tree_tc(s->dv, tree->tv, tree->tm_k[l], tree->tm_v[l], q, k_draft, v_draft,
                           s->v_cache[l], out, st)
          : launch_tree_simt(s->dv, tree->tv, (const float *)q, (const float *)k_draft,
                             (const float *)v_draft, (const float *)s->k_cache[l],
                             (const float *)s->v_cache[l], (float *)out, st);
  if (e == cudaSuccess && tree->n_pieces > s->cfg.batch * s->cfg.num_heads)
    e = launch_tree_combine(s->dv, tree->tv, out, st);
  return from_cuda(e);
}

rswa_status rswa_tree_commit(rswa_tree *tree, const void *const *k_draft,
                             const void *const *v_draft, const int32_t *path,
                             const int32_t *path_len, void *stream) {
  if (!tree || !k_draft || !v_draft || !path || !path_len) return RSWA_EINVAL;
  const rswa_state *s = tree->state;
  const int L = s->cfg.num_layers;
  for (int l = 0; l < L; ++l)
    if (!k_draft[l] || !v_draft[l] || !aligned16(k_draft[l]) || !aligned16(v_draft[l]))
      return RSWA_EINVAL;
  for (int l = 0; l < L; ++l)
    if (!s->layer_ready[(size_t)l]) return RSWA_ESTATE;
  if (current_device() != s->device) return RSWA_EINVAL;
  // blocks along a sequence's tokens until a launch fills the SMs about once
  const int64_t chunks = (int64_t)tree->tv.T * s->cfg.num_heads * s->cfg.head_dim *
                         (s->cfg.dtype == RSWA_BF16 ? 2 : 4) / 32;
  for (int l0 = 0; l0 < L; l0 += kLayersPerLaunch) {
    CommitArgs a;
    a.v = s->dv;
    a.tv = tree->tv;
    a.path = path;
    a.path_len = path_len;
    a.first = l0 == 0;
    const int n = std::min(kLayersPerLaunch, L - l0);
    for (int l = 0; l < n; ++l) {
      a.kd[l] = k_draft[l0 + l];
      a.vd[l] = v_draft[l0 + l];
      a.kc[l] = s->k_cache[(size_t)(l0 + l)];
      a.vc[l] = s->v_cache[(size_t)(l0 + l)];
    }
    const int64_t blocks = (int64_t)s->cfg.batch * n;
    const int64_t z = std::min((chunks + kCommitThreads - 1) / kCommitThreads,
                               std::max<int64_t>(1, 4 * s->num_sms / blocks));
    const dim3 grid((unsigned)s->cfg.batch, (unsigned)n, (unsigned)z);
    auto *commit = s->cfg.dtype == RSWA_BF16
                       ? (s->cfg.head_dim == 128 ? tree_commit_kernel<__nv_bfloat16, 128>
                                                 : tree_commit_kernel<__nv_bfloat16, 64>)
                       : (s->cfg.head_dim == 128 ? tree_commit_kernel<float, 128>
                                                 : tree_commit_kernel<float, 64>);
    const cudaError_t e =
        launch_overlapped(commit, grid, dim3(kCommitThreads), 0, (cudaStream_t)stream, a);
    if (e != cudaSuccess) return from_cuda(e);
  }
  return RSWA_OK;
}

rswa_status rswa_tree_advance(rswa_tree *tree, void *stream) {
  if (!tree || current_device() != tree->state->device) return RSWA_EINVAL;
  return from_cuda(
      launch_tree_advance(tree->state->dv, tree->tv.accepted, (cudaStream_t)stream));
}

}  // extern "C"
