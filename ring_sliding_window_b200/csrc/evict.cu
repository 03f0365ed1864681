// Scored decode steps and the eviction of prompt entries by accumulated
// attention weight.
//
// A scored step computes the ordinary decode attention and adds each entry's
// softmax weight p_j = 2^(s_j - m) / l to that entry's score.  The decode
// kernel leaves the raw scores s (4 bytes an entry, next to the 512 or 1,024
// bytes of K and V it streams) and (m, l) per ring; score_finish_kernel turns
// them into weights.  An eviction keeps, per ring, the P' prompt entries with
// the highest scores and moves them with the ring into a smaller cache.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <utility>
#include <vector>

#include "internal.h"
#include "ptx.cuh"
#include "tree.cuh"

using namespace rswa;

namespace rswa {
namespace {

// ------------------------------------------------------- accumulated weight
constexpr int kFinishThreads = 256;
constexpr int kFinishPer = 8;  // entries of a thread

__global__ void __launch_bounds__(kFinishThreads)
    score_finish_kernel(const DeviceView v, const float *__restrict__ raw, const float *score_in,
                        float *score_out, int chunks) {
  const int bh = (int)(blockIdx.x / (unsigned)chunks);
  const int b = bh / v.H, h = bh % v.H;
  const int P = v.plen[b];
  const int64_t t = v.t[b];
  const int held = P + (int)(t + 1 < v.W ? t + 1 : (int64_t)v.W);
  const int fresh = P + (int)(t % v.W);  // the step's own entry: its score starts over
  const int64_t lo64 = (int64_t)P + t - v.W + 1;  // standard mode: the window cuts the prompt
  const int lo = !v.swa || lo64 < 0 ? 0 : (lo64 > P ? P : (int)lo64);
  const int64_t row0 = (int64_t)v.H * v.slot_base[b] + (int64_t)h * (P + v.W);
  const float2 ml = v.ring_ml[bh];
  const float inv = 1.f / ml.y;
  const int s0 = (int)(blockIdx.x % (unsigned)chunks) * (kFinishThreads * kFinishPer) + threadIdx.x;
  float x[kFinishPer], y[kFinishPer];
#pragma unroll
  for (int j = 0; j < kFinishPer; ++j) {
    const int s = s0 + j * kFinishThreads;
    x[j] = s >= lo && s < held ? raw[row0 + s] : -INFINITY;
    y[j] = s < held && s != fresh ? score_in[row0 + s] : 0.f;
  }
#pragma unroll
  for (int j = 0; j < kFinishPer; ++j) {
    const int s = s0 + j * kFinishThreads;
    if (s < held) score_out[row0 + s] = s >= lo ? fmaf(exp2f(x[j] - ml.x), inv, y[j]) : y[j];
  }
}

// ------------------------------------------------------------- selection
// The K prompt entries with the highest scores of one ring: a radix select
// over order-preserving 32-bit keys, 8 bits a pass, by a cluster of CTAs that
// add their histograms through distributed shared memory; then every CTA lists
// its kept entries in ascending order at its offset of the ring's list.  Reads
// 4 bytes an entry five times, four of them from L2; latency-bound (about a
// dozen cluster barriers).
constexpr int kSelCtas = 8;
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;

struct SelectArgs {
  DeviceView src, dst;
  const float *score;
  int n_first, n_last;
  int32_t *kept;
};

// Larger key = kept first.  NaN ranks below everything, -0 with +0; a
// protected entry above everything.
__device__ __forceinline__ uint32_t score_key(float x, bool guarded) {
  if (guarded) return 0xffffffffu;
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __cluster_dims__(kSelCtas, 1, 1) __launch_bounds__(kSelThreads)
    evict_select_kernel(const SelectArgs a) {
  __shared__ uint32_t hist[2][256];
  __shared__ uint32_t pick[2];      // bin of the threshold, entries above it
  __shared__ uint32_t totals[2];    // this CTA's entries above / at the threshold
  __shared__ uint32_t warp_gt[kSelWarps], warp_eq[kSelWarps];
  const int ring = (int)(blockIdx.x / kSelCtas), rank = (int)(blockIdx.x % kSelCtas);
  const int b = ring / a.src.H, h = ring % a.src.H;
  const int P = a.src.plen[b], K = a.dst.plen[b];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (K == 0) return;  // the whole cluster
  const int64_t row0 = (int64_t)a.src.H * a.src.slot_base[b] + (int64_t)h * (P + a.src.W);
  const float *score = a.score + row0;
  const int seg = (P + kSelCtas - 1) / kSelCtas;
  const int s0 = min(P, rank * seg), s1 = min(P, s0 + seg);
  auto key_at = [&](int s) {
    return score_key(score[s], s < a.n_first || s >= P - a.n_last);
  };

  uint32_t prefix = 0;       // the threshold's leading bits so far
  uint32_t left = (uint32_t)K;  // entries still to take among keys with that prefix
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    uint32_t *hs = hist[pass & 1];
    for (int i = tid; i < 256; i += kSelThreads) hs[i] = 0;
    __syncthreads();
    for (int s = s0 + tid; s < s0 + (s1 - s0 + 31) / 32 * 32; s += kSelThreads) {
      uint32_t bin = 256;  // none
      if (s < s1) {
        const uint32_t k = key_at(s);
        if (pass == 0 || (k >> (shift + 8)) == prefix) bin = (k >> shift) & 255u;
      }
      // many entries share a bin (ties at zero, one exponent): the warp's first
      // lane adds for all lanes with its bin, the others one by one
      const uint32_t bin0 = __shfl_sync(0xffffffffu, bin, 0);
      const uint32_t same = __ballot_sync(0xffffffffu, bin == bin0);
      if (lane == 0) {
        if (bin0 < 256) atomicAdd(&hs[bin0], (uint32_t)__popc(same));
      } else if (bin != bin0 && bin < 256) {
        atomicAdd(&hs[bin], 1u);
      }
    }
    cluster_arrive_release();
    cluster_wait_acquire();
    // bins from the highest down: thread i holds bin 255 - i of the whole ring
    uint32_t mine = 0, run = 0;
    if (tid < 256) {
      for (int r = 0; r < kSelCtas; ++r) mine += ld_cluster_u32(map_to_rank(&hs[255 - tid], r));
      run = mine;
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += up;
      }
      if (lane == 31) warp_gt[warp] = run;
    }
    __syncthreads();
    if (tid < 256) {
      for (int w = 0; w < warp; ++w) run += warp_gt[w];
      if (run >= left && run - mine < left) {
        pick[0] = 255u - (uint32_t)tid;
        pick[1] = run - mine;
      }
    }
    __syncthreads();
    prefix = (prefix << 8) | pick[0];
    left -= pick[1];
    __syncthreads();  // pick and warp_gt are read
  }
  // kept: every key above `prefix`, and the first `left` of those equal to it
  if (tid < 2) totals[tid] = 0;
  __syncthreads();
  {
    uint32_t gt = 0, eq = 0;
    for (int s = s0 + tid; s < s1; s += kSelThreads) {
      const uint32_t k = key_at(s);
      gt += k > prefix;
      eq += k == prefix;
    }
    for (int o = 16; o > 0; o >>= 1) {
      gt += __shfl_xor_sync(0xffffffffu, gt, o);
      eq += __shfl_xor_sync(0xffffffffu, eq, o);
    }
    if (lane == 0) {
      atomicAdd(&totals[0], gt);
      atomicAdd(&totals[1], eq);
    }
  }
  cluster_arrive_release();
  cluster_wait_acquire();
  uint32_t n_gt = 0, n_eq = 0;  // in the segments before the current 512 entries
  for (int r = 0; r < rank; ++r) {
    n_gt += ld_cluster_u32(map_to_rank(&totals[0], r));
    n_eq += ld_cluster_u32(map_to_rank(&totals[1], r));
  }
  int64_t list0 = 0;  // this ring's list: H sum_{b' < b} P'_b' + h P'_b
  list0 = (int64_t)a.src.H * a.dst.tok_base[b] + (int64_t)h * K;
  for (int base = s0; base < s1; base += kSelThreads) {
    const int s = base + tid;
    const uint32_t k = s < s1 ? key_at(s) : 0u;
    const bool gt = s < s1 && k > prefix, eq = s < s1 && k == prefix;
    const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) {
      warp_gt[warp] = (uint32_t)__popc(bg);
      warp_eq[warp] = (uint32_t)__popc(be);
    }
    __syncthreads();
    uint32_t g = n_gt, e = n_eq;
    for (int w = 0; w < kSelWarps; ++w) {
      if (w < warp) {
        g += warp_gt[w];
        e += warp_eq[w];
      }
      n_gt += warp_gt[w];
      n_eq += warp_eq[w];
    }
    const uint32_t below = (1u << lane) - 1u;
    g += (uint32_t)__popc(bg & below);
    e += (uint32_t)__popc(be & below);
    if (gt || (eq && e < left)) a.kept[list0 + g + (e < left ? e : left)] = s;
    __syncthreads();
  }
  // no CTA leaves while another may still read its shared memory
  cluster_arrive_release();
  cluster_wait_acquire();
}

// ------------------------------------------------------------------ move
// Destination slot j of a ring takes prompt entry kept[j] while j < P', then
// the ring's held slots; with its score.  One warp moves kMoveRows slots, every
// load of them in flight together.  Bound by HBM bandwidth: 4 d elements read
// and written a slot.
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 4;

struct MoveArgs {
  DeviceView src, dst;
  const uint8_t *kc, *vc;
  uint8_t *kc2, *vc2;
  const float *score;
  float *score2;
  const int32_t *kept;
  int groups;  // CTAs of a ring
};

template <int kRowBytes>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const MoveArgs a) {
  constexpr int kChunks = kRowBytes / 16;
  constexpr int kPerRow = 2 * kChunks;                      // 16-byte chunks of a slot's K and V
  constexpr int kIters = (kMoveRows * kPerRow + 31) / 32;   // loads of a lane
  const int ring = (int)(blockIdx.x / (unsigned)a.groups);
  const int b = ring / a.src.H, h = ring % a.src.H;
  const int P = a.src.plen[b], K = a.dst.plen[b], W = a.src.W;
  const int64_t t = a.src.t[b];
  const int n = K + (int)(t < W ? t : (int64_t)W);
  const int64_t src0 = (int64_t)a.src.H * a.src.slot_base[b] + (int64_t)h * (P + W);
  const int64_t dst0 = (int64_t)a.src.H * a.dst.slot_base[b] + (int64_t)h * (K + W);
  const int64_t list0 = (int64_t)a.src.H * a.dst.tok_base[b] + (int64_t)h * K;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j0 = ((int)(blockIdx.x % (unsigned)a.groups) * (kMoveThreads / 32) + warp) * kMoveRows;
  if (blockIdx.x % (unsigned)a.groups == 0 && h == 0 && threadIdx.x == 0) {
    // the counters go with the entries, and so does the length positions count from
    a.dst.t[b] = t;
    a.dst.t[a.src.B + b] = t;
    a.dst.pos_base[b] = a.src.pos_base[b];
  }
  if (j0 >= n) return;
  int from = 0;  // lane r < kMoveRows: the source slot of destination slot j0 + r
  if (lane < kMoveRows && j0 + lane < n) {
    const int j = j0 + lane;
    from = j < K ? a.kept[list0 + j] : P + (j - K);
    if (a.score2) a.score2[dst0 + j] = a.score[src0 + from];
  }
  uint4 u[kIters];
#pragma unroll
  for (int i = 0; i < kIters; ++i) {
    const int e = i * 32 + lane, r = e / kPerRow, c = e % kPerRow;
    const int s = __shfl_sync(0xffffffffu, from, r < kMoveRows ? r : 0);
    if (r < kMoveRows && j0 + r < n)
      u[i] = *reinterpret_cast<const uint4 *>((c < kChunks ? a.kc : a.vc) +
                                              (src0 + s) * kRowBytes + (c % kChunks) * 16);
  }
#pragma unroll
  for (int i = 0; i < kIters; ++i) {
    const int e = i * 32 + lane, r = e / kPerRow, c = e % kPerRow;
    if (r < kMoveRows && j0 + r < n)
      *reinterpret_cast<uint4 *>((c < kChunks ? a.kc2 : a.vc2) + (dst0 + j0 + r) * kRowBytes +
                                 (c % kChunks) * 16) = u[i];
  }
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// Bytes [first, last) of every request's range in one cache buffer.
void request_ranges(const rswa_state *s, const void *cache, size_t row_bytes,
                    std::vector<std::pair<uintptr_t, uintptr_t>> &out) {
  for (int b = 0; b < s->cfg.batch; ++b) {
    const uintptr_t lo = (uintptr_t)cache +
                         (size_t)s->cfg.num_heads * (size_t)s->slot_base[(size_t)b] * row_bytes;
    out.emplace_back(lo, lo + (size_t)s->cfg.num_heads *
                                  (size_t)(s->plen[(size_t)b] + s->cfg.window) * row_bytes);
  }
}

// Whether any request's entries of `a` share memory with any of `b`'s.
bool share_memory(const std::vector<std::pair<uintptr_t, uintptr_t>> &a,
                  const std::vector<std::pair<uintptr_t, uintptr_t>> &b) {
  std::vector<std::pair<uintptr_t, uintptr_t>> x(a), y(b);
  std::sort(x.begin(), x.end());
  std::sort(y.begin(), y.end());
  size_t j = 0;
  for (const auto &r : x) {
    while (j < y.size() && y[j].second <= r.first) ++j;
    if (j < y.size() && y[j].first < r.second) return true;
  }
  return false;
}

}  // namespace

cudaError_t launch_score_finish(const DeviceView &v, const float *raw, const float *score_in,
                                float *score_out, cudaStream_t s) {
  const int chunks = (v.max_plen + v.W + kFinishThreads * kFinishPer - 1) / (kFinishThreads * kFinishPer);
  score_finish_kernel<<<(unsigned)(v.B * v.H) * (unsigned)chunks, kFinishThreads, 0, s>>>(
      v, raw, score_in, score_out, chunks);
  return cudaGetLastError();
}

}  // namespace rswa

extern "C" {

size_t rswa_score_bytes(const rswa_state *s) {
  if (!s) return 0;
  return (size_t)s->pool_slots * (size_t)s->cfg.num_heads * sizeof(float);
}

rswa_status rswa_decode_step_scored(rswa_state *s, int32_t layer, const void *q, const void *k_new,
                                    const void *v_new, void *out, const float *score_in,
                                    float *score_out, float *scratch, void *stream) {
  if (!s || layer < 0 || layer >= s->cfg.num_layers) return RSWA_EINVAL;
  if (!q || !k_new || !v_new || !out || !score_in || !score_out || !scratch) return RSWA_EINVAL;
  if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(out) ||
      !aligned16(score_in) || !aligned16(score_out) || !aligned16(scratch))
    return RSWA_EINVAL;
  if (scratch == score_in || scratch == score_out) return RSWA_EINVAL;
  if (!s->layer_ready[(size_t)layer]) return RSWA_ESTATE;
  if (current_device() != s->device) return RSWA_EINVAL;
  const cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = launch_decode(s->dv, q, k_new, v_new, s->k_cache[(size_t)layer],
                                s->v_cache[(size_t)layer], out, st, true, scratch);
  if (e == cudaSuccess) e = launch_score_finish(s->dv, scratch, score_in, score_out, st);
  return from_cuda(e);
}

rswa_status rswa_evict(const rswa_state *src, rswa_state *dst, int32_t layer, const float *score,
                       int32_t n_first, int32_t n_last, float *dst_score, int32_t *kept,
                       void *stream) {
  if (!src || !dst || src == dst || layer < 0 || layer >= src->cfg.num_layers) return RSWA_EINVAL;
  const rswa_config &a = src->cfg, &c = dst->cfg;
  if (a.batch != c.batch || a.num_layers != c.num_layers || a.num_heads != c.num_heads ||
      a.head_dim != c.head_dim || a.window != c.window || a.dtype != c.dtype)
    return RSWA_EINVAL;
  if (!score || !kept || !aligned16(score) || !aligned16(kept) ||
      (dst_score && !aligned16(dst_score)))
    return RSWA_EINVAL;
  if (n_first < 0 || n_last < 0) return RSWA_EINVAL;
  if (src->dv.swa || dst->dv.swa) return RSWA_EINVAL;
  for (int b = 0; b < a.batch; ++b) {
    const int64_t P = src->plen[(size_t)b], K = dst->plen[(size_t)b];
    if (K > P || std::min<int64_t>((int64_t)n_first + n_last, P) > K) return RSWA_EINVAL;
  }
  if (!src->layer_ready[(size_t)layer]) return RSWA_ESTATE;
  const int dev = current_device();
  if (dev != src->device || dev != dst->device) return RSWA_EINVAL;
  const size_t l = (size_t)layer;
  const size_t row_bytes = (size_t)a.head_dim * (a.dtype == RSWA_BF16 ? 2 : 4);
  try {
    std::vector<std::pair<uintptr_t, uintptr_t>> from, to;
    request_ranges(src, src->k_cache[l], row_bytes, from);
    request_ranges(src, src->v_cache[l], row_bytes, from);
    request_ranges(dst, dst->k_cache[l], row_bytes, to);
    request_ranges(dst, dst->v_cache[l], row_bytes, to);
    if (share_memory(from, to)) return RSWA_EINVAL;
    from.clear();
    to.clear();
    if (dst_score) {
      request_ranges(src, score, sizeof(float), from);
      request_ranges(dst, dst_score, sizeof(float), to);
      if (share_memory(from, to)) return RSWA_EINVAL;
    }
  } catch (const std::exception &) {
    return RSWA_ENOMEM;
  }
  const cudaStream_t st = (cudaStream_t)stream;
  const unsigned rings = (unsigned)(a.batch * a.num_heads);
  const SelectArgs sel{src->dv, dst->dv, score, n_first, n_last, kept};
  evict_select_kernel<<<rings * kSelCtas, kSelThreads, 0, st>>>(sel);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return from_cuda(e);
  MoveArgs mv;
  mv.src = src->dv;
  mv.dst = dst->dv;
  mv.kc = (const uint8_t *)src->k_cache[l];
  mv.vc = (const uint8_t *)src->v_cache[l];
  mv.kc2 = (uint8_t *)dst->k_cache[l];
  mv.vc2 = (uint8_t *)dst->v_cache[l];
  mv.score = score;
  mv.score2 = dst_score;
  mv.kept = kept;
  constexpr int kPerCta = kMoveThreads / 32 * kMoveRows;
  mv.groups = (dst->dv.max_plen + a.window + kPerCta - 1) / kPerCta;
  const unsigned grid = rings * (unsigned)mv.groups;
  if (row_bytes == 128)
    evict_move_kernel<128><<<grid, kMoveThreads, 0, st>>>(mv);
  else if (row_bytes == 256)
    evict_move_kernel<256><<<grid, kMoveThreads, 0, st>>>(mv);
  else
    evict_move_kernel<512><<<grid, kMoveThreads, 0, st>>>(mv);
  e = cudaGetLastError();
  if (e != cudaSuccess) return from_cuda(e);
  dst->dv.rope = src->dv.rope;
  dst->dv.rope_theta = src->dv.rope_theta;
  e = launch_rope_table(dst->dv, st);
  if (e != cudaSuccess) return from_cuda(e);
  dst->layer_ready[l] = 1;
  return RSWA_OK;
}

}  // extern "C"
