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
  // No early start for the kernel after this one: the next layer's decode step
  // would be placed around these CTAs' registers, unevenly (154 us for 122).
  grid_dependency_wait();
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
// The K prompt entries with the highest scores of one ring, by one CTA: a radix
// select over order-preserving 32-bit keys (11, 11 and 10 bits a pass) finds the
// K-th largest key and how many of its equals belong in; then the kept entries
// are listed in ascending order.  Scores are read once, the keys stay in shared
// memory (beyond kSelCache entries they are read again, from L2), and every loop
// after the first takes four a thread.
//
// Takes 19 us for 40 rings of 32,640 entries, on 40 SMs (8.0 until the first
// counts, 9.5 in the four loops after that), and 9 us for 80 of 8,256; short
// rings pay the latency of seven short phases.  The launch bound holds the kernel
// to 32 registers, with spills of 12 bytes stored and 24 loaded; whether more
// registers would help has not been measured.  Clusters of 2 and 4 CTAs a ring, adding
// their counts through distributed shared memory, cost 10 us more: their barriers
// and remote loads take longer than the loops that they share.
constexpr int kSelMaxThreads = 1024;
constexpr int kSelBins = 2048;
constexpr int kSelCache = 49152;  // 192 KB
constexpr int kSelAhead = 8;      // scores of a thread in flight

struct SelectArgs {
  DeviceView src, dst;
  const float *score;
  int n_first, n_last;
  int32_t *kept;
  int cache;  // keys that the launch's shared memory holds, a multiple of 4
};

// Larger key = kept first.  NaN ranks below everything, -0 with +0; a
// protected entry above everything.
__device__ __forceinline__ uint32_t score_key(float x, bool guarded) {
  if (guarded) return 0xffffffffu;
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
constexpr uint32_t kZeroKey = 0x80000000u;

__global__ void __launch_bounds__(kSelMaxThreads)
    evict_select_kernel(const SelectArgs a) {
  extern __shared__ uint4 sel_smem[];  // [kSelBins] counts, then [a.cache] keys
  __shared__ uint32_t warp_a[32], warp_b[32];
  __shared__ uint32_t pick[3];  // bin of the threshold, entries above it, entries in it
  uint32_t *hist = reinterpret_cast<uint32_t *>(sel_smem), *keys = hist + kSelBins;
  const int ring = (int)blockIdx.x;
  const int b = ring / a.src.H, h = ring % a.src.H;
  const int P = a.src.plen[b], K = a.dst.plen[b];
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = nt >> 5;
  const int64_t row0 = (int64_t)a.src.H * a.src.slot_base[b] + (int64_t)h * (P + a.src.W);
  const int64_t list0 = (int64_t)a.src.H * a.dst.tok_base[b] + (int64_t)h * K;
  const float *score = a.score + row0;
  grid_dependency_wait();
  allow_dependents();
  if (K == 0) return;
  if (K == P) {
    for (int s = tid; s < P; s += nt) a.kept[list0 + s] = s;
    return;
  }
  auto to_key = [&](float x, int s) {
    return score_key(x, s < a.n_first || s >= P - a.n_last);
  };
  // keys of entries 4 i .. 4 i + 3 (behind the last entry: anything)
  const int quads = (P + 3) / 4;
  auto key4 = [&](int i) {
    if (4 * i < a.cache) return *reinterpret_cast<const uint4 *>(keys + 4 * i);
    uint32_t k[4];
#pragma unroll
    for (int c = 0; c < 4; ++c)
      k[c] = 4 * i + c < P ? to_key(score[4 * i + c], 4 * i + c) : 0u;
    return make_uint4(k[0], k[1], k[2], k[3]);
  };

  uint32_t prefix = 0;           // the threshold's leading bits so far
  uint32_t left = (uint32_t)K;   // entries still to take among keys with that prefix
  int shift = 32;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass < 2 ? 11 : 10;
    const uint32_t bins = 1u << bits;
    const int above = shift;     // bits of a key above this pass's lie at this shift
    shift -= bits;
    for (int i = tid; i < (int)bins; i += nt) hist[i] = 0;
    __syncthreads();
    // exact zeros are many and share a bin: counted by the thread
    uint32_t zeros = 0;
    auto count = [&](uint32_t k, bool in) {
      const bool zero = k == kZeroKey;
      zeros += in && zero ? 1u : 0u;
      if (in && !zero) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1u);
    };
    if (pass == 0) {
      for (int s0 = tid; s0 < P; s0 += kSelAhead * nt) {
        float x[kSelAhead];
#pragma unroll
        for (int u = 0; u < kSelAhead; ++u) x[u] = s0 + u * nt < P ? score[s0 + u * nt] : 0.f;
#pragma unroll
        for (int u = 0; u < kSelAhead; ++u) {
          const int s = s0 + u * nt;
          const uint32_t k = to_key(x[u], s);
          if (s < min(P, a.cache)) keys[s] = k;
          count(k, s < P);
        }
      }
    } else {
#pragma unroll 4
      for (int i = tid; i < quads; i += nt) {
        const uint4 q = key4(i);
        const uint32_t k[4] = {q.x, q.y, q.z, q.w};
        bool in[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) in[c] = (k[c] >> above) == prefix && 4 * i + c < P;
        if (in[0] || in[1] || in[2] || in[3])
#pragma unroll
          for (int c = 0; c < 4; ++c) count(k[c], in[c]);
      }
    }
    __syncwarp();
    zeros = __reduce_add_sync(0xffffffffu, zeros);
    if (lane == 0 && zeros) atomicAdd(&hist[(kZeroKey >> shift) & (bins - 1)], zeros);
    __syncthreads();
    // bins from the highest down, bins / nt of them a thread
    const int per = (int)bins / nt;
    const int top = (int)bins - 1 - tid * per;
    uint32_t mine = 0;
    for (int i = 0; i < per; ++i) mine += hist[top - i];
    uint32_t run = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += up;
    }
    if (lane == 31) warp_a[warp] = run;
    __syncthreads();
    run += __reduce_add_sync(0xffffffffu, lane < warp ? warp_a[lane] : 0u);
    uint32_t before = run - mine;
    if (before < left && run >= left) {
      int i = 0;
      for (; before + hist[top - i] < left; ++i) before += hist[top - i];
      pick[0] = (uint32_t)(top - i);
      pick[1] = before;
      pick[2] = hist[top - i];
    }
    __syncthreads();
    prefix = (prefix << bits) | pick[0];
    left -= pick[1];
    if (pick[2] == left) {  // the whole bin is kept: no need to look further into it
      left = 0xffffffffu;
      break;
    }
  }
  // kept: every key above the threshold, and the first `left` of those equal to
  // it; a warp takes a stretch of the ring, a lane four neighbours of every 128
  const uint32_t thr = prefix << shift;
  const int span = ((quads + 31) / 32 + warps - 1) / warps * 32;  // quads of a warp
  const int i0 = warp * span, i1 = min((quads + 31) / 32 * 32, i0 + span);
  uint32_t gt = 0, eq = 0;
#pragma unroll 4
  for (int i = i0 + lane; i < min(i1, quads); i += 32) {
    const uint4 q = key4(i);
    const uint32_t k[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      gt += 4 * i + c < P && k[c] > thr ? 1u : 0u;
      eq += 4 * i + c < P && k[c] == thr ? 1u : 0u;
    }
  }
  __syncwarp();
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  __syncthreads();  // warp_a is read
  if (lane == 0) {
    warp_a[warp] = gt;
    warp_b[warp] = eq;
  }
  __syncthreads();
  // entries above and at the threshold before this warp's next 128
  uint32_t g = __reduce_add_sync(0xffffffffu, lane < warp ? warp_a[lane] : 0u);
  uint32_t e = __reduce_add_sync(0xffffffffu, lane < warp ? warp_b[lane] : 0u);
#pragma unroll 4
  for (int i = i0 + lane; i < i1; i += 32) {
    const uint4 q = i < quads ? key4(i) : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t k[4] = {q.x, q.y, q.z, q.w};
    uint32_t mine = 0, each[4];  // above the threshold, and at it in the upper half
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      each[c] = k[c] > thr ? 1u : k[c] == thr ? 0x10000u : 0u;
      if (4 * i + c >= P) each[c] = 0u;
      mine += each[c];
    }
    uint32_t run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, run, o);
      run += lane >= o ? up : 0u;
    }
    const uint32_t all = __shfl_sync(0xffffffffu, run, 31);
    uint32_t my_g = g + ((run - mine) & 0xffffu), my_e = e + ((run - mine) >> 16);
    if (mine)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (each[c] == 1u || (each[c] && my_e < left))
          a.kept[list0 + my_g + min(my_e, left)] = 4 * i + c;
        my_g += each[c] & 1u;
        my_e += each[c] >> 16;
      }
    g += all & 0xffffu;
    e += all >> 16;
  }
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
  grid_dependency_wait();  // (and no early start for the next kernel: this one writes prompt rows)
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
  return launch_overlapped(score_finish_kernel, dim3((unsigned)(v.B * v.H) * (unsigned)chunks),
                           dim3(kFinishThreads), 0, s, v, raw, score_in, score_out, chunks);
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
                                s->v_cache[(size_t)layer], out, st, true,
                                {scratch, score_in, score_out});
  if (e == cudaSuccess && s->dv.cluster_size == 0)
    e = launch_score_finish(s->dv, scratch, score_in, score_out, st);
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
  // (the list of a dst without prompt entries is empty: it may have no address)
  if (!score || !aligned16(score) || !aligned16(kept) || (dst_score && !aligned16(dst_score)))
    return RSWA_EINVAL;
  if (!kept && dst->dv.total_tokens > 0) return RSWA_EINVAL;
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
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  cudaError_t e = cudaStreamIsCapturing(st, &capture);
  if (e != cudaSuccess) return from_cuda(e);
  const unsigned rings = (unsigned)(a.batch * a.num_heads);
  const int max_p = src->dv.max_plen;
  const SelectArgs sel{src->dv, dst->dv, score, n_first, n_last, kept,
                       std::min((max_p + 3) / 4 * 4, kSelCache)};
  static bool attr_set[64] = {};  // per device
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    const cudaError_t err =
        cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (kSelBins + kSelCache) * (int)sizeof(uint32_t));
    if (err != cudaSuccess) return from_cuda(err);
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  // about four entries a thread, in the longest ring, until a CTA is full
  int threads = 128;
  while (threads < kSelMaxThreads && threads * 4 < max_p) threads *= 2;
  e = launch_overlapped(evict_select_kernel, dim3(rings), dim3((unsigned)threads),
                                    (size_t)(kSelBins + sel.cache) * sizeof(uint32_t), st, sel);
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
  auto *move = row_bytes == 128   ? evict_move_kernel<128>
               : row_bytes == 256 ? evict_move_kernel<256>
                                  : evict_move_kernel<512>;
  e = launch_overlapped(move, dim3(grid), dim3(kMoveThreads), 0, st, mv);
  if (e != cudaSuccess) return from_cuda(e);
  dst->dv.rope = src->dv.rope;
  dst->dv.rope_theta = src->dv.rope_theta;
  e = launch_rope_table(dst->dv, st);
  if (e != cudaSuccess) return from_cuda(e);
  dst->layer_ready[l] = kLayerEvicted;
  if (capture != cudaStreamCaptureStatusNone) dst->evict_captured = true;
  return RSWA_OK;
}

}  // extern "C"
