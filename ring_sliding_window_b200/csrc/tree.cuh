// Which cache entries a drafted token attends to; shared by the tree kernels.
#pragma once

#include <limits.h>
#include <stdint.h>

#include "internal.h"

namespace rswa {

// This step's view of one ring: entry `slot` has an age, the number of
// positions it lies before the first drafted token's (position P + t), and a
// draft at depth e, which is e positions further on, attends to it iff
//   age <= W - 1 - e,
// the same entries that the (e + 1)-th ordinary decode step would see.  Prompt
// entries have no age limit unless the standard sliding window cuts them too.
struct RingView {
  int plen, W;
  int held;     // slots [0, held) hold entries: P + min(t, W)
  int lo;       // slots below it are outside every draft's window (standard mode)
  int newest;   // ring index of the newest generated token, (t - 1) mod W
  int64_t t;
  bool swa;
};

__device__ __forceinline__ RingView ring_view(const DeviceView &v, int b, int plen) {
  RingView r;
  r.plen = plen;
  r.W = v.W;
  r.t = v.t[b];
  r.swa = v.swa != 0;
  r.held = plen + (int)(r.t < v.W ? r.t : (int64_t)v.W);
  // (32-bit division where it will do: this stands at the head of every piece)
  r.newest = r.t <= 0 ? 0
             : r.t <= INT_MAX ? (int)((uint32_t)(r.t - 1) % (uint32_t)v.W)
                              : (int)((r.t - 1) % v.W);
  const int64_t lo = (int64_t)plen + r.t - v.W + 1;
  r.lo = !r.swa || lo < 0 ? 0 : (lo > plen ? plen : (int)lo);
  return r;
}

// INT_MIN: every draft attends to the slot; INT_MAX: none does.
__device__ __forceinline__ int slot_age(const RingView &r, int slot) {
  if (slot >= r.held) return INT_MAX;
  if (slot < r.plen) {
    if (!r.swa) return INT_MIN;
    const int64_t a = (int64_t)r.plen + r.t - slot;
    return a > INT_MAX ? INT_MAX : (int)a;
  }
  const int a = r.newest - (slot - r.plen);
  return (a < 0 ? a + r.W : a) + 1;
}

}  // namespace rswa
