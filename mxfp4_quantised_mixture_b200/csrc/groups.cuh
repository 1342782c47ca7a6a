// Row groups given by device offsets: group e holds rows [offsets[e],
// offsets[e + 1]).  In the padded order along a contraction axis every group
// starts at a multiple of kGroupAlign positions.
#pragma once

#include <stdint.h>

namespace moe {

constexpr int kMaxGroups = 256;
constexpr int kGroupAlign = 128;

// Rows [lo, hi) of group e, kept inside [0, S] whatever the offsets hold.
__device__ __forceinline__ void group_rows(const int32_t* __restrict__ offsets, int e, int64_t S,
                                           int64_t& lo, int64_t& hi) {
  const int64_t a = __ldg(offsets + e), b = __ldg(offsets + e + 1);
  lo = a < 0 ? 0 : (a > S ? S : a);
  hi = b < lo ? lo : (b > S ? S : b);
}

// Exclusive prefix sums of units(e) over e in [0, E) into pfx[0..E] (shared
// memory), by one whole warp; E <= kMaxGroups.
template <typename Int, typename Units>
__device__ __forceinline__ void group_prefix(int E, Int* pfx, Units units) {
  const int lane = threadIdx.x & 31;
  Int carry = 0;
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    const Int n = e < E ? units(e) : 0;
    Int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Int up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += up;
    }
    if (e < E) pfx[e] = carry + incl - n;
    carry += __shfl_sync(0xFFFFFFFFu, incl, 31);
  }
  if (lane == 0) pfx[E] = carry;
}

// The group whose units hold unit u: the last e with pfx[e] <= u (empty
// groups before it share its start, and are passed over).
__device__ __forceinline__ int group_of(const int64_t* pfx, int E, int64_t u) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pfx[mid] <= u)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

}  // namespace moe
