// The selection order of the routing kernels.
#pragma once

#include <climits>
#include <cstdint>

namespace moe {

// Selection order: key descending, then expert index ascending.  A key is
// mapped to an unsigned integer that orders the same way (-0 as +0; NaN, and
// "no candidate", as 0, below every key), so one warp-wide max reduction
// finds the best key and one min reduction over the lanes holding it the
// lowest expert index.
__device__ __forceinline__ uint32_t key_order(float key) {
  uint32_t u = __float_as_uint(key);
  if (key != key) return 0u;
  if (u == 0x80000000u) u = 0u;  // -0 ranks as +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Best (order, expert) pair of the warp; every lane gets the winner.
__device__ __forceinline__ void warp_best(uint32_t& bu, int& be) {
  const uint32_t m = __reduce_max_sync(0xffffffffu, bu);
  const uint32_t e = __reduce_min_sync(0xffffffffu, bu == m ? (uint32_t)be : 0xffffffffu);
  bu = m;
  be = (int)e;
}

}  // namespace moe
