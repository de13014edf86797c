// lane_ops.hpp -- sums over groups of lanes by register moves (no LDS).
#pragma once

#include <hip/hip_runtime.h>

namespace eqtp {

template <int CTRL>
__device__ __forceinline__ float dpp_plus(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}

// Sum over groups of G consecutive lanes (a power of two up to 64), the same bits in each of them: every step adds
// the two halves of a pair in either order.
template <int G>
__device__ __forceinline__ float lane_sum(float v) {
  if constexpr (G >= 2) v = dpp_plus<0xB1>(v);    // lanes 1 0 3 2
  if constexpr (G >= 4) v = dpp_plus<0x4E>(v);    // lanes 2 3 0 1
  if constexpr (G >= 8) v = dpp_plus<0x141>(v);   // mirrored in 8
  if constexpr (G >= 16) v = dpp_plus<0x140>(v);  // mirrored in 16
  if constexpr (G >= 32) {                        // odd rows of 16 lanes change places with the even ones
    const unsigned a = __builtin_bit_cast(unsigned, v);
    const auto r = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    v = __builtin_bit_cast(float, (unsigned)r[0]) + __builtin_bit_cast(float, (unsigned)r[1]);
  }
  if constexpr (G >= 64) {                        // the halves of the wave
    const unsigned a = __builtin_bit_cast(unsigned, v);
    const auto r = __builtin_amdgcn_permlane32_swap(a, a, false, false);
    v = __builtin_bit_cast(float, (unsigned)r[0]) + __builtin_bit_cast(float, (unsigned)r[1]);
  }
  return v;
}

}  // namespace eqtp
