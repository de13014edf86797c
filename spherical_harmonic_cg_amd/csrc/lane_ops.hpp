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

// One value from the lanes of a pair: lanes without the bit keep a, lanes with it b; CTRL brings the other lane's.
template <int CTRL>
__device__ __forceinline__ float dpp_fold(float a, float b, bool bit) {
  const float keep = bit ? b : a, give = bit ? a : b;
  return keep + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, give), CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ float fold16(float a, float b) {  // odd rows of 16 lanes end with b's sum
  const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, a), __builtin_bit_cast(unsigned, b), false, false);
  return __builtin_bit_cast(float, (unsigned)r[0]) + __builtin_bit_cast(float, (unsigned)r[1]);
}
__device__ __forceinline__ float fold32(float a, float b) {  // the upper half of the wave ends with b's sum
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, a), __builtin_bit_cast(unsigned, b), false, false);
  return __builtin_bit_cast(float, (unsigned)r[0]) + __builtin_bit_cast(float, (unsigned)r[1]);
}

// Sums of eight values over groups of G lanes (8 to 64): lane i of a group ends with the sum of value i / (G / 8).
// Every step halves the values a lane holds, about 20 instructions in all; one sum after the other takes eight times
// log2 G steps.
template <int G>
__device__ __forceinline__ float lane_sums8(const float (&v)[8]) {
  const int lane = threadIdx.x & 63;
  float a[4], b[2];
  if constexpr (G == 64) {
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = fold32(v[i], v[i + 4]);
    b[0] = fold16(a[0], a[2]);
    b[1] = fold16(a[1], a[3]);
    return dpp_plus<0xB1>(dpp_plus<0x4E>(dpp_plus<0x141>(dpp_fold<0x140>(b[0], b[1], lane & 8))));
  } else if constexpr (G == 32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = fold16(v[i], v[i + 4]);
    b[0] = dpp_fold<0x140>(a[0], a[2], lane & 8);
    b[1] = dpp_fold<0x140>(a[1], a[3], lane & 8);
    return dpp_plus<0xB1>(dpp_plus<0x4E>(dpp_fold<0x141>(b[0], b[1], lane & 4)));
  } else if constexpr (G == 16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = dpp_fold<0x140>(v[i], v[i + 4], lane & 8);
    b[0] = dpp_fold<0x141>(a[0], a[2], lane & 4);
    b[1] = dpp_fold<0x141>(a[1], a[3], lane & 4);
    return dpp_plus<0xB1>(dpp_fold<0x4E>(b[0], b[1], lane & 2));
  } else {
    static_assert(G == 8, "groups of 8 to 64 lanes");
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = dpp_fold<0x141>(v[i], v[i + 4], lane & 4);
    b[0] = dpp_fold<0x4E>(a[0], a[2], lane & 2);
    b[1] = dpp_fold<0x4E>(a[1], a[3], lane & 2);
    return dpp_fold<0xB1>(b[0], b[1], lane & 1);
  }
}
// Which value's sum this lane has, and the sum (or what was made of it) of value d.
template <int G>
__device__ __forceinline__ int sum8_index() { return (threadIdx.x & (G - 1)) / (G / 8); }
template <int G>
__device__ __forceinline__ float sum8_of(float mine, int d) {
  const int lane = (threadIdx.x & 63 & ~(G - 1)) + d * (G / 8);
  return __builtin_bit_cast(float, __builtin_amdgcn_ds_bpermute(4 * lane, __builtin_bit_cast(int, mine)));
}

}  // namespace eqtp
