// expert_device.hpp -- what the experts' linear and its weight gradient share:
// operand types, and the stretches of components that a pass holds at once.
#pragma once

#include "eqtp_device.hpp"
#include "eqtp_kernels.hpp"

namespace eqtp {

constexpr int kTile = 16;  // nodes (or places) of a tile: the columns of a matrix-core product
constexpr int kMaxPlanes = 16;
constexpr int expert_threads(int C) { return C >= 128 ? 512 : 256; }  // a workgroup's

__device__ __forceinline__ int degree_of_plane(int m) {
  return m >= 9 ? (m >= 25 ? (m >= 36 ? 6 : 5) : (m >= 16 ? 4 : 3)) : (m >= 4 ? 2 : (m >= 1 ? 1 : 0));
}

// Components are worked on in stretches of whole degrees with at most 16 of them: degrees 0 to 3 together (or up to
// lmax), then 4, 5 and 6 one at a time.
__host__ __device__ constexpr int stretches_of(int lmax) { return lmax <= 3 ? 1 : lmax - 2; }
__host__ __device__ constexpr int stretch_first(int s) { return s == 0 ? 0 : (s + 3) * (s + 3); }
__host__ __device__ constexpr int stretch_planes(int s, int lmax) {
  return s == 0 ? num_comp(lmax < 3 ? lmax : 3) : 2 * (s + 3) + 1;
}

}  // namespace eqtp
