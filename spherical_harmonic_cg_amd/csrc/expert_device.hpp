// expert_device.hpp -- what the experts' linear and its weight gradient share:
// operands of the matrix-core products and how they are read from features.
#pragma once

#include "eqtp_device.hpp"
#include "eqtp_kernels.hpp"

namespace eqtp {

constexpr int kTile = 16;  // nodes of a tile: the columns of a matrix-core product

__device__ __forceinline__ int degree_of_plane(int m) {
  return m >= 9 ? (m >= 25 ? (m >= 36 ? 6 : 5) : (m >= 16 ? 4 : 3)) : (m >= 4 ? 2 : (m >= 1 ? 1 : 0));
}

// NP consecutive elements, aligned as a whole, or as one element only
template <class S, int NP, bool ALIGNED = false>
struct Run {
  typedef S V __attribute__((ext_vector_type(NP), aligned(ALIGNED ? NP * sizeof(S) : sizeof(S))));
  typedef S R __attribute__((ext_vector_type(NP)));
  static __device__ __forceinline__ R load(const S* p) { return *reinterpret_cast<const V*>(p); }
  static __device__ __forceinline__ void store(S* p, const R& v) { *reinterpret_cast<V*>(p) = v; }
};

// Components that a wave takes of a channel: 16 bytes of them where a channel has as many (fp32: 4; bf16: 8, or 4 at
// lmax 1), one at lmax 0.
constexpr int planes_at_once(bool bf16, int lmax) { return lmax == 0 ? 1 : (bf16 && lmax > 1 ? 8 : 4); }
constexpr int plane_groups(int K, int np) { return (K + np - 1) / np; }
// first component of a group: the last one ends with the channel, and takes some that the one before has, too
__device__ __forceinline__ int group_first(int g, int K, int np) { return min(g * np, K - np); }

}  // namespace eqtp
