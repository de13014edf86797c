// norm_device.hpp -- what the layer norm's forward and backward kernels share:
// the way a row of D = C K elements lies in a group of threads, sums over a
// group, the keep bits of a row's channels, and the choice of the group.
#pragma once

#include "eqtp_device.hpp"
#include "eqtp_kernels.hpp"
#include "philox.hpp"

namespace eqtp {

constexpr int kMaxDeg = 7;  // degrees 0..6

__device__ __forceinline__ int degree_of(int m) {
  return m >= 9 ? (m >= 25 ? (m >= 36 ? 6 : 5) : (m >= 16 ? 4 : 3)) : (m >= 4 ? 2 : (m >= 1 ? 1 : 0));
}

// ---- four consecutive elements, aligned as one element only ---------------
typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));
typedef __bf16 b4u __attribute__((ext_vector_type(4), aligned(2)));

__device__ __forceinline__ void load4(const float* p, int left, float (&v)[4]) {
  if (left >= 4) {
    const f4u t = *reinterpret_cast<const f4u*>(p);
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = t[q];
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = q < left ? p[q] : 0.0f;
  }
}
__device__ __forceinline__ void load4(const __bf16* p, int left, float (&v)[4]) {
  if (left >= 4) {
    const b4u t = *reinterpret_cast<const b4u*>(p);
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = (float)t[q];
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = q < left ? (float)p[q] : 0.0f;
  }
}
__device__ __forceinline__ void store4(float* p, int left, const float (&v)[4]) {
  if (left >= 4) {
    *reinterpret_cast<f4u*>(p) = f4u{v[0], v[1], v[2], v[3]};
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q < left) p[q] = v[q];
  }
}
__device__ __forceinline__ void store4(__bf16* p, int left, const float (&v)[4]) {
  if (left >= 4) {
    *reinterpret_cast<b4u*>(p) = b4u{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q < left) p[q] = (__bf16)v[q];
  }
}

// ---- sums over a group ------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
// over 16 lanes (rotations by 8, 4, 2, 1), every lane the same bits
__device__ __forceinline__ float sum16(float v) {
  v = dpp_add<0x128>(v);
  v = dpp_add<0x124>(v);
  v = dpp_add<0x122>(v);
  return dpp_add<0x121>(v);
}
// over a wave: the odd 16-lane rows change places with the even ones, then the halves
__device__ __forceinline__ float sum64(float v) {
  v = sum16(v);
  const unsigned a = __builtin_bit_cast(unsigned, v);
  const auto r = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  v = __builtin_bit_cast(float, (unsigned)r[0]) + __builtin_bit_cast(float, (unsigned)r[1]);
  const unsigned b = __builtin_bit_cast(unsigned, v);
  const auto s = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return __builtin_bit_cast(float, (unsigned)s[0]) + __builtin_bit_cast(float, (unsigned)s[1]);
}

// Sums of the first `count` of v over a group of T threads, the same in each.
// Groups of more than a wave use red [2][waves * NV]; `turn` alternates its
// halves, so one barrier a sum suffices.
template <int T, int NV>
__device__ __forceinline__ void group_sums(float (&v)[NV], int count, float* red, int& turn) {
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (i < count) v[i] = T == 16 ? sum16(v[i]) : sum64(v[i]);
  if constexpr (T > 64) {
    constexpr int W = T / 64;
    float* r = red + turn * (W * (kMaxDeg + 1));
    turn ^= 1;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i < count) r[i * W + (threadIdx.x >> 6)] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i < count) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) s += r[i * W + w];
        v[i] = s;
      }
  }
}

// ---- which channels of a row are kept -------------------------------------
// A nibble of keep bits for each counter block that the row touches, in LDS.
// With one component a channel and C a multiple of 4 a thread's quad is one
// whole block, and it makes its own nibble (no LDS).
template <int T, int KT>
struct KeepBits {
  uint8_t* nib;
  uint64_t first;  // first channel number of the row
  bool direct;
  __device__ __forceinline__ void begin(const DropState& s, int64_t n, int C, int t, uint8_t* lds) {
    nib = lds;
    first = (uint64_t)n * (uint64_t)C;
    direct = KT == 0 && (C & 3) == 0;
    if (direct) return;
    const uint64_t b0 = first >> 2;
    const int blocks = (int)(((first + C - 1) >> 2) - b0) + 1;
    sync();  // the row before has been read
    for (int i = t; i < blocks; i += T) nib[i] = (uint8_t)keep_nibble(s, b0 + i);
    sync();
  }
  static __device__ __forceinline__ void sync() {
    if constexpr (T > 64) __syncthreads();
    else wave_lds_sync();
  }
  // keep bits of the channels of slots 0..3 of a quad (c: their channels)
  __device__ __forceinline__ uint32_t quad(const DropState& s, const int (&c)[4]) const {
    if (direct) return keep_nibble(s, (first + c[0]) >> 2);
    const int off = (int)(first & 3);
    if constexpr (KT == 1) return (nib[(off + c[0]) >> 2] >> ((off + c[0]) & 3) & 1) ? 15u : 0u;
    uint32_t bits = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) bits |= (uint32_t)(nib[(off + c[q]) >> 2] >> ((off + c[q]) & 3) & 1) << q;
    return bits;
  }
};

// KT: 0 for K = 1, 1 for K a multiple of 4 (a quad lies in one channel), 2 for the odd K > 1.
// What a thread's four slots are.  The degrees are kept in one register and
// taken apart where they are used: held as lane masks they would fill the
// scalar registers several times over.  Component 0 is the one of degree 0.
template <int T, int KT>
struct Slots {
  int t, degrees, step, C, K;
  bool on;  // takes quads
  __device__ __forceinline__ Slots(int C_, int K_, int A) : C(C_), K(K_) {
    t = threadIdx.x % T;
    on = t < A;
    step = 4 * A / K;
    degrees = 0;
    if constexpr (KT != 0)
#pragma unroll
      for (int q = 0; q < 4; ++q) degrees |= degree_of((4 * t + q) % K) << (8 * q);
  }
  // at the head of a row: keeps what follows from t and the degrees out of the registers between rows
  __device__ __forceinline__ void row() { asm volatile("" : "+v"(t), "+v"(degrees)); }
  __device__ __forceinline__ int l(int q) const { return KT == 0 ? 0 : degrees >> (8 * q) & 255; }
  __device__ __forceinline__ int channel(int q, int j) const {
    return (KT == 0 ? 4 * t + q : (KT == 1 ? 4 * t / K : (4 * t + q) / K)) + j * step;
  }
  // sums of slot values by degree, added into s
  __device__ __forceinline__ void by_degree(const float (&v)[4], int deg, float* s) const {
    if constexpr (KT == 0) {
      s[0] += (v[0] + v[1]) + (v[2] + v[3]);
    } else {
#pragma unroll
      for (int d = 0; d < kMaxDeg; ++d)
        if (d < deg)
#pragma unroll
          for (int q = 0; q < 4; ++q) s[d] += l(q) == d ? v[q] : 0.0f;
    }
  }
  __device__ __forceinline__ void of_degree(const float* s, int deg, float (&v)[4]) const {
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = s[0];
    if constexpr (KT != 0)
#pragma unroll
      for (int d = 1; d < kMaxDeg; ++d)
        if (d < deg)
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = l(q) == d ? s[d] : v[q];
  }
  // the value at component 0, or the sum of the values there (K = 1)
  __device__ __forceinline__ float scalars(const float (&v)[4]) const {
    if constexpr (KT == 0) return (v[0] + v[1]) + (v[2] + v[3]);
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q) s += l(q) == 0 ? v[q] : 0.0f;
    return s;
  }
};

constexpr int norm_threads(int T) { return T > 256 ? T : 256; }

// ---- choice of the group ----------------------------------------------------
// The smallest group whose threads hold the row in at most four quads (five
// for 1024 threads, so that every row of up to 16384 elements fits).
struct NormShape {
  int T, NV, A;
};
inline NormShape norm_shape(int C, int K) {
  const int D = C * K, Q = (D + 3) / 4;
  const int P = K % 4 == 0 ? K / 4 : K;
  NormShape s = {1024, 5, 1024 / P * P};
  for (int T : {16, 64, 256, 1024}) {
    const int A = T / P * P;
    if (A == 0) continue;
    const int nv = (Q + A - 1) / A;
    if (nv <= 4) {
      s = {T, nv, A};
      break;
    }
  }
  return s;
}

// workgroups that walk over the rows: at most per_cu of 256 threads a compute unit
inline int norm_grid(int64_t N, int T, int per_cu) {
  const int64_t rows = norm_threads(T) / T;
  const int64_t want = (N + rows - 1) / rows, most = (int64_t)num_cus() * (T > 256 ? per_cu / 4 : per_cu);
  return (int)(want < most ? want : most);
}

// Calls F<T, NV> for a shape: NV is the next of the built sizes.
#define EQTP_NORM_SHAPES(s, F)                                            \
  ((s).T == 16   ? ((s).NV <= 1 ? F(16, 1) : ((s).NV <= 2 ? F(16, 2) : F(16, 4))) \
   : (s).T == 64  ? ((s).NV <= 2 ? F(64, 2) : F(64, 4))                   \
   : (s).T == 256 ? ((s).NV <= 2 ? F(256, 2) : F(256, 4))                 \
                  : ((s).NV <= 2 ? F(1024, 2) : F(1024, 5)))

}  // namespace eqtp
