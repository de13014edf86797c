// norm_device.hpp -- what the layer norm's forward and backward kernels share:
// the way a row of D = C K elements lies in a group of threads, sums over a
// group, the keep bits of a row's channels, and the choice of the group.
#pragma once

#include "eqtp_device.hpp"
#include "eqtp_kernels.hpp"
#include "lane_ops.hpp"
#include "philox.hpp"

namespace eqtp {

constexpr int kMaxDeg = 7;  // degrees 0..6

__device__ __forceinline__ int degree_of(int m) {
  return m >= 9 ? (m >= 25 ? (m >= 36 ? 6 : 5) : (m >= 16 ? 4 : 3)) : (m >= 4 ? 2 : (m >= 1 ? 1 : 0));
}

// ---- four consecutive elements, aligned as one element only ---------------
typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));
typedef __bf16 b4u __attribute__((ext_vector_type(4), aligned(2)));
typedef __bf16 b4 __attribute__((ext_vector_type(4)));

template <class T>
struct Quad;
template <>
struct Quad<float> {
  typedef f4 Raw;
  static __device__ __forceinline__ Raw load(const float* p) { return *reinterpret_cast<const f4u*>(p); }
  static __device__ __forceinline__ void store(float* p, const float (&v)[4]) {
    *reinterpret_cast<f4u*>(p) = f4u{v[0], v[1], v[2], v[3]};
  }
};
template <>
struct Quad<__bf16> {
  typedef b4 Raw;
  static __device__ __forceinline__ Raw load(const __bf16* p) { return *reinterpret_cast<const b4u*>(p); }
  static __device__ __forceinline__ void store(__bf16* p, const float (&v)[4]) {
    *reinterpret_cast<b4u*>(p) = b4u{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
  }
};

// `left` elements of the row are left from p on (0 or less: none); `tail`: there are rows whose last quad is short
// (the same for every thread).
template <class T>
__device__ __forceinline__ void store4(T* p, int left, bool tail, const float (&v)[4]) {
  if (left <= 0) return;
  if (tail && left < 4) {
#pragma unroll
    for (int q = 0; q < 3; ++q)
      if (q < left) p[q] = (T)v[q];
  } else {
    Quad<T>::store(p, v);
  }
}

// A thread's quads of a row as they lie in memory.  All loads of a row are issued before the first value is used, and
// none stands behind a branch of its own (a conversion inside such a branch waits for its load, and the next load for
// the conversion: bf16 rows took 1.8 times as long): a quad past the row, or the short one at its end, is loaded from
// the row's last four elements and put right afterwards.
template <class T, int NV>
struct RowQuads {
  typename Quad<T>::Raw raw[NV];
  template <class S>
  __device__ __forceinline__ void load(const T* row, const S& sl, int A, int D) {
    if (D >= 4) {
#pragma unroll
      for (int j = 0; j < NV; ++j) raw[j] = Quad<T>::load(row + (sl.on ? min(4 * (sl.t + A * j), D - 4) : 0));
    } else {  // (a row of one to three elements, in the first thread)
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) raw[j][q] = (T)0.0f;
      if (sl.t == 0)
#pragma unroll
        for (int q = 0; q < 3; ++q)
          if (q < D) raw[0][q] = row[q];
    }
  }
  // the values, zeros past the row (in the threads that take quads)
  template <class S>
  __device__ __forceinline__ void values(const S& sl, int A, int D, bool full, bool tail, float (&v)[NV][4]) const {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) v[j][q] = (float)raw[j][q];
    if (full || D < 4) return;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (4 * A * (j + 1) <= D) continue;             // all threads' quads lie in the row
      const int over = 4 * (sl.t + A * j) - (D - 4);  // places that the quad reaches past the row
      if (tail) {
        if (!__any(sl.on && over > 0)) continue;
        const float w[7] = {v[j][0], v[j][1], v[j][2], v[j][3], 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int q = 0; q < 4; ++q)
          v[j][q] = over <= 0 ? w[q] : (over == 1 ? w[q + 1] : (over == 2 ? w[q + 2] : (over == 3 ? w[q + 3] : 0.0f)));
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) v[j][q] = over > 0 ? 0.0f : v[j][q];
      }
    }
  }
};

// Waits for a value before a loop: left to its first use inside, the wait would be for everything in flight there,
// the stores of the round before included.
__device__ __forceinline__ void arrived(float& v) { asm volatile("" : "+v"(v)); }

// ---- sums over a group ------------------------------------------------------
// Sums of the first `count` of v over a group of T threads, the same in each.
// Groups of more than a wave use red [2][waves * (kMaxDeg + 1)], as
// group_sums8 does; `turn` alternates its halves, so one barrier a sum
// suffices.
template <int T, int NV>
__device__ __forceinline__ void group_sums(float (&v)[NV], int count, float* red, int& turn) {
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (i < count) v[i] = lane_sum<(T < 64 ? T : 64)>(v[i]);
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

// Sums of eight values over a group of T threads: a thread ends with that of value sum8_index.
template <int T>
__device__ __forceinline__ float group_sums8(const float (&v)[8], float* red, int& turn) {
  constexpr int G = T < 64 ? T : 64;
  float mine = lane_sums8<G>(v);
  if constexpr (T > 64) {
    constexpr int W = T / 64;
    float* r = red + turn * (W * (kMaxDeg + 1));
    turn ^= 1;
    const int k = sum8_index<64>();
    if ((threadIdx.x & 7) == 0) r[k * W + (threadIdx.x >> 6)] = mine;
    __syncthreads();
    mine = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) mine += r[k * W + w];
  }
  return mine;
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
#pragma unroll 1
    for (int i = t; i < blocks; i += T) nib[i] = (uint8_t)keep_nibble(s, b0 + i);
    sync();
  }
  static __device__ __forceinline__ void sync() {
    if constexpr (T > 64) __syncthreads();
    else wave_lds_sync();
  }
  // keep bits of a quad's slots (c: their channels, below C)
  __device__ __forceinline__ uint32_t quad(const DropState& s, const int (&c)[4]) const {
    if (direct) return keep_nibble(s, (first + c[0]) >> 2);
    const int off = (int)(first & 3);
    if constexpr (KT == 1) return 0u - (nib[(off + c[0]) >> 2] >> ((off + c[0]) & 3) & 1u);
    uint32_t bits = 0;
    if constexpr (KT == 2) {  // two channels at most
      const uint32_t a = nib[(off + c[0]) >> 2] >> ((off + c[0]) & 3) & 1u;
      const uint32_t b = nib[(off + c[3]) >> 2] >> ((off + c[3]) & 3) & 1u;
#pragma unroll
      for (int q = 0; q < 4; ++q) bits |= (c[q] == c[0] ? a : b) << q;
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) bits |= (nib[(off + c[q]) >> 2] >> ((off + c[q]) & 3) & 1u) << q;
    }
    return bits;
  }
};

// KT: 0 for K = 1, 1 for K a multiple of 4 (a quad lies in one channel), 2 for the odd K > 1.
// What a thread's four slots are.  The degrees are kept in one register and
// taken apart where they are used: held as lane masks they would fill the
// scalar registers several times over.  Component 0 is the one of degree 0.
template <int T, int KT>
struct Slots {
  int t, degrees, c0, wrap, step;
  bool on;  // takes quads
  __device__ __forceinline__ Slots(int K, int A) {
    t = threadIdx.x % T;
    on = t < A;
    step = 4 * A / K;
    degrees = 0;
    c0 = 4 * t / K;
    wrap = K - (4 * t - c0 * K);  // the first slot of the next channel (K > 4: there is one at most)
    if constexpr (KT != 0)
#pragma unroll
      for (int q = 0; q < 4; ++q) degrees |= degree_of((4 * t + q) % K) << (8 * q);
  }
  // at the head of a row: keeps what follows from t and the degrees out of the registers between rows
  __device__ __forceinline__ void row() { asm volatile("" : "+v"(t), "+v"(degrees), "+v"(c0), "+v"(wrap)); }
  __device__ __forceinline__ int l(int q) const { return KT == 0 ? 0 : degrees >> (8 * q) & 255; }
  __device__ __forceinline__ int channel(int q, int j) const {
    return c0 + j * step + (KT == 0 ? q : (KT == 1 ? 0 : (q >= wrap ? 1 : 0)));
  }
  // sums of slot values by degree, added into s
  __device__ __forceinline__ void by_degree(const float (&v)[4], int deg, float* s) const {
    if constexpr (KT == 0) {
      s[0] += (v[0] + v[1]) + (v[2] + v[3]);
    } else if constexpr (KT == 1) {
      // degrees begin at squares, which are 0 or 1 modulo 4: slots 1 to 3 share one, slot 0 may have another
      const int a = l(0), b = l(1);
      const float rest = (v[1] + v[2]) + (v[3] + (a == b ? v[0] : 0.0f));
#pragma unroll
      for (int d = 0; d < kMaxDeg; ++d)
        if (d < deg) s[d] += b == d ? rest : (a == d ? v[0] : 0.0f);
    } else {
#pragma unroll
      for (int d = 0; d < kMaxDeg; ++d)
        if (d < deg)
#pragma unroll
          for (int q = 0; q < 4; ++q) s[d] += l(q) == d ? v[q] : 0.0f;
    }
  }
  // the slots' own of values that lie as group_sums8 leaves them, degree l as value first + l
  __device__ __forceinline__ void of_degree(float mine, int first, float (&v)[4]) const {
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = sum8_of<(T < 64 ? T : 64)>(mine, first + l(q));
  }
  // slot q holds component 0 (KT = 1: quads begin at multiples of 4, so slot 0 only)
  __device__ __forceinline__ bool zero(int q) const { return KT == 0 || ((KT == 2 || q == 0) && l(q) == 0); }
  // the value at component 0, or the sum of the values there (K = 1)
  __device__ __forceinline__ float scalars(const float (&v)[4]) const {
    if constexpr (KT == 0) return (v[0] + v[1]) + (v[2] + v[3]);
    if constexpr (KT == 1) return zero(0) ? v[0] : 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q) s = zero(q) ? v[q] : s;
    return s;
  }
};

// threads of a workgroup: several rows of up to 64 threads, or one
constexpr int norm_threads(int T) { return T > 64 ? T : 256; }

// 1 / (C (2 d + 1)): what turns a degree's sum into a mean
struct NormInv {
  float v[kMaxDeg];
};
inline NormInv norm_inv(int C) {
  NormInv r;
  for (int d = 0; d < kMaxDeg; ++d) r.v[d] = (float)(1.0 / ((double)C * (2 * d + 1)));
  return r;
}

// ---- choice of the group ----------------------------------------------------
// The smallest group whose threads hold the row in four quads or fewer (512
// threads take the rest, up to nine: every row of up to 16384 elements).  The
// work beside the elements (two sums over the group, a square root for each
// degree) is the same for every thread of a group, so fewer threads do less of
// it; more quads a thread cost registers, and with them waves in flight.
// 825 fp32 elements, gradients: 128 threads of two quads 25 us, 64 of six 30;
// 64 bf16 elements, forward: 16 threads of one 17 us, 8 of two 16, 4 of four 21.
struct NormShape {
  int T, NV, A;
};
inline NormShape norm_shape(int C, int K) {
  const int D = C * K, Q = (D + 3) / 4;
  const int P = K % 4 == 0 ? K / 4 : K;
  NormShape s = {512, 0, 512 / P * P};
  for (int T : {8, 16, 32, 64, 128, 256}) {
    const int A = T / P * P;
    if (A > 0 && (Q + A - 1) / A <= 4) {
      s = {T, 0, A};
      break;
    }
  }
  s.NV = (Q + s.A - 1) / s.A;
  return s;
}

// Workgroups that walk over the rows: what the card holds at once, so that all of them finish together (with 4 a
// compute unit where registers allow 3, the last ones ran alone: half as fast).
template <auto kernel, int T>
inline int norm_grid(int64_t N) {
  static const int held = [&] {  // per kernel
    int n = 0;
    return hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, norm_threads(T), 0) == hipSuccess && n > 0 ? n : 1;
  }();
  const int64_t rows = norm_threads(T) / T;
  const int64_t want = (N + rows - 1) / rows, most = (int64_t)num_cus() * held;
  return (int)(want < most ? want : most);
}

// Calls F(T, NV) for a shape: NV is the next of the built sizes.  Fewer quads than a row may need are built where rows
// that need no more are common, because quads that stay empty cost registers, and in the gradients LDS and with it
// workgroups (bf16, us forward / trained, against the largest size alone): 8 threads, 200k x 64: 11.8 / 36 against 13.9 /
// 43; 16 threads, 200k x 8 x 9: 24 / 65, 29 / 88; 64 threads, 20k x 8 x 49 (two): 14 / 37, 16.6 / 47; 40k x 38 x 16
// (three): 19.6 / 60, 20.4 / 66; 128 threads, 20k x 33 x 25: 27 / 74, 30 / 99; 512 threads, 4k x 8192 (five): 34 / 104,
// 57 / 250.  32 and 256 threads meet fewer than three quads at odd K and K = 36 only.
#define EQTP_NORM_SHAPES(s, F)                                                     \
  ((s).T == 8     ? ((s).NV <= 2 ? F(8, 2) : F(8, 4))                              \
   : (s).T == 16  ? ((s).NV <= 2 ? F(16, 2) : F(16, 4))                            \
   : (s).T == 32  ? F(32, 4)                                                       \
   : (s).T == 64  ? ((s).NV <= 2 ? F(64, 2) : ((s).NV <= 3 ? F(64, 3) : F(64, 4))) \
   : (s).T == 128 ? ((s).NV <= 2 ? F(128, 2) : F(128, 4))                          \
   : (s).T == 256 ? F(256, 4)                                                      \
                  : ((s).NV <= 5 ? F(512, 5) : F(512, 9)))

}  // namespace eqtp
