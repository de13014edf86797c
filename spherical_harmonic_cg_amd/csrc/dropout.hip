// dropout.hip -- dropout of whole channels from a counter-based generator,
// with an optional residual sum: out = residual + keep(n, c) x / (1 - p).
//
// Bound by HBM (each element read and written once) next to the vector ALUs
// that make the random words: one Philox block (ten rounds) serves four
// channels, 4 K elements.  A wave takes a stretch of 4 x 64 units of 16 bytes.
// With K = 1 a thread's four (eight, bf16) elements are one (two) whole blocks and it
// makes its own bits.  With K > 1 the stretch touches few channels: the lanes
// make one block each, once, leave the keep bits in LDS and read them back
// element by element; made by every thread for itself, the words would take
// K times the work.  266k x 64 bf16 (K = 1): 14 us (68 MB), 18 us beside a
// residual (102 MB); the vector ALUs, the words' multiplications (18 of four
// passes a block) above all, are busy 69% of the time; fp32 with K = 49:
// 5.8 TB/s.
#include <type_traits>

#include "eqtp_device.hpp"
#include "eqtp_kernels.hpp"
#include "philox.hpp"

namespace eqtp {

template <class T>
struct Unit {  // 16 bytes of elements, aligned as one element only
  static constexpr int VE = 16 / (int)sizeof(T);
  typedef T V __attribute__((ext_vector_type(VE), aligned(sizeof(T))));
  static __device__ __forceinline__ V load(const T* p, int left) {
    if (left >= VE) return *reinterpret_cast<const V*>(p);
    V t;
#pragma unroll
    for (int q = 0; q < VE; ++q) t[q] = q < left ? p[q] : (T)0.0f;
    return t;
  }
  static __device__ __forceinline__ void store(T* p, int left, const float (&v)[VE]) {
    if (left >= VE) {
      V t;
#pragma unroll
      for (int q = 0; q < VE; ++q) t[q] = (T)v[q];
      *reinterpret_cast<V*>(p) = t;
    } else {
#pragma unroll
      for (int q = 0; q < VE; ++q)
        if (q < left) p[q] = (T)v[q];
    }
  }
};

constexpr int kDropUnits = 4;  // units a thread in a stretch

// One stretch of `have` elements from `base` on; FULL: all of its units are whole, RES: with a residual.
template <class T, int K, bool FULL, bool RES>
__device__ __forceinline__ void drop_stretch(int64_t base, int have, int lane, uint8_t* nib, const T* x,
                                             const T* residual, const int64_t* __restrict__ rng, uint32_t thr,
                                             float scale, T* out) {
  using U = Unit<T>;
  constexpr int VE = U::VE, NJ = kDropUnits;
  typename U::V v[NJ], r[RES ? NJ : 1];  // as they lie in memory: all are on their way before the first is converted
#pragma unroll
  for (int j = 0; j < NJ; ++j) v[j] = U::load(x + base + VE * (lane + 64 * j), FULL ? VE : have - VE * (lane + 64 * j));
  if constexpr (RES) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      r[j] = U::load(residual + base + VE * (lane + 64 * j), FULL ? VE : have - VE * (lane + 64 * j));
  }
  float o[NJ][VE];
  auto put = [&](uint32_t keep, int place, int j, int q) {
    if constexpr (RES)
      o[j][q] = drop_add<T>(keep, place, (float)v[j][q], scale, (float)r[j][q]);
    else
      o[j][q] = drop(keep, place, (float)v[j][q], scale);
  };
  if (rng) {
    const DropState s = drop_state(rng, thr, scale);
    if constexpr (K == 1) {
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int h = 0; h < VE; h += 4) {
          // stretches begin at multiples of their length, a power of two: no carry into the high word
          const uint32_t keep = keep_nibble(s, (uint32_t)(base >> 2) + (VE * (lane + 64 * j) + h) / 4, (uint32_t)(base >> 34));
#pragma unroll
          for (int q = 0; q < 4; ++q) put(keep, q, j, h + q);
        }
    } else {
      const int64_t c0 = base / K;             // first channel number of the stretch
      const int shift = (int)(base - c0 * K);  // elements of it before the stretch
      const int64_t b0 = c0 >> 2;
      const int blocks = (int)(((base + have - 1) / K >> 2) - b0) + 1, first = (int)(c0 & 3);
      wave_lds_sync();  // the stretch before has been read
#pragma unroll 1
      for (int i = lane; i < blocks; i += 64) nib[i] = (uint8_t)keep_nibble(s, (uint64_t)(b0 + i));
      wave_lds_sync();
      constexpr int G = K % 4 == 0 ? 4 : 1;  // elements that surely share a channel
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int q = 0; q < VE; q += G) {
          int i = VE * (lane + 64 * j) + q;
          if (!FULL) i = min(i, have - 1);
          const int c = first + (shift + i) / K;
          const uint32_t keep = nib[c >> 2] >> (c & 3);
#pragma unroll
          for (int k = q; k < q + G; ++k) put(keep, 0, j, k);
        }
    }
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int q = 0; q < VE; ++q) put(1, 0, j, q);
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) U::store(out + base + VE * (lane + 64 * j), FULL ? VE : have - VE * (lane + 64 * j), o[j]);
}

template <class T, int K, bool RES>
__global__ __launch_bounds__(256) void dropout_kernel(int64_t total, const T* x, const T* residual,
                                                      const int64_t* __restrict__ rng, uint32_t thr, float scale,
                                                      T* out) {
  constexpr int STRETCH = 64 * kDropUnits * Unit<T>::VE;
  __shared__ uint8_t nib[4][K == 1 ? 1 : STRETCH / (4 * K) + 3];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int64_t base = ((int64_t)blockIdx.x * 4 + wv) * STRETCH; base < total; base += (int64_t)gridDim.x * 4 * STRETCH) {
    if (total - base >= STRETCH)
      drop_stretch<T, K, true, RES>(base, STRETCH, lane, nib[wv], x, residual, rng, thr, scale, out);
    else
      drop_stretch<T, K, false, RES>(base, (int)(total - base), lane, nib[wv], x, residual, rng, thr, scale, out);
  }
}

template <class T, int K>
static hipError_t dropout_t(const DropArgs& a) {
  const int64_t total = a.N * a.C * K, stretch = 4 * 64 * kDropUnits * Unit<T>::VE;
  if (total == 0) return hipSuccess;
  const int64_t want = (total + stretch - 1) / stretch, most = 1 << 20;
  auto* kernel = a.residual ? dropout_kernel<T, K, true> : dropout_kernel<T, K, false>;
  kernel<<<dim3((unsigned)(want < most ? want : most)), dim3(256), 0, a.stream>>>(
      total, (const T*)a.x, (const T*)a.residual, a.rng, a.thr, a.scale, (T*)a.out);
  return hipGetLastError();
}

template <class T>
static hipError_t dropout_k(const DropArgs& a) {
  switch (a.K) {
    case 1: return dropout_t<T, 1>(a);
    case 4: return dropout_t<T, 4>(a);
    case 9: return dropout_t<T, 9>(a);
    case 16: return dropout_t<T, 16>(a);
    case 25: return dropout_t<T, 25>(a);
    case 36: return dropout_t<T, 36>(a);
    case 49: return dropout_t<T, 49>(a);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_dropout(const DropArgs& a) { return a.bf16 ? dropout_k<__bf16>(a) : dropout_k<float>(a); }

}  // namespace eqtp
