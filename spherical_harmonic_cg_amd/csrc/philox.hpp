// philox.hpp -- the counter-based random words of dropout: Philox 4x32 with
// ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", 2011).  One block of four 32-bit words for a 128-bit
// counter (block, offset) under a 64-bit key (seed); channel number j uses
// word j mod 4 of block j / 4.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

namespace eqtp {

struct DropState {
  uint32_t k0, k1, c2, c3;  // key, and the counter's high half
  uint32_t thr;             // keep if word >= thr = floor(p 2^32)
  float scale;              // 1 / (1 - p)
};

__device__ __forceinline__ DropState drop_state(const int64_t* __restrict__ rng, uint32_t thr, float scale) {
  const uint64_t seed = (uint64_t)rng[0], off = (uint64_t)rng[1];
  auto uni = [](uint64_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v); };
  return {uni(seed), uni(seed >> 32), uni(off), uni(off >> 32), thr, scale};
}
// At the head of a loop: the ten rounds' keys are made again instead of being kept in scalar registers.
__device__ __forceinline__ void forget_keys(DropState& s) { asm volatile("" : "+s"(s.k0), "+s"(s.k1)); }

// a ^ b ^ c as one instruction (its truth table is 0x96).
__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
  return (uint32_t)__builtin_amdgcn_bitop3_b32((int)a, (int)b, (int)c, 0x96);
}

// One round multiplies words 0 and 2 by the method's constants and crosses the
// halves of the products over; the key moves by two Weyl constants a round.
// The block's high word is an argument of its own: where it is the same for a wave, as the offset is, the first
// rounds' products of these words are scalar ones.
__device__ __forceinline__ void philox_words(const DropState& s, uint32_t lo, uint32_t hi, uint32_t (&w)[4]) {
  uint32_t c0 = lo, c1 = hi, c2 = s.c2, c3 = s.c3, k0 = s.k0, k1 = s.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
    c0 = r == 0 ? (uint32_t)(b >> 32) ^ c1 ^ k0 : xor3((uint32_t)(b >> 32), c1, k0);
    c2 = xor3((uint32_t)(a >> 32), c3, k1);
    c1 = (uint32_t)b;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  w[0] = c0, w[1] = c1, w[2] = c2, w[3] = c3;
}

// Bit i set: channel 4 block + i is kept.
__device__ __forceinline__ uint32_t keep_nibble(const DropState& s, uint32_t lo, uint32_t hi) {
  uint32_t w[4];
  philox_words(s, lo, hi, w);
  return (uint32_t)(w[0] >= s.thr) | (uint32_t)(w[1] >= s.thr) << 1 | (uint32_t)(w[2] >= s.thr) << 2 |
         (uint32_t)(w[3] >= s.thr) << 3;
}

__device__ __forceinline__ uint32_t keep_nibble(const DropState& s, uint64_t block) {
  return keep_nibble(s, (uint32_t)block, (uint32_t)(block >> 32));
}

// The value at place q of a quad with these keep bits.  The choice goes through a mask in a vector register: lane
// masks for every place of a row would not fit in the scalar registers.
__device__ __forceinline__ float drop_choose(uint32_t keep, int q, float kept, float dropped) {
  const uint32_t m = (uint32_t)__builtin_amdgcn_sbfe((int)keep, q, 1);
  return __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, kept) & m) | (__builtin_bit_cast(uint32_t, dropped) & ~m));
}

__device__ __forceinline__ float drop(uint32_t keep, int q, float x, float scale) {
  return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, x * scale) & (uint32_t)__builtin_amdgcn_sbfe((int)keep, q, 1));
}

// The same beside a residual; the norm's kernels and the dropout kernel share this expression, so their sums have
// the same bits.  fp32 values (E) take one rounding.  bf16 values take the rounded product and then the sum, as the
// separate fp32 operations do: 1 / (1 - p) is often a short fraction (10/9), multiples of its denominator then fall
// on exact ties of the bf16 steps, and a last bit more or less in fp32 would send them the other way (of bf16
// normal values at p = 0.1 about one sum in 2000, 1.3e-4 of an fp32 norm behind it).  Only where the sum cancels to
// less than 1/64 of the residual, and the product's rounding would weigh more than 2^-18 of it, the fused one.
template <class E>
__device__ __forceinline__ float drop_add(uint32_t keep, int q, float x, float scale, float residual) {
#pragma clang fp contract(off)
  float sum = fmaf(x, scale, residual);
  if constexpr (sizeof(E) == 2) {
    const float kept = x * scale, apart = kept + residual;
    sum = fabsf(apart) < 0.015625f * fabsf(residual) ? sum : apart;
  }
  return drop_choose(keep, q, sum, residual);
}

}  // namespace eqtp
