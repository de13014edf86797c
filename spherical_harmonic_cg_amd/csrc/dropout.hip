// dropout.hip -- dropout of whole channels from a counter-based generator,
// with an optional residual sum: out = residual + keep(n, c) x / (1 - p).
#include "eqtp_device.hpp"
#include "eqtp_kernels.hpp"
#include "philox.hpp"

namespace eqtp {

// One element a thread.
template <class T>
__global__ __launch_bounds__(256) void dropout_kernel(int64_t total, int K, const T* x, const T* residual,
                                                      const int64_t* __restrict__ rng, uint32_t thr, float scale,
                                                      T* out) {
  const DropState s = rng ? drop_state(rng, thr, scale) : DropState{0, 0, 0, 0, 0, scale};
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t j = i / K;
    const bool keep = rng == nullptr || (keep_nibble(s, (uint64_t)j >> 2) >> (j & 3) & 1);
    out[i] = (T)drop_add(keep, (float)x[i], scale, residual ? (float)residual[i] : 0.0f);
  }
}

hipError_t launch_dropout(const DropArgs& a) {
  const int64_t total = a.N * a.C * a.K;
  if (total == 0) return hipSuccess;
  const int64_t want = (total + 255) / 256, most = 1 << 20;
  const dim3 grid((unsigned)(want < most ? want : most));
  if (a.bf16)
    hipLaunchKernelGGL((dropout_kernel<__bf16>), grid, dim3(256), 0, a.stream, total, a.K, (const __bf16*)a.x,
                       (const __bf16*)a.residual, a.rng, a.thr, a.scale, (__bf16*)a.out);
  else
    hipLaunchKernelGGL((dropout_kernel<float>), grid, dim3(256), 0, a.stream, total, a.K, (const float*)a.x,
                       (const float*)a.residual, a.rng, a.thr, a.scale, (float*)a.out);
  return hipGetLastError();
}

}  // namespace eqtp
