// norm.hip -- layer norm by degree of features [N, C, K], forward and
// backward, with the residual branch's dropout and sum in the same pass:
//   z = x, or residual + keep x / (1 - p);
//   zc = z - [l = 0] mean_c z;  r_l = 1 / sqrt(mean_{c, m of l} zc^2 + eps);
//   out = zc r_l weight[l, c] + [l = 0] bias[c].
// One workgroup a node; sums in fp32.
#include "eqtp_device.hpp"
#include "eqtp_kernels.hpp"
#include "philox.hpp"

namespace eqtp {

constexpr int kMaxDeg = 7;  // degrees 0..6

__device__ __forceinline__ int degree_of(int m) {
  return m >= 9 ? (m >= 25 ? (m >= 36 ? 6 : 5) : (m >= 16 ? 4 : 3)) : (m >= 4 ? 2 : (m >= 1 ? 1 : 0));
}

// Sums of NV values over a workgroup of 256, the same in every thread.
template <int NV>
__device__ __forceinline__ void block_sums(float (&v)[NV], float* lds) {
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int off = 32; off; off >>= 1) v[i] += __shfl_xor(v[i], off, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int i = 0; i < NV; ++i) lds[(threadIdx.x >> 6) * NV + i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = lds[i] + lds[NV + i] + lds[2 * NV + i] + lds[3 * NV + i];
}

template <class T, class O>
__global__ __launch_bounds__(256) void norm_kernel(NormArgs a) {
  __shared__ float red[4 * kMaxDeg];
  const int K = a.K, D = a.C * K;
  const int64_t n = blockIdx.x;
  const T* x = (const T*)a.x + n * D;
  const T* z = a.total ? (const T*)a.total + n * D : x;
  if (a.total) {
    const DropState s = a.rng ? drop_state(a.rng, a.thr, a.scale) : DropState{0, 0, 0, 0, 0, a.scale};
    const T* res = (const T*)a.residual + n * D;
    T* tot = (T*)a.total + n * D;
    for (int i = threadIdx.x; i < D; i += 256) {
      const int64_t j = n * a.C + i / K;
      const bool keep = a.rng == nullptr || (keep_nibble(s, (uint64_t)j >> 2) >> (j & 3) & 1);
      tot[i] = (T)drop_add(keep, (float)x[i], a.scale, (float)res[i]);  // read back by the thread that wrote it
    }
  }
  float mean[1] = {0.0f};
  for (int i = threadIdx.x; i < D; i += 256)
    if (i % K == 0) mean[0] += (float)z[i];
  block_sums<1>(mean, red);
  const float mu = mean[0] / a.C;
  float r[kMaxDeg] = {};
  for (int i = threadIdx.x; i < D; i += 256) {
    const int m = i % K, l = degree_of(m);
    const float t = (float)z[i] - (m == 0 ? mu : 0.0f);
#pragma unroll
    for (int d = 0; d < kMaxDeg; ++d) r[d] += l == d ? t * t : 0.0f;
  }
  block_sums<kMaxDeg>(r, red);
#pragma unroll
  for (int d = 0; d < kMaxDeg; ++d) r[d] = 1.0f / sqrtf(r[d] / (float)(a.C * (2 * d + 1)) + a.eps);
  for (int i = threadIdx.x; i < D; i += 256) {
    const int m = i % K, l = degree_of(m), c = i / K;
    float rl = r[0];
#pragma unroll
    for (int d = 1; d < kMaxDeg; ++d) rl = l == d ? r[d] : rl;
    const float zh = ((float)z[i] - (m == 0 ? mu : 0.0f)) * rl;
    ((O*)a.out)[n * D + i] = (O)fmaf(zh, a.weight ? a.weight[l * a.C + c] : 1.0f, m == 0 && a.bias ? a.bias[c] : 0.0f);
  }
  if (a.stats && threadIdx.x == 0) {
    float* st = a.stats + n * (a.lmax + 2);
    st[0] = mu;
#pragma unroll
    for (int d = 0; d < kMaxDeg; ++d)
      if (d <= a.lmax) st[1 + d] = r[d];
  }
}

template <class T, class O>
__global__ __launch_bounds__(256) void norm_grad_kernel(NormGradArgs a) {
  __shared__ float red[4 * (kMaxDeg + 1)];
  const int K = a.K, D = a.C * K;
  const int64_t n = blockIdx.x;
  const T* z = (const T*)a.total + n * D;
  const O* g = (const O*)a.gout + n * D;
  const float* st = a.stats + n * (a.lmax + 2);
  const float mu = st[0];
  float s[kMaxDeg + 1] = {};  // sums of a zhat by degree, then of a over the scalars
  for (int i = threadIdx.x; i < D; i += 256) {
    const int m = i % K, l = degree_of(m), c = i / K;
    const float zh = ((float)z[i] - (m == 0 ? mu : 0.0f)) * st[1 + l];
    const float av = (float)g[i] * (a.weight ? a.weight[l * a.C + c] : 1.0f);
#pragma unroll
    for (int d = 0; d < kMaxDeg; ++d) s[d] += l == d ? av * zh : 0.0f;
    s[kMaxDeg] += m == 0 ? av : 0.0f;
  }
  block_sums<kMaxDeg + 1>(s, red);
  const DropState ds = a.rng ? drop_state(a.rng, a.thr, a.scale) : DropState{0, 0, 0, 0, 0, a.scale};
  for (int i = threadIdx.x; i < D; i += 256) {
    const int m = i % K, l = degree_of(m), c = i / K;
    const float rl = st[1 + l];
    const float zh = ((float)z[i] - (m == 0 ? mu : 0.0f)) * rl;
    const float av = (float)g[i] * (a.weight ? a.weight[l * a.C + c] : 1.0f);
    float sl = s[0];
#pragma unroll
    for (int d = 1; d < kMaxDeg; ++d) sl = l == d ? s[d] : sl;
    float gz = rl * (av - (m == 0 ? s[kMaxDeg] / a.C : 0.0f) - zh * (sl / (float)(a.C * (2 * l + 1))));
    if (a.gtotal) gz += (float)((const T*)a.gtotal)[n * D + i];
    if (a.gres) ((T*)a.gres)[n * D + i] = (T)gz;
    if (a.gx) {
      const int64_t j = n * a.C + c;
      const bool keep = a.rng == nullptr || (keep_nibble(ds, (uint64_t)j >> 2) >> (j & 3) & 1);
      ((T*)a.gx)[n * D + i] = (T)drop_add(keep, gz, a.scale, 0.0f);
    }
  }
}

// Partial sums of grad_weight and grad_bias over a stretch of nodes: part
// [stretches][(lmax+2) C], one thread a column (the last C are the bias's).
template <class T, class O>
__global__ __launch_bounds__(256) void norm_weight_part_kernel(NormGradArgs a, int64_t stretch, float* part) {
  const int cols = (a.lmax + 2) * a.C, K = a.K;
  const int col = blockIdx.x * 256 + threadIdx.x;
  if (col >= cols) return;
  const int l = col / a.C, c = col % a.C;
  const int64_t n0 = blockIdx.y * stretch, n1 = n0 + stretch < a.N ? n0 + stretch : a.N;
  float acc = 0.0f;
  for (int64_t n = n0; n < n1; ++n) {
    const int64_t at = (n * a.C + c) * K;
    const float* st = a.stats + n * (a.lmax + 2);
    if (l > a.lmax) {
      acc += (float)((const O*)a.gout)[at];
    } else {
      for (int m = l * l; m < (l + 1) * (l + 1); ++m)
        acc += (float)((const O*)a.gout)[at + m] * (((float)((const T*)a.total)[at + m] - (m == 0 ? st[0] : 0.0f)) * st[1 + l]);
    }
  }
  part[(int64_t)blockIdx.y * cols + col] = acc;
}

__global__ __launch_bounds__(256) void norm_weight_sum_kernel(int cols, int wcols, int parts, const float* part,
                                                              float* gw, float* gb) {
  const int col = blockIdx.x * 256 + threadIdx.x;
  if (col >= cols) return;
  float acc = 0.0f;
  for (int p = 0; p < parts; ++p) acc += part[(int64_t)p * cols + col];
  if (col < wcols) {
    if (gw) gw[col] = acc;
  } else if (gb) {
    gb[col - wcols] = acc;
  }
}

constexpr int kParts = 256;

int64_t norm_workspace_floats(int64_t N, int C, int lmax) { return (int64_t)kParts * (lmax + 2) * C; }

template <class T, class O>
static hipError_t norm_t(const NormArgs& a) {
  hipLaunchKernelGGL((norm_kernel<T, O>), dim3((unsigned)a.N), dim3(256), 0, a.stream, a);
  return hipGetLastError();
}

hipError_t launch_norm(const NormArgs& a) {
  if (a.N == 0) return hipSuccess;
  if (a.x_bf16) return a.out_bf16 ? norm_t<__bf16, __bf16>(a) : norm_t<__bf16, float>(a);
  return a.out_bf16 ? norm_t<float, __bf16>(a) : norm_t<float, float>(a);
}

template <class T, class O>
static hipError_t norm_grad_t(const NormGradArgs& a) {
  if (a.N > 0 && (a.gres || a.gx)) {
    hipLaunchKernelGGL((norm_grad_kernel<T, O>), dim3((unsigned)a.N), dim3(256), 0, a.stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.gw || a.gb) {
    const int cols = (a.lmax + 2) * a.C;
    const int64_t stretch = (a.N + kParts - 1) / kParts;
    const unsigned cb = (unsigned)((cols + 255) / 256);
    hipLaunchKernelGGL((norm_weight_part_kernel<T, O>), dim3(cb, kParts), dim3(256), 0, a.stream, a, stretch, a.ws);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(norm_weight_sum_kernel, dim3(cb), dim3(256), 0, a.stream, cols, (a.lmax + 1) * a.C, kParts,
                       a.ws, a.gw, a.gb);
    return hipGetLastError();
  }
  return hipSuccess;
}

hipError_t launch_norm_grad(const NormGradArgs& a) {
  if (a.x_bf16) return a.out_bf16 ? norm_grad_t<__bf16, __bf16>(a) : norm_grad_t<__bf16, float>(a);
  return a.out_bf16 ? norm_grad_t<float, __bf16>(a) : norm_grad_t<float, float>(a);
}

}  // namespace eqtp
