// attention.hip -- attention over the edges of a graph (CSR rows), forward and
// backward; no per-edge vectors are formed in memory.
//   s = scale q[dst] . k[src] + bias,  w = softmax of s over the row,
//   out[n] = sum w v[src].
// One wave a (row, head); the softmax runs along the row with a running
// maximum and sum.
#include "eqtp_device.hpp"
#include "eqtp_kernels.hpp"

namespace eqtp {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

struct RowRange {
  int64_t b, e;
};
// The edges of row n, clamped into [0, E].
__device__ __forceinline__ RowRange row_range(const int32_t* __restrict__ ptr, int64_t n, int64_t E) {
  int64_t b = ptr[n], e = ptr[n + 1];
  b = b < 0 ? 0 : (b > E ? E : b);
  e = e < b ? b : (e > E ? E : e);
  return {b, e};
}

template <class T, int NE>
__global__ __launch_bounds__(256) void attn_kernel(AttnArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t task = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (task >= a.N * a.heads) return;
  const int64_t n = task / a.heads;
  const int h = (int)(task - n * a.heads), hk = h / (a.heads / a.kv_heads);
  const T* q = (const T*)a.q + task * a.D;
  float qr[NE], acc[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int d = lane + 64 * i;
    qr[i] = d < a.D ? (float)q[d] : 0.0f;
    acc[i] = 0.0f;
  }
  const RowRange r = row_range(a.row_ptr, n, a.E);
  float top = -INFINITY, sum = 0.0f;
  for (int64_t e = r.b; e < r.e; ++e) {
    const float bias = a.bias ? a.bias[e * a.heads + h] : 0.0f;
    if (bias == -INFINITY) continue;
    const int64_t at = ((int64_t)clamp_index(a.src[e], (int)a.M) * a.kv_heads + hk) * a.D;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int d = lane + 64 * i;
      if (d < a.D) dot = fmaf(qr[i], (float)((const T*)a.k)[at + d], dot);
    }
    const float s = fmaf(a.scale, wave_sum(dot), bias);
    const float t = fmaxf(top, s);
    const float w = s == -INFINITY ? 0.0f : __expf(s - t), keep = top == -INFINITY ? 0.0f : __expf(top - t);
    top = t;
    sum = fmaf(sum, keep, w);
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int d = lane + 64 * i;
      if (d < a.D) acc[i] = fmaf(acc[i], keep, w * (float)((const T*)a.v)[at + d]);
    }
  }
  const bool any = !(sum == 0.0f);
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int d = lane + 64 * i;
    if (d < a.D) ((T*)a.out)[task * a.D + d] = (T)(any ? acc[i] / sum : 0.0f);
  }
  if (a.lse && lane == 0) a.lse[task] = any ? top + logf(sum) : -INFINITY;
}

// Row pass of the gradients: grad_q, and per edge and head the weight w and
// u = w (a - t), a = g . v, which the source pass reads.  t = sum w a is known
// only at the row's end, so sum u k is formed as sum w a k - t sum w k, and a
// waits in u's place until then.
template <class T, int NE>
__global__ __launch_bounds__(256) void attn_grad_row_kernel(AttnGradArgs a, float* wts, float* us) {
  const int lane = threadIdx.x & 63;
  const int64_t task = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (task >= a.N * a.heads) return;
  const int64_t n = task / a.heads;
  const int h = (int)(task - n * a.heads), hk = h / (a.heads / a.kv_heads);
  float qr[NE], g[NE], wak[NE], wk[NE], t = 0.0f;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int d = lane + 64 * i;
    qr[i] = d < a.D ? (float)((const T*)a.q)[task * a.D + d] : 0.0f;
    g[i] = d < a.D ? (float)((const T*)a.gout)[task * a.D + d] : 0.0f;
    wak[i] = wk[i] = 0.0f;
  }
  const float lse = a.lse[task];
  const RowRange r = row_range(a.row_ptr, n, a.E);
  for (int64_t e = r.b; e < r.e; ++e) {
    const float bias = a.bias ? a.bias[e * a.heads + h] : 0.0f;
    float w = 0.0f, av = 0.0f;
    if (bias != -INFINITY) {
      const int64_t at = ((int64_t)clamp_index(a.src[e], (int)a.M) * a.kv_heads + hk) * a.D;
      float kr[NE], dot = 0.0f;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int d = lane + 64 * i;
        kr[i] = d < a.D ? (float)((const T*)a.k)[at + d] : 0.0f;
        dot = fmaf(qr[i], kr[i], dot);
        av = d < a.D ? fmaf(g[i], (float)((const T*)a.v)[at + d], av) : av;
      }
      const float s = fmaf(a.scale, wave_sum(dot), bias);
      av = wave_sum(av);
      if (s != -INFINITY) {
        w = __expf(s - lse);
        t = fmaf(w, av, t);
#pragma unroll
        for (int i = 0; i < NE; ++i) {
          wak[i] = fmaf(w * av, kr[i], wak[i]);
          wk[i] = fmaf(w, kr[i], wk[i]);
        }
      }
    }
    if (lane == 0) {
      wts[e * a.heads + h] = w;
      us[e * a.heads + h] = av;
    }
  }
  if (lane == 0)  // the lane that wrote them
    for (int64_t e = r.b; e < r.e; ++e) {
      const float w = wts[e * a.heads + h];
      us[e * a.heads + h] = w == 0.0f ? 0.0f : w * (us[e * a.heads + h] - t);
    }
  if (a.gq)
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int d = lane + 64 * i;
      if (d < a.D) ((T*)a.gq)[task * a.D + d] = (T)(fmaf(-t, wk[i], wak[i]) * a.scale);
    }
}

// Source pass: grad_k and grad_v of one (source, key and value head).
template <class T, int NE>
__global__ __launch_bounds__(256) void attn_grad_source_kernel(AttnGradArgs a, const float* wts, const float* us) {
  const int lane = threadIdx.x & 63;
  const int64_t task = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (task >= a.M * a.kv_heads) return;
  const int64_t m = task / a.kv_heads;
  const int R = a.heads / a.kv_heads, h0 = (int)(task - m * a.kv_heads) * R;
  float ka[NE] = {}, va[NE] = {};
  const RowRange r = row_range(a.src_ptr, m, a.E);
  for (int64_t i = r.b; i < r.e; ++i) {
    const int64_t e = clamp_index(a.perm[i], (int)a.E), n = clamp_index(a.dst_s[i], (int)a.N);
    for (int j = 0; j < R; ++j) {
      const float w = wts[e * a.heads + h0 + j], u = us[e * a.heads + h0 + j] * a.scale;
      if (w == 0.0f && u == 0.0f) continue;  // masked: whatever the row holds
      const int64_t at = (n * a.heads + h0 + j) * a.D;
#pragma unroll
      for (int x = 0; x < NE; ++x) {
        const int d = lane + 64 * x;
        if (d < a.D) {
          ka[x] = fmaf(u, (float)((const T*)a.q)[at + d], ka[x]);
          va[x] = fmaf(w, (float)((const T*)a.gout)[at + d], va[x]);
        }
      }
    }
  }
#pragma unroll
  for (int x = 0; x < NE; ++x) {
    const int d = lane + 64 * x;
    if (d < a.D) {
      if (a.gk) ((T*)a.gk)[task * a.D + d] = (T)ka[x];
      if (a.gv) ((T*)a.gv)[task * a.D + d] = (T)va[x];
    }
  }
}

int64_t attn_workspace_bytes(int64_t, int64_t, int64_t, int, int, int) { return 0; }

int64_t attn_grad_workspace_bytes(int64_t, int64_t, int64_t E, int, int heads, int) { return 2 * 4 * E * heads; }

template <class T, int NE>
static hipError_t attn_t(const AttnArgs& a) {
  hipLaunchKernelGGL((attn_kernel<T, NE>), dim3((unsigned)((a.N * a.heads + 3) / 4)), dim3(256), 0, a.stream, a);
  return hipGetLastError();
}

template <class T, int NE>
static hipError_t attn_grad_t(const AttnGradArgs& a) {
  float* wts = (float*)a.ws;
  float* us = a.gbias ? a.gbias : wts + a.E * a.heads;
  if (a.N > 0) {
    hipLaunchKernelGGL((attn_grad_row_kernel<T, NE>), dim3((unsigned)((a.N * a.heads + 3) / 4)), dim3(256), 0, a.stream, a,
                       wts, us);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.M > 0 && (a.gk || a.gv))
    hipLaunchKernelGGL((attn_grad_source_kernel<T, NE>), dim3((unsigned)((a.M * a.kv_heads + 3) / 4)), dim3(256), 0,
                       a.stream, a, wts, us);
  return hipGetLastError();
}

#define EQTP_BY_WIDTH(F, T, a)              \
  ((a).D <= 64     ? F<T, 1>(a)             \
   : (a).D <= 128  ? F<T, 2>(a)             \
   : (a).D <= 256  ? F<T, 4>(a)             \
   : (a).D <= 512  ? F<T, 8>(a)             \
   : (a).D <= 1024 ? F<T, 16>(a)            \
                   : F<T, 32>(a))

hipError_t launch_attention(const AttnArgs& a) {
  return a.bf16 ? EQTP_BY_WIDTH(attn_t, __bf16, a) : EQTP_BY_WIDTH(attn_t, float, a);
}

hipError_t launch_attention_grad(const AttnGradArgs& a) {
  return a.bf16 ? EQTP_BY_WIDTH(attn_grad_t, __bf16, a) : EQTP_BY_WIDTH(attn_grad_t, float, a);
}

}  // namespace eqtp
