// route.hip -- routing of nodes to experts, and its gradient.
//   s[x] = exp(t[x]) / sum exp(t), or 1 / (1 + exp(-t[x]));  v = s + bias;
//   the groups of experts with the largest sum of their two best v stay open;
//   the k largest v of them are taken, the lower index first where v is equal;
//   weight = scale s / (sum of s over those taken), or scale s.
//
// Reads 4 N X bytes and writes 8 N k: bound by HBM where N is large, in
// practice by the choice's instructions.  A node's experts lie eight by eight
// in G lanes (G = 1 for up to 8 experts, 32 for 256), so a wave works on 64 / G
// nodes and a round of the choice costs each lane eight comparisons and log2 G
// exchanges.  v is held in 64 bits: an expert that leads by a hair leads here
// as in the formula.
#include "norm_device.hpp"

namespace eqtp {

constexpr int kPer = 8;  // experts of a lane

template <class T>
__device__ __forceinline__ float logit(const void* p, int64_t i) { return (float)static_cast<const T*>(p)[i]; }

// s of one expert in 64 bits; for softmax `top` and `total` are the row's
__device__ __forceinline__ double score64(double t, bool sigmoid, double top, double total) {
  return sigmoid ? 1.0 / (1.0 + exp(-t)) : exp(t - top) / total;
}

template <int G>
__device__ __forceinline__ double group_sum64(double v) {
#pragma unroll
  for (int o = 1; o < G; o <<= 1) v += __shfl_xor(v, o, G);
  return v;
}
template <int G>
__device__ __forceinline__ float group_sum32(float v) {
#pragma unroll
  for (int o = 1; o < G; o <<= 1) v += __shfl_xor(v, o, G);
  return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = 1; o < G; o <<= 1) v = fmaxf(v, __shfl_xor(v, o, G));
  return v;
}

// takes part: not -inf and not NaN
__device__ __forceinline__ bool open_to(double v) { return v > -__builtin_inf(); }

// Groups of experts: closes (v = -inf) the experts of all but the best groups.
// vals [X] and sums [groups] of the row in LDS (one wave's own).
template <int G>
__device__ __forceinline__ void close_groups(const RouteArgs& a, int lane, double (&v)[kPer], double* vals, double* sums) {
  const int size = a.X / a.groups;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (lane * kPer + i < a.X) vals[lane * kPer + i] = v[i];
  wave_lds_sync();
  for (int g = lane; g < a.groups; g += G) {
    double first = -__builtin_inf(), second = first;
    for (int i = 0; i < size; ++i) {
      const double t = vals[g * size + i];
      if (t > first) {
        second = first;
        first = t;
      } else if (t > second) {
        second = t;
      }
    }
    sums[g] = open_to(second) ? first + second : first;
  }
  wave_lds_sync();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int x = lane * kPer + i;
    if (x >= a.X) continue;
    const int g = x / size;
    const double mine = sums[g];
    int ahead = 0;
    for (int o = 0; o < a.groups; ++o) ahead += sums[o] > mine || (sums[o] == mine && o < g);
    if (ahead >= a.top_groups) v[i] = -__builtin_inf();
  }
  wave_lds_sync();  // the next row's values come into the same place
}

template <class T, int G>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
  constexpr int R = 256 / G;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int lane = threadIdx.x % G, row = threadIdx.x / G;
  double* vals = reinterpret_cast<double*>(lds) + row * (a.X + a.groups);
  float bias[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) bias[i] = a.bias && lane * kPer + i < a.X ? a.bias[lane * kPer + i] : 0.0f;
  for (int64_t n = (int64_t)blockIdx.x * R + row; n < a.N; n += (int64_t)gridDim.x * R) {
    float t[kPer];
    float top = -__builtin_inff();
    int spoilt = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int x = lane * kPer + i;
      t[i] = x < a.X ? logit<T>(a.logits, n * a.X + x) : -__builtin_inff();
      top = fmaxf(top, t[i]);
      spoilt |= t[i] != t[i];
    }
#pragma unroll
    for (int o = 1; o < G; o <<= 1) spoilt |= __shfl_xor(spoilt, o, G);
    const bool plain = a.bias == nullptr && a.groups == 1;  // the logits' order is the scores'
    double v[kPer];
    float all = 0.0f;  // sum of exp(t - top)
    if (!a.sigmoid) {
      top = group_max<G>(top);
      if (!plain) {
        double total = 0.0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          v[i] = exp((double)t[i] - (double)top);
          total += lane * kPer + i < a.X ? v[i] : 0.0;
        }
        total = group_sum64<G>(total);
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = v[i] / total + (double)bias[i];
        all = (float)total;
      } else if (!a.renormalise) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) all += lane * kPer + i < a.X ? expf(t[i] - top) : 0.0f;
        all = group_sum32<G>(all);
      }
    } else if (!plain) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = 1.0 / (1.0 + exp(-(double)t[i])) + (double)bias[i];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (plain) v[i] = (double)t[i];
      // a masked expert (logit -inf) is never taken, whatever its bias
      if (!(t[i] > -__builtin_inff()) || !open_to(v[i])) v[i] = -__builtin_inf();
    }
    if (a.groups > 1) close_groups<G>(a, lane, v, vals, vals + a.X);
    // k rounds: the largest v, the lower index where equal; lane j of the row keeps the one of round j (j + G, ..)
    float logit_of[kMaxTopK];
    int taken[kMaxTopK];
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j) {
      if (j >= a.k) break;
      double best = -__builtin_inf();
      int at = -1;
      float mine = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (v[i] > best) {
          best = v[i];
          at = lane * kPer + i;
          mine = t[i];
        }
#pragma unroll
      for (int o = 1; o < G; o <<= 1) {
        const double ob = __shfl_xor(best, o, G);
        const int oa = __shfl_xor(at, o, G);
        const float om = __shfl_xor(mine, o, G);
        if (ob > best || (ob == best && oa >= 0 && (at < 0 || oa < at))) {
          best = ob;
          at = oa;
          mine = om;
        }
      }
      taken[j] = spoilt ? -1 : at;
      logit_of[j] = mine;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (at == lane * kPer + i) v[i] = -__builtin_inf();
    }
    // weights: s = exp(min(t, 0)) / (1 + exp(-|t|)), or exp(t - top) / all; renormalised ones from
    // exp(.. - the largest exponent among those taken), which neither under- nor overflows
    float ref = 0.0f;
    if (a.renormalise) {
      ref = -__builtin_inff();
#pragma unroll
      for (int j = 0; j < kMaxTopK; ++j)
        if (j < a.k && taken[j] >= 0) ref = fmaxf(ref, a.sigmoid ? fminf(logit_of[j], 0.0f) : logit_of[j]);
    } else if (!a.sigmoid) {
      ref = top;
    }
    float w[kMaxTopK], sum = 0.0f;
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j) {
      if (j >= a.k) break;
      w[j] = 0.0f;
      if (taken[j] >= 0)
        w[j] = a.sigmoid ? expf(fminf(logit_of[j], 0.0f) - ref) / (1.0f + expf(-fabsf(logit_of[j]))) : expf(logit_of[j] - ref);
      sum += w[j];
    }
    if (!a.renormalise) sum = a.sigmoid ? 1.0f : all;
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j) {
      if (j >= a.k) break;
      if (j % G == lane) {
        a.idx[n * a.k + j] = taken[j];
        a.weight[n * a.k + j] = taken[j] >= 0 ? w[j] / sum * a.scale : (spoilt ? __builtin_nanf("") : 0.0f);
      }
    }
  }
}

// Gradient: only those taken get one where the weights are renormalised or the scores are the logits' own.
//   p = s / sum (or s), g = scale gweight, dot = sum over those taken of g p:
//   renormalised: p (g - dot) [(1 - s) for sigmoid];  else s (1 - s) g, or p (g - dot) for every expert (g = 0 where not taken).
template <class T, int G>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteArgs a) {
  constexpr int R = 256 / G;
  const int lane = threadIdx.x % G, row = threadIdx.x / G;
  for (int64_t n = (int64_t)blockIdx.x * R + row; n < a.N; n += (int64_t)gridDim.x * R) {
    const bool whole = !a.sigmoid && !a.renormalise;
    float t[kPer], top = -__builtin_inff(), all = 0.0f;
    if (whole) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int x = lane * kPer + i;
        t[i] = x < a.X ? logit<T>(a.logits, n * a.X + x) : -__builtin_inff();
        top = fmaxf(top, t[i]);
      }
      top = group_max<G>(top);
      if (top == -__builtin_inff()) top = 0.0f;  // (every expert is masked)
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        t[i] = lane * kPer + i < a.X ? expf(t[i] - top) : 0.0f;
        all += t[i];
      }
      all = group_sum32<G>(all);
      if (all == 0.0f) all = 1.0f;
    }
    int taken[kMaxTopK];
    float lt[kMaxTopK], p[kMaxTopK], g[kMaxTopK], ref = -__builtin_inff(), sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j) {
      if (j >= a.k) break;
      taken[j] = a.idx[n * a.k + j];
      if (taken[j] < 0 || taken[j] >= a.X) taken[j] = -1;
      g[j] = a.gweight[n * a.k + j] * a.scale;
      lt[j] = taken[j] >= 0 ? logit<T>(a.logits, n * a.X + taken[j]) : 0.0f;
      if (taken[j] >= 0) ref = fmaxf(ref, a.sigmoid ? fminf(lt[j], 0.0f) : lt[j]);
    }
    if (!a.renormalise) ref = a.sigmoid ? 0.0f : top;
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j) {
      if (j >= a.k) break;
      p[j] = 0.0f;
      if (taken[j] >= 0)
        p[j] = a.sigmoid ? expf(fminf(lt[j], 0.0f) - ref) / (1.0f + expf(-fabsf(lt[j]))) : expf(lt[j] - ref);
      sum += p[j];
    }
    if (!a.renormalise) sum = a.sigmoid ? 1.0f : all;
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j) {
      if (j >= a.k) break;
      p[j] = taken[j] >= 0 ? p[j] / sum : 0.0f;
      dot = taken[j] >= 0 ? fmaf(g[j], p[j], dot) : dot;
    }
    if (a.sigmoid && !a.renormalise) dot = 0.0f;
    float out[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) out[i] = whole ? 0.0f - t[i] / all * dot : 0.0f;
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j) {
      if (j >= a.k) break;
      float v = p[j] * (g[j] - dot);
      if (a.sigmoid) v /= 1.0f + expf(lt[j]);  // 1 - s
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (taken[j] >= 0 && taken[j] == lane * kPer + i) out[i] = v;
    }
    T* o = static_cast<T*>(a.glogits) + n * a.X;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane * kPer + i < a.X) o[lane * kPer + i] = (T)out[i];
  }
}

template <class T, int G, bool GRAD>
static hipError_t route_launch(const RouteArgs& a) {
  constexpr int R = 256 / G;
  const int64_t want = (a.N + R - 1) / R, most = (int64_t)num_cus() * 8;
  const dim3 grid((unsigned)(want < most ? want : most));
  if constexpr (GRAD) {
    route_grad_kernel<T, G><<<grid, dim3(256), 0, a.stream>>>(a);
  } else {
    const size_t bytes = a.groups > 1 ? sizeof(double) * R * (a.X + a.groups) : 0;
    route_kernel<T, G><<<grid, dim3(256), bytes, a.stream>>>(a);
  }
  return hipGetLastError();
}

template <class T, bool GRAD>
static hipError_t route_t(const RouteArgs& a) {
  if (a.X <= 8) return route_launch<T, 1, GRAD>(a);
  if (a.X <= 16) return route_launch<T, 2, GRAD>(a);
  if (a.X <= 32) return route_launch<T, 4, GRAD>(a);
  if (a.X <= 64) return route_launch<T, 8, GRAD>(a);
  if (a.X <= 128) return route_launch<T, 16, GRAD>(a);
  return route_launch<T, 32, GRAD>(a);
}

hipError_t launch_route(const RouteArgs& a) {
  if (a.N == 0) return hipSuccess;
  return a.bf16 ? route_t<__bf16, false>(a) : route_t<float, false>(a);
}
hipError_t launch_route_grad(const RouteArgs& a) {
  if (a.N == 0) return hipSuccess;
  return a.bf16 ? route_t<__bf16, true>(a) : route_t<float, true>(a);
}

}  // namespace eqtp
