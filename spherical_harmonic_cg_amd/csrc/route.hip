// route.hip -- routing of nodes to experts, and its gradient.
//   s[x] = exp(t[x]) / sum exp(t), or 1 / (1 + exp(-t[x]));  v = s + bias;
//   the groups of experts with the largest sum of their two best v stay open;
//   the k largest v of them are taken, the lower index first where v is equal;
//   weight = scale s / (sum of s over those taken), or scale s.
//
// Reads 4 N X bytes and writes 8 N k; bound by the choice's instructions: 100k
// nodes, 6 of 64 experts, 4 of 8 groups, sigmoid with a bias 31 us, where a copy
// of the bytes takes 6; its gradient 10 us (its bytes' time is the same).  1000 nodes, 2 of 8: 6 us.  A node's experts lie eight by eight
// in G lanes (G = 1 for up to 8 experts, 32 for 256), so a wave works on 64 / G
// nodes.  Each lane sorts its eight once; a round of the choice then compares
// the lanes' first ones, and the lane that had the best moves on.
//
// An expert that leads by a hair has to lead as in the formula, whatever fp32
// makes of it.  The choice is made in fp32 and looked at: an fp32 v is off by
// 2^-19 (1 + the largest |bias|) at most (the hardware's exponential and
// reciprocal, a step each, their arguments, the sum, the bias, and the three
// bits of its key that say where it lies), so where every one taken leads the
// next by more than twice that, and open groups the closed ones by four times,
// it is the formula's.  Where not -- one node in some hundreds, or equal scores
// -- the wave chooses again in 64 bits, with the index beside the value.
#include "norm_device.hpp"

namespace eqtp {

constexpr int kPer = 8;  // experts of a lane

// values of consecutive elements from index x on: `have` of them (0 to 8), the others `none`
template <class T>
__device__ __forceinline__ void load8(const T* p, int have, float none, float (&t)[kPer]) {
  if (have >= kPer) {
    const typename Quad<T>::Raw a = Quad<T>::load(p), b = Quad<T>::load(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t[i] = (float)a[i];
      t[4 + i] = (float)b[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) t[i] = i < have ? (float)p[i] : none;
  }
}

template <int CTRL>
__device__ __forceinline__ float dpp_max(float v) {
  return fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false)));
}
// largest of v over groups of G lanes (up to 32)
template <int G>
__device__ __forceinline__ float lane_max(float v) {
  if constexpr (G >= 2) v = dpp_max<0xB1>(v);
  if constexpr (G >= 4) v = dpp_max<0x4E>(v);
  if constexpr (G >= 8) v = dpp_max<0x141>(v);
  if constexpr (G >= 16) v = dpp_max<0x140>(v);
  if constexpr (G >= 32) {
    const unsigned a = __builtin_bit_cast(unsigned, v);
    const auto r = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    v = fmaxf(__builtin_bit_cast(float, (unsigned)r[0]), __builtin_bit_cast(float, (unsigned)r[1]));
  }
  return v;
}
template <int G>
__device__ __forceinline__ double lane_sum64(double v) {
#pragma unroll
  for (int o = 1; o < G; o <<= 1) v += __shfl_xor(v, o, G);
  return v;
}

// exp(t) by the hardware's power of two: 2 steps and t's rounding off
__device__ __forceinline__ float fast_exp(float t) { return __builtin_amdgcn_exp2f(t * 1.44269504088896340736f); }

constexpr float kNone = -__builtin_inff();
// takes part: not -inf and not NaN
template <class F>
__device__ __forceinline__ bool open_to(F v) { return v > -__builtin_inf(); }

// Groups of experts: closes (v = -inf) the experts of all but the best groups.  Returns by how much the worst open
// group leads the best closed one (the same in all lanes).  of: the experts' groups, of `size` each; vals [X] and sums [groups] of the row in LDS.
template <int G, class F>
__device__ __forceinline__ F close_groups(const RouteArgs& a, int lane, int size, const int (&of)[kPer], F (&v)[kPer], F* vals, F* sums) {
  const F low = (F)-__builtin_inf();
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (lane * kPer + i < a.X) vals[lane * kPer + i] = v[i];
  wave_lds_sync();
  for (int g = lane; g < a.groups; g += G) {
    F first = low, second = low;
    for (int i0 = 0; i0 < size; i0 += 8) {  // (eight reads beside each other, not one after the other's wait)
      F t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = vals[g * size + min(i0 + i, size - 1)];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i0 + i >= size) t[i] = low;
        second = t[i] > first ? first : (t[i] > second ? t[i] : second);
        first = t[i] > first ? t[i] : first;
      }
    }
    sums[g] = open_to(second) ? first + second : first;
  }
  wave_lds_sync();
  // lane's groups: whether each is among the best, marked in vals; and the border
  F worst = (F)__builtin_inf(), best = low;
  for (int g = lane; g < a.groups; g += G) {
    const F mine = sums[g];
    int ahead = 0;
    for (int o0 = 0; o0 < a.groups; o0 += 8) {
      F other[8];
#pragma unroll
      for (int o = 0; o < 8; ++o) other[o] = sums[min(o0 + o, a.groups - 1)];
#pragma unroll
      for (int o = 0; o < 8; ++o)
        ahead += o0 + o < a.groups && (other[o] > mine || (other[o] == mine && o0 + o < g));
    }
    const bool kept = ahead < a.top_groups;
    vals[g] = kept ? (F)1 : (F)0;  // (a group has at least one expert: g < X)
    if (kept) worst = mine < worst ? mine : worst;
    else best = mine > best ? mine : best;
  }
  wave_lds_sync();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int x = lane * kPer + i;
    if (x < a.X && vals[of[i]] == (F)0) v[i] = low;
  }
#pragma unroll
  for (int o = 1; o < G; o <<= 1) {
    const F w = __shfl_xor(worst, o, G), b = __shfl_xor(best, o, G);
    worst = w < worst ? w : worst;
    best = b > best ? b : best;
  }
  wave_lds_sync();  // the next values come into the same place
  return open_to(best) ? worst - best : (F)__builtin_inf();
}

// Keys: whole numbers in the order of the values, their lowest three bits the place in the lane (the lower index the
// larger key), so that a lane's eight are all different; values lose 2^-20 of themselves at most.
__device__ __forceinline__ int key_of(float v, int i) {
  const int s = __builtin_bit_cast(int, v);
  return ((s ^ (s >> 31 & 0x7fffffff)) & ~7) | (7 - i);
}
__device__ __forceinline__ float key_value(int key) {
  const int s = key & ~7;
  return __builtin_bit_cast(float, s ^ (s >> 31 & 0x7fffffff));
}
constexpr int kNoKey = (int)0x807fffff;  // -inf's, and those below: closed

__device__ __forceinline__ void order_two(int& a, int& b) {
  const int hi = max(a, b), lo = min(a, b);
  a = hi;
  b = lo;
}
// descending; 19 exchanges (odd-even merge sort)
__device__ __forceinline__ void sort8(int (&k)[kPer]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) order_two(k[i], k[i + 1]);
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    order_two(k[i], k[i + 2]);
    order_two(k[i + 1], k[i + 3]);
    order_two(k[i + 1], k[i + 2]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) order_two(k[i], k[i + 4]);
  order_two(k[2], k[4]);
  order_two(k[3], k[5]);
  order_two(k[1], k[2]);
  order_two(k[3], k[4]);
  order_two(k[5], k[6]);
}

template <int CTRL>
__device__ __forceinline__ int dpp_maxi(int v) {
  return max(v, __builtin_amdgcn_update_dpp(v, v, CTRL, 0xf, 0xf, false));
}
template <int G>
__device__ __forceinline__ int lane_maxi(int v) {
  if constexpr (G >= 2) v = dpp_maxi<0xB1>(v);
  if constexpr (G >= 4) v = dpp_maxi<0x4E>(v);
  if constexpr (G >= 8) v = dpp_maxi<0x141>(v);
  if constexpr (G >= 16) v = dpp_maxi<0x140>(v);
  if constexpr (G >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap((unsigned)v, (unsigned)v, false, false);
    v = max((int)r[0], (int)r[1]);
  }
  return v;
}

// close_groups for groups of 8, 16, 32, .. experts -- whole lanes -- from the lanes' sorted keys.
template <int G>
__device__ __forceinline__ float close_lanes(const RouteArgs& a, int lane, int size, int (&key)[kPer], float* sums) {
  float first = key[0] > kNoKey ? key_value(key[0]) : kNone, second = key[1] > kNoKey ? key_value(key[1]) : kNone;
  const int span = size / kPer;
  for (int o = 1; o < span; o <<= 1) {
    const float f = __shfl_xor(first, o, G), s = __shfl_xor(second, o, G);
    second = fmaxf(fminf(first, f), fmaxf(second, s));
    first = fmaxf(first, f);
  }
  const float mine = open_to(second) ? first + second : first;
  const int g = lane / span;
  if (g < a.groups && lane == g * span) sums[g] = mine;
  wave_lds_sync();
  int ahead = 0;
  for (int o0 = 0; o0 < a.groups; o0 += 8) {
    float other[8];
#pragma unroll
    for (int o = 0; o < 8; ++o) other[o] = sums[min(o0 + o, a.groups - 1)];
#pragma unroll
    for (int o = 0; o < 8; ++o) ahead += o0 + o < a.groups && (other[o] > mine || (other[o] == mine && o0 + o < g));
  }
  wave_lds_sync();  // the next row's sums come into the same place
  const bool kept = ahead < a.top_groups, is = g < a.groups;
  const float best = lane_max<G>(is && !kept ? mine : kNone);
  const float worst = -lane_max<G>(is && kept ? -mine : kNone);
  if (!kept)
#pragma unroll
    for (int i = 0; i < kPer; ++i) key[i] = kNoKey;
  return open_to(best) ? worst - best : __builtin_inff();
}

// The choice in 64 bits: taken[r] is the expert of place lane + r G.
template <int G, int P>
__device__ __forceinline__ void choose_wide(const RouteArgs& a, int lane, const float (&t)[kPer], const float (&bias)[kPer],
                                            float top, bool direct, int size, const int (&of)[kPer], double* vals, int (&taken)[P]) {
  double v[kPer];
  if (direct) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = (double)t[i];
  } else if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = 1.0 / (1.0 + exp(-(double)t[i])) + (double)bias[i];
  } else {
    double total = 0.0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      v[i] = exp((double)t[i] - (double)top);
      total += v[i];  // (0 past the last expert)
    }
    total = lane_sum64<G>(total);
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = v[i] / total + (double)bias[i];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (!(t[i] > kNone) || !open_to(v[i])) v[i] = -__builtin_inf();
  if (a.groups > 1) close_groups<G, double>(a, lane, size, of, v, vals, vals + a.X);
  for (int j = 0; j < a.k; ++j) {
    double best = -__builtin_inf();
    int at = -1;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (v[i] > best) {
        best = v[i];
        at = lane * kPer + i;
      }
#pragma unroll
    for (int o = 1; o < G; o <<= 1) {
      const double ob = __shfl_xor(best, o, G);
      const int oa = __shfl_xor(at, o, G);
      if (ob > best || (ob == best && oa >= 0 && (at < 0 || oa < at))) {
        best = ob;
        at = oa;
      }
    }
#pragma unroll
    for (int r = 0; r < P; ++r)
      if (j == lane + r * G) taken[r] = at;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (at == lane * kPer + i) v[i] = -__builtin_inf();
  }
}

// (four waves a SIMD: the choice in 64 bits would take registers from the ordinary one, 35 us with three)
template <class T, int G>
__global__ __launch_bounds__(256, 4) void route_kernel(RouteArgs a) {
  constexpr int R = 256 / G, P = (kMaxTopK + G - 1) / G;  // rows of a workgroup; places of a lane
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int lane = threadIdx.x % G, row = threadIdx.x / G;
  double* vals = reinterpret_cast<double*>(lds) + row * (a.X + a.groups);
  const int have = min(max(a.X - lane * kPer, 0), kPer);
  const int size = a.X / a.groups;
  const bool whole_lanes = size % kPer == 0 && (size & (size - 1)) == 0;
  int of[kPer];
  float bias[kPer], most = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    of[i] = (lane * kPer + i) / size;
    bias[i] = a.bias && i < have ? a.bias[lane * kPer + i] : 0.0f;
    const float b = fabsf(bias[i]);
    most = fmaxf(most, b < __builtin_inff() ? b : 0.0f);
  }
  const bool direct = a.bias == nullptr && a.groups == 1;  // the logits' order is the scores'
  const float off = direct ? 0.0f : 0x1p-19f * (1.0f + lane_max<G>(most));  // of a v, at most (keys' part included)
  for (int64_t n = (int64_t)blockIdx.x * R + row; n < a.N; n += (int64_t)gridDim.x * R) {
    float t[kPer], v[kPer], top = kNone, all = 0.0f;
    load8(static_cast<const T*>(a.logits) + n * a.X + (have ? lane * kPer : 0), have, kNone, t);
    bool nan = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      top = fmaxf(top, t[i]);
      nan |= t[i] != t[i];
    }
    const bool spoilt = lane_maxi<G>(nan) != 0;
    if (!a.sigmoid) {
      top = lane_max<G>(top);
      if (!direct || !a.renormalise) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          v[i] = fast_exp(t[i] - top);  // (0 past the last expert)
          all += v[i];
        }
        all = lane_sum<G>(all);
      }
    }
    if (direct) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = t[i] > kNone ? t[i] + 0.0f : kNone;  // (-0 becomes 0: keys tell them apart)
    } else {
      const float inv = a.sigmoid ? 1.0f : __builtin_amdgcn_rcpf(all);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        v[i] = (a.sigmoid ? __builtin_amdgcn_rcpf(1.0f + fast_exp(-t[i])) : v[i] * inv) + bias[i];
        if (!(t[i] > kNone) || !open_to(v[i])) v[i] = kNone;
      }
    }
    bool close = false;
    if (a.groups > 1 && !whole_lanes) {
      float* f = reinterpret_cast<float*>(vals);
      close = !(close_groups<G, float>(a, lane, size, of, v, f, f + a.X) > 4.0f * off);
    }
    int key[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) key[i] = key_of(v[i], i);
    sort8(key);
    if (a.groups > 1 && whole_lanes) close = !(close_lanes<G>(a, lane, size, key, reinterpret_cast<float*>(vals)) > 4.0f * off);
    // k rounds, and one for who comes next: the largest of the lanes' first keys; lane j of the row keeps the expert of
    // place j (j + G, ..).  Equal keys of two lanes: the one with the higher index goes, the next round meets the other.
    int taken[P];
#pragma unroll
    for (int r = 0; r < P; ++r) taken[r] = -1;
    float last = __builtin_inff();
    for (int j = 0; j <= a.k; ++j) {
      const int best = lane_maxi<G>(key[0]);
      const float value = key_value(best);
      // (an infinite v: looked at again, too)
      close |= best > kNoKey && !(last - value > fmaf(0x1p-20f, fmaxf(fabsf(value), last < __builtin_inff() ? fabsf(last) : 0.0f), 2.0f * off));
      last = value;
      if (j == a.k) break;
      const bool mine = key[0] == best && best > kNoKey;
      const int expert = lane_maxi<G>(mine ? lane * kPer + 7 - (best & 7) : -1);
#pragma unroll
      for (int r = 0; r < P; ++r)
        if (j == lane + r * G) taken[r] = expert;
      if (expert >> 3 == lane) {
#pragma unroll
        for (int i = 0; i < kPer - 1; ++i) key[i] = key[i + 1];
        key[kPer - 1] = kNoKey;
      }
    }
    if (__any(close)) choose_wide<G, P>(a, lane, t, bias, top, direct, size, of, vals, taken);
    // weights: s = exp(min(t, 0)) / (1 + exp(-|t|)), or exp(t - top) / all; renormalised ones from
    // exp(.. - the largest exponent among those taken), which neither under- nor overflows
    float w[P], lt[P], ref = a.renormalise ? kNone : (a.sigmoid ? 0.0f : top), sum = 0.0f;
#pragma unroll
    for (int r = 0; r < P; ++r) {
      if (spoilt) taken[r] = -1;
      lt[r] = taken[r] >= 0 ? (float)static_cast<const T*>(a.logits)[n * a.X + taken[r]] : 0.0f;
      if (a.renormalise && taken[r] >= 0) ref = fmaxf(ref, a.sigmoid ? fminf(lt[r], 0.0f) : lt[r]);
    }
    if (a.renormalise) ref = lane_max<G>(ref);
#pragma unroll
    for (int r = 0; r < P; ++r) {
      w[r] = 0.0f;
      if (taken[r] >= 0)
        w[r] = a.sigmoid ? expf(fminf(lt[r], 0.0f) - ref) / (1.0f + expf(-fabsf(lt[r]))) : expf(lt[r] - ref);
      sum += w[r];
    }
    sum = a.renormalise ? lane_sum<G>(sum) : (a.sigmoid ? 1.0f : all);
#pragma unroll
    for (int r = 0; r < P; ++r) {
      const int j = lane + r * G;
      if (j < a.k) {
        a.idx[n * a.k + j] = taken[r];
        a.weight[n * a.k + j] = taken[r] >= 0 ? w[r] / sum * a.scale : (spoilt ? __builtin_nanf("") : 0.0f);
      }
    }
  }
}

// Gradient: only those taken get one where the weights are renormalised or the scores are the logits' own.
//   p = s / sum (or s), g = scale gweight, dot = sum over those taken of g p:
//   renormalised: p (g - dot) [(1 - s) for sigmoid];  else s (1 - s) g, or p (g - dot) for every expert (g = 0 where not taken).
// Lane j of a row works on place j; the row goes through LDS, where the places' gradients are put among the others'.
template <class T, int G>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteArgs a) {
  constexpr int R = 256 / G, P = (kMaxTopK + G - 1) / G;
  __shared__ float rows[R][G * kPer];
  const int lane = threadIdx.x % G, row = threadIdx.x / G;
  const int have = min(max(a.X - lane * kPer, 0), kPer);
  const bool whole = !a.sigmoid && !a.renormalise;
  for (int64_t n = (int64_t)blockIdx.x * R + row; n < a.N; n += (int64_t)gridDim.x * R) {
    float t[kPer], top = kNone, all = 0.0f;
    if (whole) {
      load8(static_cast<const T*>(a.logits) + n * a.X + (have ? lane * kPer : 0), have, kNone, t);
#pragma unroll
      for (int i = 0; i < kPer; ++i) top = fmaxf(top, t[i]);
      top = lane_max<G>(top);
      if (top == kNone) top = 0.0f;  // (every expert is masked)
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        t[i] = expf(t[i] - top);
        all += t[i];
      }
      all = lane_sum<G>(all);
      if (all == 0.0f) all = 1.0f;
    }
    int taken[P];
    float lt[P], p[P], g[P], ref = a.renormalise ? kNone : (a.sigmoid ? 0.0f : top), sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int r = 0; r < P; ++r) {
      const int j = lane + r * G;
      taken[r] = j < a.k ? a.idx[n * a.k + j] : -1;
      g[r] = j < a.k ? a.gweight[n * a.k + j] * a.scale : 0.0f;
      if (taken[r] >= a.X) taken[r] = -1;
      lt[r] = taken[r] >= 0 ? (float)static_cast<const T*>(a.logits)[n * a.X + taken[r]] : 0.0f;
      if (a.renormalise && taken[r] >= 0) ref = fmaxf(ref, a.sigmoid ? fminf(lt[r], 0.0f) : lt[r]);
    }
    if (a.renormalise) ref = lane_max<G>(ref);
#pragma unroll
    for (int r = 0; r < P; ++r) {
      p[r] = 0.0f;
      if (taken[r] >= 0)
        p[r] = a.sigmoid ? expf(fminf(lt[r], 0.0f) - ref) / (1.0f + expf(-fabsf(lt[r]))) : expf(lt[r] - ref);
      sum += p[r];
    }
    sum = a.renormalise ? lane_sum<G>(sum) : (a.sigmoid ? 1.0f : all);
#pragma unroll
    for (int r = 0; r < P; ++r) {
      p[r] = taken[r] >= 0 ? p[r] / sum : 0.0f;
      dot = taken[r] >= 0 ? fmaf(g[r], p[r], dot) : dot;
    }
    dot = a.sigmoid && !a.renormalise ? 0.0f : lane_sum<G>(dot);
    float* mine = rows[row];
#pragma unroll
    for (int i = 0; i < kPer; i += 4)
      *reinterpret_cast<f4*>(mine + lane * kPer + i) =
          whole ? f4{0.0f - t[i] / all * dot, 0.0f - t[i + 1] / all * dot, 0.0f - t[i + 2] / all * dot, 0.0f - t[i + 3] / all * dot}
                : f4{0.0f, 0.0f, 0.0f, 0.0f};
    wave_lds_sync();
#pragma unroll
    for (int r = 0; r < P; ++r) {
      float v = p[r] * (g[r] - dot);
      if (a.sigmoid) v /= 1.0f + expf(lt[r]);  // 1 - s
      if (taken[r] >= 0) mine[taken[r]] = v;
    }
    wave_lds_sync();
    T* o = static_cast<T*>(a.glogits) + n * a.X + lane * kPer;
#pragma unroll
    for (int i = 0; i < kPer; i += 4) {
      const f4 q = *reinterpret_cast<const f4*>(mine + lane * kPer + i);
      const float v[4] = {q[0], q[1], q[2], q[3]};
      store4(o + i, have - i, true, v);
    }
    wave_lds_sync();  // the next row comes into the same place
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
