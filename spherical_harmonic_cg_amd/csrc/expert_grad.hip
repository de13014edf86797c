// expert_grad.hip -- gradient of the experts' weights,
//   grad_W[x, l, c', c] = sum over the places (n, j) of expert x of
//                         weight[n, j] sum_m grad_out[n, c', l m] h[n, c, l m].
//
// Places come grouped by expert (expert_plan.hip); a workgroup takes a chunk of
// one expert's places and keeps all of its C x C matrices in registers: 16x16
// tiles of outer products over 16 places at a time on the matrix cores.  fp32:
// the products' operands are fp32.  bf16: a gate's product with the gradient is
// held in two bf16 parts, both multiplied: 2^-16 of a term at most is lost.  Chunks go to lines of part, which a second kernel adds in a fixed
// order: no atomics, the same bits from call to call.
#include <type_traits>

#include "expert_device.hpp"

namespace eqtp {

template <class S, int C, bool GATES>
struct ExpertGradCfg {
  static constexpr bool BF16 = std::is_same<S, __bf16>::value;
  static constexpr int ES = (int)sizeof(S);
  // fp32: planes [place][channel], bf16: [channel][place], as the operands are read
  static constexpr int TS = BF16 ? 16 : (C >= 128 ? 8 : 16);  // places at a time (LDS)
  static constexpr int RS = BF16 ? 16 + 4 : C + 16;
  static constexpr int PLANE = BF16 ? C * RS : TS * RS;
  static constexpr int WAVES = expert_threads(C) / 64;
  static constexpr int CT = (C + 15) / 16;
  static constexpr int PG = WAVES / CT > 0 ? WAVES / CT : 1;  // waves that share a tile of output channels: parts of the degrees
  static constexpr int LPW = (4 + PG - 1) / PG;               // degrees of a wave
  static constexpr int SETS = BF16 && GATES ? 3 : 2;          // gradient (in two parts) and features
  static constexpr int PP = 8;                                // planes at a time (LDS)
  static size_t lds_bytes(int planes) { return (size_t)SETS * (planes < PP ? planes : PP) * PLANE * ES; }
};

struct ChunkOf {
  int x;            // expert, or -1
  int64_t s0, s1;   // its places
};
// chunk b of the experts' places, `per` places at most each
__device__ __forceinline__ ChunkOf chunk_of(const int32_t* ptr, int X, int64_t places, int per, int b) {
  ChunkOf r = {-1, 0, 0};
  int at = 0;
  for (int x = 0; x < X; ++x) {
    const int64_t lo = min(max((int64_t)ptr[x], (int64_t)0), places), hi = min(max((int64_t)ptr[x + 1], lo), places);
    const int n = (int)((hi - lo + per - 1) / per);
    if (b < at + n) {
      r.x = x;
      r.s0 = lo + (int64_t)(b - at) * per;
      r.s1 = min(r.s0 + per, hi);
      return r;
    }
    at += n;
  }
  return r;
}

typedef short bf16x4s __attribute__((ext_vector_type(4)));

template <class S, int C, bool GATES>
__global__ __launch_bounds__(expert_threads(C)) void expert_grad_kernel(ExpertGradArgs a, int per) {
  using Cfg = ExpertGradCfg<S, C, GATES>;
  constexpr int TH = 64 * Cfg::WAVES, TS = Cfg::TS;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  __shared__ int node[TS];
  __shared__ float gate[TS];
  const int st = blockIdx.y;
  const int K = num_comp(a.lmax), m0 = stretch_first(st), np = stretch_planes(st, a.lmax);
  const int l0 = st == 0 ? 0 : st + 3, ln = st == 0 ? min(a.lmax, 3) + 1 : 1;
  constexpr int PP = Cfg::PP;
  const int held = min(np, PP);
  S* gT = reinterpret_cast<S*>(lds);
  S* gL = gT + held * Cfg::PLANE;  // bf16: what the first part leaves
  S* hT = gT + (Cfg::SETS - 1) * held * Cfg::PLANE;
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i16 = lane & 15, kq = lane >> 4, ct = wv % Cfg::CT, pg = wv / Cfg::CT;
  const ChunkOf ch = chunk_of(a.ptr, a.X, a.N * a.k, per, blockIdx.x);
  if (ch.x < 0) return;
  f4 acc[Cfg::LPW][Cfg::CT];
#pragma unroll
  for (int i = 0; i < Cfg::LPW; ++i)
#pragma unroll
    for (int t = 0; t < Cfg::CT; ++t) acc[i][t] = f4{0.f, 0.f, 0.f, 0.f};
  for (int64_t s = ch.s0; s < ch.s1; s += TS) {
    const int nv = (int)min((int64_t)TS, ch.s1 - s);
    __syncthreads();
    if (tid < TS) {
      const int64_t slot = tid < nv ? (int64_t)clamp_index(a.slots[s + tid], (int)min(a.N * a.k, (int64_t)0x7fffffff)) : 0;
      node[tid] = (int)(slot / a.k);
      gate[tid] = GATES ? a.weight[slot] : 1.0f;
    }
    for (int pm = 0; pm < np; pm += PP) {
      const int pn = min(PP, np - pm);
      __syncthreads();
      for (int i = tid; i < TS * C; i += TH) {
        const int r = i / C, c = i - r * C;
        const int64_t at = ((int64_t)node[r] * C + c) * K + m0 + pm;
        const float w = gate[r];
        for (int m = 0; m < pn; ++m) {
          const S g = r < nv ? static_cast<const S*>(a.gout)[at + m] : (S)0.0f;
          const S h = r < nv ? static_cast<const S*>(a.h)[at + m] : (S)0.0f;
          const int to = m * Cfg::PLANE + (Cfg::BF16 ? c * Cfg::RS + r : r * Cfg::RS + c);
          hT[to] = h;
          const float wg = GATES && r < nv ? w * (float)g : (float)g;
          gT[to] = (S)wg;
          if constexpr (Cfg::BF16 && GATES) gL[to] = (S)(wg - (float)(S)wg);
        }
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < Cfg::LPW; ++i) {
        const int dl = pg + i * Cfg::PG;
        if (dl >= ln) break;
        const int l = l0 + dl;
        const int ma = max(l * l - m0 - pm, 0), mb = min((l + 1) * (l + 1) - m0 - pm, pn);
        for (int m = ma; m < mb; ++m) {
          const int row = ct * 16 + i16 < C ? ct * 16 + i16 : 0;
          if constexpr (Cfg::BF16) {
            const int at = m * Cfg::PLANE + row * Cfg::RS + 4 * kq;
            const bf16x4s ga = *reinterpret_cast<const bf16x4s*>(gT + at);
            bf16x4s gb = {};
            if constexpr (GATES) gb = *reinterpret_cast<const bf16x4s*>(gL + at);
#pragma unroll
            for (int t = 0; t < Cfg::CT; ++t) {
              const int col = t * 16 + i16 < C ? t * 16 + i16 : 0;
              const bf16x4s hb = *reinterpret_cast<const bf16x4s*>(hT + m * Cfg::PLANE + col * Cfg::RS + 4 * kq);
              acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(ga, hb, acc[i][t], 0, 0, 0);
              if constexpr (GATES) acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(gb, hb, acc[i][t], 0, 0, 0);
            }
          } else {
#pragma unroll
            for (int q = 0; q < TS; q += 4) {
              const int base = m * Cfg::PLANE + (q + kq) * Cfg::RS;
              const float ga = gT[base + row];
#pragma unroll
              for (int t = 0; t < Cfg::CT; ++t) {
                const int col = t * 16 + i16 < C ? t * 16 + i16 : 0;
                acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(ga, hT[base + col], acc[i][t], 0, 0, 0);
              }
            }
          }
        }
      }
    }
  }
  // lane (i16, kq) holds D[c' = 16 ct + 4 kq + v][c = 16 t + i16]
  float* line = a.part + (int64_t)blockIdx.x * (a.lmax + 1) * C * C;
#pragma unroll
  for (int i = 0; i < Cfg::LPW; ++i) {
    const int dl = pg + i * Cfg::PG;
    if (dl >= ln) break;
#pragma unroll
    for (int t = 0; t < Cfg::CT; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int r = ct * 16 + 4 * kq + v, c = t * 16 + i16;
        if (r < C && c < C) line[((int64_t)(l0 + dl) * C + r) * C + c] = acc[i][t][v];
      }
  }
}

// grad_W[x] = the sum of its chunks' lines, in order, in 64 bits (zeros without one); blockIdx.y: the expert
__global__ __launch_bounds__(256) void expert_grad_sum_kernel(ExpertGradArgs a, int per, int64_t size, int lines) {
  int at = 0, n = 0;
  for (int x = 0; x <= (int)blockIdx.y; ++x) {
    at += n;
    const int64_t places = a.N * a.k;
    const int64_t lo = min(max((int64_t)a.ptr[x], (int64_t)0), places), hi = min(max((int64_t)a.ptr[x + 1], lo), places);
    n = (int)((hi - lo + per - 1) / per);
  }
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= size) return;
  double s = 0.0;
  for (int j = 0; j < n && at + j < lines; ++j) s += a.part[(at + j) * size + i];
  a.gW[blockIdx.y * size + i] = (float)s;
}

// Places of a chunk: enough that a chunk's line is a small part of what it reads, and about 1024 chunks at most.
static int chunk_places(int64_t N, int C, int lmax, int k, bool bf16) {
  const int64_t K = num_comp(lmax), es = bf16 ? 2 : 4;
  int64_t per = (8 * (int64_t)(lmax + 1) * C / (K * es) + 15) / 16 * 16;
  if (per < 64) per = 64;
  const int64_t fill = (N * k / 1024 + 15) / 16 * 16;
  if (per < fill) per = fill;
  return (int)(per < (1 << 30) ? per : (1 << 30));
}
static int64_t chunks_at_most(int64_t N, int C, int lmax, int X, int k, bool bf16) {
  const int64_t per = chunk_places(N, C, lmax, k, bf16), met = X < N * k ? X : N * k;
  return N * k / per + met;
}

int64_t expert_grad_floats(int64_t N, int C, int lmax, int X, int k, bool bf16) {
  return chunks_at_most(N, C, lmax, X, k, bf16) * (lmax + 1) * C * C;
}

template <class S, int C, bool GATES>
static hipError_t expert_grad_launch(const ExpertGradArgs& a) {
  using Cfg = ExpertGradCfg<S, C, GATES>;
  const int per = chunk_places(a.N, a.C, a.lmax, a.k, a.bf16);
  const int64_t chunks = chunks_at_most(a.N, a.C, a.lmax, a.X, a.k, a.bf16), size = (int64_t)(a.lmax + 1) * C * C;
  static const hipError_t allowed =
      hipFuncSetAttribute(reinterpret_cast<const void*>(expert_grad_kernel<S, C, GATES>),
                          hipFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg::lds_bytes(kMaxPlanes));
  if (allowed != hipSuccess) return allowed;
  if (chunks > 0)
    expert_grad_kernel<S, C, GATES><<<dim3((unsigned)chunks, stretches_of(a.lmax)), dim3(64 * Cfg::WAVES),
                                      Cfg::lds_bytes(a.lmax <= 3 ? num_comp(a.lmax) : kMaxPlanes), a.stream>>>(a, per);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  expert_grad_sum_kernel<<<dim3((unsigned)((size + 255) / 256), a.X), dim3(256), 0, a.stream>>>(a, per, size, (int)chunks);
  return hipGetLastError();
}

template <class S, bool GATES>
static hipError_t expert_grad_c(const ExpertGradArgs& a) {
  switch (a.C) {
    case 8: return expert_grad_launch<S, 8, GATES>(a);
    case 16: return expert_grad_launch<S, 16, GATES>(a);
    case 32: return expert_grad_launch<S, 32, GATES>(a);
    case 64: return expert_grad_launch<S, 64, GATES>(a);
    case 128: return expert_grad_launch<S, 128, GATES>(a);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_expert_grad(const ExpertGradArgs& a) {
  if (a.weight) return a.bf16 ? expert_grad_c<__bf16, true>(a) : expert_grad_c<float, true>(a);
  return a.bf16 ? expert_grad_c<__bf16, false>(a) : expert_grad_c<float, false>(a);
}

}  // namespace eqtp
