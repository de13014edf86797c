// expert.hip -- the experts' per-degree channel linears,
//   out[n, c', l m] = sum_j weight[n, j] sum_c W[idx[n, j], l, c', c] h[n, c, l m],
// and, with the weights transposed and the output's gradient in h's place, the
// gradients of h and of the gates:
//   grad_weight[n, j] = sum_{c, l m} (W^T g)[n, c, l m] h[n, c, l m].
//
// Bytes per node: its features once in, once out; flops 2 k C^2 K.  A workgroup
// takes 16 nodes, stages their features in LDS as planes [component][node][channel] and goes over the experts
// that any of the 16 has: for each, 16x16 products D[c'][node] on the matrix
// cores (bf16 operands, or fp32), then total += gate D in the lanes of the
// nodes that have it.  Nodes in an order in which neighbours share experts
// (expert_plan.hip) keep that list short; the results do not depend on the
// order: a node adds its experts in ascending order whatever the others have.
// A wave keeps a tile of 16 output channels, so each weight is read once a
// workgroup, from the L2, straight into the operand's registers.  Totals leave
// through LDS in the features' layout.
#include <type_traits>

#include "expert_device.hpp"

namespace eqtp {

template <class S, int C>
struct ExpertCfg {
  static constexpr bool BF16 = std::is_same<S, __bf16>::value;
  static constexpr int PAD = BF16 ? 8 : 4;
  static constexpr int RS = C + PAD;                       // row stride of a plane (elements)
  static constexpr int ES = (int)sizeof(S);
  static constexpr int PLANE = kTile * RS + 16 / ES;       // 16 rows and 16 bytes, which spread the planes over the banks
  static constexpr int WAVES = expert_threads(C) / 64;
  static constexpr int CT = (C + 15) / 16;                 // tiles of output channels
  static constexpr int PG = WAVES / CT > 0 ? WAVES / CT : 1;  // waves that share a tile of channels: parts of the planes
  static constexpr int PPW = kMaxPlanes / PG;              // planes of a wave at most
  static constexpr int KS = BF16 ? (C + 31) / 32 : (C + 15) / 16;  // steps over the input channels
  static size_t lds_bytes(int planes) {
    const size_t in = (size_t)planes * PLANE * ES, out = (size_t)kTile * (C * planes + 4) * 4;
    return in > out ? in : out;
  }
};

template <class S>
struct Operand;
template <>
struct Operand<__bf16> {
  typedef bf16x8 V;
  static constexpr int N = 8;
  static __device__ __forceinline__ V zero() { return V{}; }
  static __device__ __forceinline__ f4 mul(const V& a, const V& b, const f4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Operand<float> {
  typedef f4 V;
  static constexpr int N = 4;
  static __device__ __forceinline__ V zero() { return V{0.f, 0.f, 0.f, 0.f}; }
  static __device__ __forceinline__ f4 mul(const V& a, const V& b, f4 c) {
#pragma unroll
    for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[s], c, 0, 0, 0);
    return c;
  }
};

template <class S, int C, bool DOT>
__global__ __launch_bounds__(expert_threads(C)) void expert_kernel(ExpertArgs a) {
  using Cfg = ExpertCfg<S, C>;
  using Op = Operand<S>;
  typedef typename Op::V V;
  constexpr int TH = 64 * Cfg::WAVES;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  __shared__ int node[kTile];
  __shared__ int expert[kTile][kMaxTopK];
  __shared__ float gate[kTile][kMaxTopK];
  __shared__ unsigned met[kMaxExperts / 32];
  __shared__ float dots[DOT ? Cfg::WAVES : 1][kTile][kMaxTopK];
  S* hT = reinterpret_cast<S*>(lds);
  float* ot = reinterpret_cast<float*>(lds);
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i16 = lane & 15, kq = lane >> 4;
  const int ct = wv % Cfg::CT, pg = wv / Cfg::CT;
  const int K = num_comp(a.lmax);
  const int64_t p0 = (int64_t)blockIdx.x * kTile;
  const int nv = (int)min((int64_t)kTile, a.N - p0);

  // the nodes of the tile, their experts and gates, and the experts that any of them has
  if (tid < kTile) {
    const int64_t p = p0 + tid;
    node[tid] = tid < nv ? (a.order ? clamp_index(a.order[p], (int)a.N) : (int)p) : -1;
  }
  if (tid < kMaxExperts / 32) met[tid] = 0u;
  if constexpr (DOT)
    for (int i = tid; i < Cfg::WAVES * kTile * kMaxTopK; i += TH) (&dots[0][0][0])[i] = 0.0f;
  __syncthreads();
  for (int i = tid; i < kTile * a.k; i += TH) {
    const int r = i / a.k, j = i - r * a.k;
    int e = -1;
    float w = 0.0f;
    if (r < nv) {
      const int64_t s = (int64_t)node[r] * a.k + j;
      e = a.idx[s];
      if (e < 0 || e >= a.X) e = -1;
      w = a.weight ? a.weight[s] : 1.0f;
      if (e >= 0) atomicOr(&met[e >> 5], 1u << (e & 31));
    }
    expert[r][j] = e;
    gate[r][j] = w;
  }

  for (int st = 0; st < stretches_of(a.lmax); ++st) {
    const int m0 = stretch_first(st), np = stretch_planes(st, a.lmax);
    __syncthreads();
    // stage the features: (node, channel) rows of np components
    for (int i = tid; i < kTile * C; i += TH) {
      const int r = i / C, c = i - r * C;
      const S* src = static_cast<const S*>(a.h) + ((int64_t)(r < nv ? node[r] : 0) * C + c) * K + m0;
      for (int m = 0; m < np; ++m) hT[m * Cfg::PLANE + r * Cfg::RS + c] = r < nv ? src[m] : (S)0.0f;
    }
    __syncthreads();
    const int share = (np + Cfg::PG - 1) / Cfg::PG;
    const int first = pg * share, mine = min(share, np - first);  // this wave's planes
    f4 total[Cfg::PPW];
    float held[DOT ? Cfg::PPW : 1][4];
#pragma unroll
    for (int i = 0; i < Cfg::PPW; ++i) {
      total[i] = f4{0.f, 0.f, 0.f, 0.f};
      if constexpr (DOT) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int c = ct * 16 + 4 * kq + v;
          held[i][v] = 0.0f;
          if (i < mine && c < C && node[i16] >= 0)
            held[i][v] = (float)static_cast<const S*>(a.dot_with)[((int64_t)node[i16] * C + c) * K + m0 + first + i];
        }
      }
    }
    const int co = ct * 16 + i16;
    for (int word = 0; word < (a.X + 31) / 32; ++word) {
      unsigned bits = __builtin_amdgcn_readfirstlane(met[word]);
      while (bits) {
        const int e = word * 32 + __builtin_ctz(bits);
        bits &= bits - 1;
        float g = 0.0f;
        bool has = false;
        for (int j = 0; j < a.k; ++j)
          if (expert[i16][j] == e) {
            g += gate[i16][j];
            has = true;
          }
        const S* We = static_cast<const S*>(a.W) + ((int64_t)e * (a.lmax + 1)) * C * C;
        V wf[Cfg::KS];
        float dot = 0.0f;
        int have = -1;
#pragma unroll
        for (int i = 0; i < Cfg::PPW; ++i) {
          if (i >= mine) break;
          const int l = degree_of_plane(m0 + first + i);
          if (l != have) {
            have = l;
#pragma unroll
            for (int s = 0; s < Cfg::KS; ++s) {
              const int c = (s * 4 + kq) * Op::N;
              wf[s] = c < C && co < C ? *reinterpret_cast<const V*>(We + ((int64_t)l * C + co) * C + c) : Op::zero();
            }
          }
          const S* row = hT + (first + i) * Cfg::PLANE + i16 * Cfg::RS;
          f4 acc = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < Cfg::KS; ++s) {
            const int c = (s * 4 + kq) * Op::N;
            const V b = c < C ? *reinterpret_cast<const V*>(row + c) : Op::zero();
            acc = Op::mul(wf[s], b, acc);
          }
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            total[i][v] = has ? fmaf(g, acc[v], total[i][v]) : total[i][v];
            if constexpr (DOT) dot = fmaf(acc[v], held[i][v], dot);
          }
        }
        if constexpr (DOT) {
          dot += __shfl_xor(dot, 16, 64);
          dot += __shfl_xor(dot, 32, 64);
          if (kq == 0 && has)
            for (int j = 0; j < a.k; ++j)
              if (expert[i16][j] == e) dots[wv][i16][j] += dot;
        }
      }
    }
    if (a.out == nullptr) continue;
    __syncthreads();  // the features are dead: the place holds the output [node][channel][plane] (stride of a node padded)
    const int NS = C * np + 4;
#pragma unroll
    for (int i = 0; i < Cfg::PPW; ++i) {
      if (i >= mine) break;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int c = ct * 16 + 4 * kq + v;
        if (c < C) ot[i16 * NS + c * np + first + i] = total[i][v];
      }
    }
    __syncthreads();
    for (int i = tid; i < nv * C * np; i += TH) {
      const int r = i / (C * np), at = i - r * (C * np), c = at / np, m = at - c * np;
      const int64_t o = ((int64_t)node[r] * C + c) * K + m0 + m;
      const float v = ot[r * NS + at];
      if (a.out_bf16) static_cast<__bf16*>(a.out)[o] = (__bf16)v;
      else static_cast<float*>(a.out)[o] = v;
    }
  }
  if constexpr (DOT) {
    __syncthreads();
    for (int i = tid; i < nv * a.k; i += TH) {
      const int r = i / a.k, j = i - r * a.k;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < Cfg::WAVES; ++w) v += dots[w][r][j];
      a.gweight[(int64_t)node[r] * a.k + j] = v;
    }
  }
}

// WT[i][c][c'] = W[i][c'][c] for each of `matrices` C x C matrices
template <class S>
__global__ __launch_bounds__(256) void transpose_weights_kernel(int64_t matrices, int C, const S* __restrict__ W,
                                                                S* __restrict__ WT) {
  __shared__ S t[16][17];
  const int x = threadIdx.x & 15, y = threadIdx.x >> 4, tiles = (C + 15) / 16;
  for (int64_t b = blockIdx.x; b < matrices * tiles * tiles; b += gridDim.x) {
    const int64_t i = b / (tiles * tiles);
    const int q = (int)(b - i * tiles * tiles), r0 = q / tiles * 16, c0 = q % tiles * 16;
    if (r0 + y < C && c0 + x < C) t[y][x] = W[(i * C + r0 + y) * C + c0 + x];
    __syncthreads();
    if (c0 + y < C && r0 + x < C) WT[(i * C + c0 + y) * C + r0 + x] = t[x][y];
    __syncthreads();
  }
}

hipError_t launch_transpose_weights(int64_t matrices, int C, bool bf16, const void* W, void* WT, hipStream_t stream) {
  const int tiles = (C + 15) / 16;
  const int64_t want = matrices * tiles * tiles;
  const dim3 grid((unsigned)(want < 65536 ? want : 65536));
  if (bf16)
    transpose_weights_kernel<uint16_t><<<grid, dim3(256), 0, stream>>>(matrices, C, (const uint16_t*)W, (uint16_t*)WT);
  else
    transpose_weights_kernel<uint32_t><<<grid, dim3(256), 0, stream>>>(matrices, C, (const uint32_t*)W, (uint32_t*)WT);
  return hipGetLastError();
}

template <class S, int C, bool DOT>
static hipError_t expert_launch(const ExpertArgs& a) {
  using Cfg = ExpertCfg<S, C>;
  const size_t bytes = Cfg::lds_bytes(a.lmax <= 3 ? num_comp(a.lmax) : kMaxPlanes);
  static const hipError_t allowed =  // more than 64 KB of LDS has to be asked for, once a kernel
      hipFuncSetAttribute(reinterpret_cast<const void*>(expert_kernel<S, C, DOT>),
                          hipFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg::lds_bytes(kMaxPlanes));
  if (allowed != hipSuccess) return allowed;
  expert_kernel<S, C, DOT><<<dim3((unsigned)((a.N + kTile - 1) / kTile)), dim3(64 * Cfg::WAVES), bytes, a.stream>>>(a);
  return hipGetLastError();
}

template <class S, bool DOT>
static hipError_t expert_c(const ExpertArgs& a) {
  switch (a.C) {
    case 8: return expert_launch<S, 8, DOT>(a);
    case 16: return expert_launch<S, 16, DOT>(a);
    case 32: return expert_launch<S, 32, DOT>(a);
    case 64: return expert_launch<S, 64, DOT>(a);
    case 128: return expert_launch<S, 128, DOT>(a);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_expert(const ExpertArgs& a) {
  if (a.N == 0) return hipSuccess;
  if (a.gweight) return a.bf16 ? expert_c<__bf16, true>(a) : expert_c<float, true>(a);
  return a.bf16 ? expert_c<__bf16, false>(a) : expert_c<float, false>(a);
}

}  // namespace eqtp
