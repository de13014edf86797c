// expert.hip -- the experts' per-degree channel linears,
//   out[n, c', l m] = sum_j weight[n, j] sum_c W[idx[n, j], l, c', c] h[n, c, l m],
// and, with the weights transposed and the output's gradient in h's place, the
// gradients of h and of the gates:
//   grad_weight[n, j] = sum_{c, l m} (W^T g)[n, c, l m] h[n, c, l m].
//
// Bytes per node: its features once in, once out; flops 2 k C^2 K.  A workgroup
// takes 16 nodes, a wave of it a group of NP components (16 bytes of a channel)
// and a share of the output channels.  A 16x16 product D[c'][node] of one
// component wants, in lane (node i, k), the component's values of 4 (fp32) or
// 8 (bf16) input channels.  The lane reads those channels' 16-byte runs of
// components, so its registers hold the operands of NP products, in fp32 as
// they are, in bf16 after a transposition within the lane; D holds NP
// components of four output channels of the lane's node, which leave as runs.
// No LDS, no barriers: waves are on their own.
//
// The wave goes over the experts that any of the 16 nodes has, in ascending order: total += gate D in the
// lanes of the nodes that have it.  Nodes in an order in which neighbours share
// experts (expert_plan.hip) keep that list short; the results do not depend on
// it.  Weights come from the L2, each once a wave and expert.
#include <type_traits>

#include "expert_device.hpp"

namespace eqtp {

template <class S>
struct Operand;
template <>
struct Operand<__bf16> {
  typedef bf16x8 V;
  static constexpr int N = 8;  // input channels of a lane and step
  static __device__ __forceinline__ f4 mul(const V& a, const V& b, const f4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Operand<float> {
  typedef f4 V;
  static constexpr int N = 4;
  static __device__ __forceinline__ f4 mul(const V& a, const V& b, f4 c) {
#pragma unroll
    for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[s], c, 0, 0, 0);
    return c;
  }
};

// smallest of v over the wave
__device__ __forceinline__ int wave_min(int v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v = min(v, __shfl_xor(v, o, 64));
  return __builtin_amdgcn_readfirstlane(v);
}

constexpr int kListed = kMaxTopK / 4;  // places of a node's list that a lane holds (lane (i, k): k, k + 4, ..)

template <class S, int C, int NP, int CTW, bool DOT>
__global__ __launch_bounds__(512) void expert_kernel(ExpertArgs a, int groups) {
  using Op = Operand<S>;
  typedef typename Op::V V;
  typedef Run<S, NP> In;
  constexpr int CT = (C + 15) / 16, CS = CT / CTW;
  constexpr int STEP = 4 * Op::N;                       // input channels of a step
  constexpr int NS = (C + STEP - 1) / STEP;
  __shared__ float dots[DOT ? 8 : 1][kTile][kMaxTopK];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int i16 = lane & 15, kq = lane >> 4;
  const int K = num_comp(a.lmax);
  const int64_t p0 = (int64_t)blockIdx.x * kTile;
  const int nv = (int)min((int64_t)kTile, a.N - p0);
  const int64_t p = p0 + min(i16, nv - 1);
  const int64_t node = a.order ? clamp_index(a.order[p], (int)a.N) : p;
  int ex[kListed];
  float gate[kListed];
#pragma unroll
  for (int i = 0; i < kListed; ++i) {
    const int j = kq + 4 * i;
    ex[i] = kMaxExperts;
    gate[i] = 0.0f;
    if (j < a.k && i16 < nv) {
      const int e = a.idx[node * a.k + j];
      ex[i] = e >= 0 && e < a.X ? e : kMaxExperts;
      gate[i] = a.weight ? a.weight[node * a.k + j] : 1.0f;
    }
  }
  if constexpr (DOT) {
    for (int i = lane; i < kTile * kMaxTopK; i += 64) (&dots[wv][0][0])[i] = 0.0f;
    wave_lds_sync();
  }

  for (int task = wv; task < groups * CS; task += waves) {
    const int g = task / CS, ct0 = (task - g * CS) * CTW;
    const int m0 = group_first(g, K, NP), dup = g * NP - m0;  // components below dup are the group before's, too
    // operands: B[s][p] holds this node's component m0 + p of the lane's channels of step s
    V B[NS][NP];
    const S* row = static_cast<const S*>(a.h) + node * C * K + m0;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int c = s * STEP + kq * Op::N;
      if constexpr (NP == 1) {
        B[s][0] = V{};
        if (c < C) B[s][0] = *reinterpret_cast<const V*>(row + c);
      } else {
        typename In::R r[Op::N];
#pragma unroll
        for (int i = 0; i < Op::N; ++i) r[i] = In::load(row + (c < C ? c + i : 0) * K);
#pragma unroll
        for (int q = 0; q < NP; ++q)
#pragma unroll
          for (int i = 0; i < Op::N; ++i) B[s][q][i] = c < C ? r[i][q] : (S)0.0f;
      }
    }
    f4 total[CTW][NP];
#pragma unroll
    for (int t = 0; t < CTW; ++t)
#pragma unroll
      for (int q = 0; q < NP; ++q) total[t][q] = f4{0.f, 0.f, 0.f, 0.f};
    // (the gates' gradient: what the lane's results meet)
    typename In::R held[DOT ? CTW : 1][4];
    if constexpr (DOT) {
      const S* with = static_cast<const S*>(a.dot_with) + node * C * K + m0;
#pragma unroll
      for (int t = 0; t < CTW; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int c = (ct0 + t) * 16 + 4 * kq + v;
          held[t][v] = In::load(with + (c < C ? c : 0) * K);
        }
    }
    const int lf = degree_of_plane(m0), ll = degree_of_plane(m0 + NP - 1);
    // a tile's weights of one expert and degree
    auto weights = [&](V(&wf)[NS], int e, int t, int l) {
      const int co = (ct0 + t) * 16 + i16;
      const S* wr = static_cast<const S*>(a.W) + (((int64_t)e * (a.lmax + 1) + l) * C + (co < C ? co : 0)) * C;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int c = s * STEP + kq * Op::N;
        wf[s] = *reinterpret_cast<const V*>(wr + (c < C ? c : 0));
        if constexpr (C % STEP != 0) wf[s] = c < C ? wf[s] : V{};
      }
    };
    auto after = [&](int e) {  // the next expert of the tile
      int next = kMaxExperts;
#pragma unroll
      for (int i = 0; i < kListed; ++i) next = ex[i] > e ? min(next, ex[i]) : next;
      return wave_min(next);
    };
    int e = after(-1);
    V wf[NS];
    weights(wf, min(e, a.X - 1), 0, lf);
    while (e < kMaxExperts) {
      const int then = after(e);
      float w = 0.0f;
      int has = 0;
#pragma unroll
      for (int i = 0; i < kListed; ++i)
        if (ex[i] == e) {
          w += gate[i];
          has = 1;
        }
      w += __shfl_xor(w, 16, 64);
      w += __shfl_xor(w, 32, 64);
      has |= __shfl_xor(has, 16, 64);
      has |= __shfl_xor(has, 32, 64);
      float dot = 0.0f;
#pragma unroll
      for (int t = 0; t < CTW; ++t) {
        for (int l = lf; l <= ll; ++l) {
          // the weights after these are on their way while these are multiplied
          const bool same = l < ll;
          V wn[NS];
          weights(wn, same || t + 1 < CTW ? e : min(then, a.X - 1), same ? t : (t + 1 < CTW ? t + 1 : 0), same ? l + 1 : lf);
#pragma unroll
          for (int q = 0; q < NP; ++q) {
            if (degree_of_plane(m0 + q) != l) continue;
            f4 acc = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < NS; ++s) acc = Op::mul(wf[s], B[s][q], acc);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              total[t][q][v] = has ? fmaf(w, acc[v], total[t][q][v]) : total[t][q][v];
              if constexpr (DOT)
                if (q >= dup && (ct0 + t) * 16 + 4 * kq + v < C) dot = fmaf(acc[v], (float)held[t][v][q], dot);
            }
          }
#pragma unroll
          for (int s = 0; s < NS; ++s) wf[s] = wn[s];
        }
      }
      if constexpr (DOT) {
        dot += __shfl_xor(dot, 16, 64);
        dot += __shfl_xor(dot, 32, 64);
#pragma unroll
        for (int i = 0; i < kListed; ++i)
          if (ex[i] == e) dots[wv][i16][kq + 4 * i] += dot;
      }
      e = then;
    }
    if (a.out == nullptr || i16 >= nv) continue;
#pragma unroll
    for (int t = 0; t < CTW; ++t) {
      const int c = (ct0 + t) * 16 + 4 * kq;
      if (c >= C) continue;
      const int64_t at = (node * C + c) * K + m0;
      if constexpr (NP == 1) {
        if (a.out_bf16) {
          Run<__bf16, 4>::R o;
#pragma unroll
          for (int v = 0; v < 4; ++v) o[v] = (__bf16)total[t][0][v];
          Run<__bf16, 4>::store(static_cast<__bf16*>(a.out) + at, o);
        } else {
          Run<float, 4>::store(static_cast<float*>(a.out) + at, total[t][0]);
        }
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          if (a.out_bf16) {
            typename Run<__bf16, NP>::R o;
#pragma unroll
            for (int q = 0; q < NP; ++q) o[q] = (__bf16)total[t][q][v];
            Run<__bf16, NP>::store(static_cast<__bf16*>(a.out) + at + v * K, o);
          } else {
#pragma unroll
            for (int q = 0; q < NP; q += 4)
              Run<float, 4>::store(static_cast<float*>(a.out) + at + v * K + q,
                                   f4{total[t][q][v], total[t][q + 1][v], total[t][q + 2][v], total[t][q + 3][v]});
          }
        }
      }
    }
  }
  if constexpr (DOT) {
    __syncthreads();
    for (int i = threadIdx.x; i < nv * a.k; i += blockDim.x) {
      const int r = i / a.k, j = i - r * a.k;
      float v = 0.0f;
      for (int w = 0; w < waves; ++w) v += dots[w][r][j];
      const int64_t n = a.order ? clamp_index(a.order[p0 + r], (int)a.N) : p0 + r;
      a.gweight[n * a.k + j] = v;
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

template <class S, int C, int NP, int CTW, bool DOT>
static hipError_t expert_launch(const ExpertArgs& a) {
  const int groups = plane_groups(num_comp(a.lmax), NP), tasks = groups * ((C + 15) / 16 / CTW);
  expert_kernel<S, C, NP, CTW, DOT><<<dim3((unsigned)((a.N + kTile - 1) / kTile)), dim3(64 * (tasks < 8 ? tasks : 8)), 0,
                                      a.stream>>>(a, groups);
  return hipGetLastError();
}

// Output tiles of a wave: all of them up to C = 64, so that a tile's features are read once; fewer where the totals
// would not leave two waves' registers.
template <class S, int C, int NP, bool DOT>
static hipError_t expert_ctw(const ExpertArgs& a) {
  constexpr int CT = (C + 15) / 16, MOST = 2;
  return expert_launch<S, C, NP, (CT < MOST ? CT : MOST), DOT>(a);
}

template <class S, int NP, bool DOT>
static hipError_t expert_c(const ExpertArgs& a) {
  switch (a.C) {
    case 8: return expert_ctw<S, 8, NP, DOT>(a);
    case 16: return expert_ctw<S, 16, NP, DOT>(a);
    case 32: return expert_ctw<S, 32, NP, DOT>(a);
    case 64: return expert_ctw<S, 64, NP, DOT>(a);
    case 128: return expert_ctw<S, 128, NP, DOT>(a);
    default: return hipErrorInvalidValue;
  }
}

template <bool DOT>
static hipError_t expert_np(const ExpertArgs& a) {
  const int np = planes_at_once(a.bf16, a.lmax);
  if (a.bf16) return np == 1 ? expert_c<__bf16, 1, DOT>(a) : (np == 4 ? expert_c<__bf16, 4, DOT>(a) : expert_c<__bf16, 8, DOT>(a));
  return np == 1 ? expert_c<float, 1, DOT>(a) : expert_c<float, 4, DOT>(a);
}

hipError_t launch_expert(const ExpertArgs& a) {
  if (a.N == 0) return hipSuccess;
  return a.gweight ? expert_np<true>(a) : expert_np<false>(a);
}

}  // namespace eqtp
