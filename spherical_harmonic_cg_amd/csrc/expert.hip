// expert.hip -- the experts' per-degree channel linears,
//   out[n, c', l m] = sum_j weight[n, j] sum_c W[idx[n, j], l, c', c] h[n, c, l m],
// and, with the weights transposed and the output's gradient in h's place, the
// gradients of h and of the gates:
//   grad_weight[n, j] = sum_{c, l m} (W^T g)[n, c, l m] h[n, c, l m].
//
// Bytes per node: its features once in, once out; flops 2 k C^2 K.  Tiles: a
// workgroup takes 16 nodes, a wave of it a group of NP components (16 bytes of a
// channel) and a share of the output channels.  A 16x16 product D[c'][node] of one
// component wants, in lane (node i, k), the component's values of 4 (fp32) or
// 8 (bf16) input channels.  The lane reads those channels' 16-byte runs of
// components, so its registers hold the operands of NP products, in fp32 as
// they are, in bf16 after a transposition within the lane; D holds NP
// components of four output channels of the lane's node, which leave as runs.
//
// The wave goes over the experts that any of the 16 nodes has, in ascending
// order: total += gate D in the lanes of the nodes that have it.  Nodes in an
// order in which neighbours share experts (expert_plan.hip) keep that list short;
// the results do not depend on it.  Weights come from the L2, each once a wave
// and expert.
//
// Four forms:
//   few nodes (up to 512): a thread an output, on the vector ALUs;
//   fp32 rows that fit (expert_f32_kernel): rows go through LDS, operands are
//     read 16 channels at a time.  10k nodes x 64 x 16, one of 10 experts: 37 to
//     41 us, 35 TFLOP/s (bytes 15 us, products 9): 626 tiles on 512 workgroups
//     at a time, and LDS reads between a wave's products;
//   bf16 rows that fit, without the gates' gradient (expert_staged_kernel): rows
//     through LDS, tiles one after the other.  100k nodes x 32 x 16, 2 of 8: 57
//     to 59 us, 3.6 TB/s, where the direct form took 71;
//   the rest (expert_kernel: rows that do not fit, lmax 4 and above, and bf16
//     with the gates' gradient): runs from and to memory, no barriers.  The
//     gradients of h and of the gates of that case: 94 us, 3.3 TB/s; with the
//     gradient's rows through LDS a tile ahead 113, with both tensors' rows
//     through LDS, a tile a workgroup, 115.
// At 128 channels above lmax 0 a wave's operands, weights and sums are more than
// its registers in most forms: 10k nodes, two of 8, forward and gradients of h
// and gates, fp32 at lmax 3 and 4 210 + 270 and 1220 + 1690 us, bf16 100 + 220 and
// 260 + 520.
#include <atomic>
#include <type_traits>

#include "expert_device.hpp"
#include "lane_ops.hpp"

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

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// Smallest of v over the wave; sum over the lanes with the same i16 (both by register moves).
template <int CTRL>
__device__ __forceinline__ int dpp_min(int v) {
  return min(v, __builtin_amdgcn_update_dpp(v, v, CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ int wave_min(int v) {
  v = dpp_min<0x140>(dpp_min<0x141>(dpp_min<0x4E>(dpp_min<0xB1>(v))));
  const auto a = __builtin_amdgcn_permlane16_swap((unsigned)v, (unsigned)v, false, false);
  v = min((int)a[0], (int)a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap((unsigned)v, (unsigned)v, false, false);
  return __builtin_amdgcn_readfirstlane(min((int)b[0], (int)b[1]));
}
__device__ __forceinline__ float rows_sum(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

constexpr int kListed = kMaxTopK / 4;  // places of a node's list that a lane holds (lane (i, k): k, k + 4, ..)

// The experts and gates of the lane's node (kMaxExperts: none).
struct Listed {
  int ex[kListed];
  float gate[kListed];
  __device__ __forceinline__ void load(const ExpertArgs& a, int64_t node, bool live, int kq) {
#pragma unroll
    for (int i = 0; i < kListed; ++i) {
      const int j = kq + 4 * i;
      ex[i] = kMaxExperts;
      gate[i] = 0.0f;
      if (j < a.k && live) {
        const int e = a.idx[node * a.k + j];
        ex[i] = e >= 0 && e < a.X ? e : kMaxExperts;
        gate[i] = a.weight ? a.weight[node * a.k + j] : 1.0f;
      }
    }
  }
  // the tile's lowest expert above e (whole waves)
  __device__ __forceinline__ int after(int e) const {
    int next = kMaxExperts;
#pragma unroll
    for (int i = 0; i < kListed; ++i) next = ex[i] > e ? min(next, ex[i]) : next;
    return wave_min(next);
  }
  // whether the lane's node has e, and its gate
  __device__ __forceinline__ bool has(int e, int i16, float& w) const {
    bool mine = false;
    w = 0.0f;
#pragma unroll
    for (int i = 0; i < kListed; ++i)
      if (ex[i] == e) {
        w += gate[i];
        mine = true;
      }
    w = rows_sum(w);
    const uint64_t b = __ballot(mine);
    return (unsigned)((b | b >> 16 | b >> 32 | b >> 48) >> i16) & 1u;
  }
};

__host__ __device__ constexpr int staged_row(int C, int K, int es) { return C * K * es + 16; }  // bytes, 16 spread the banks
constexpr int kStagedMost = 144 << 10;  // bytes of LDS for whole rows

template <class S, int C, int L>
struct ExpertCfg {
  using Op = Operand<S>;
  static constexpr bool BF16 = std::is_same<S, __bf16>::value;
  static constexpr int K = num_comp(L), NP = planes_at_once(BF16, L), GROUPS = plane_groups(K, NP);
  static constexpr int CT = (C + 15) / 16;                  // tiles of output channels
  static constexpr int CTW = CT < 2 ? CT : (C == 128 && NP == 4 ? 4 : 2), CS = CT / CTW;  // of a wave; shares of waves
  static constexpr int TASKS = GROUPS * CS, WAVES = TASKS < 8 ? TASKS : 8;
  static constexpr int STEP = 4 * Op::N;                    // input channels of a step
  static constexpr int NS = (C + STEP - 1) / STEP;
  static constexpr int ROW = staged_row(C, K, sizeof(S));
  // rows go through LDS where there is a wave for each task and they fit (in fp32, as the output may be)
  static constexpr bool STAGED = TASKS <= 8 && kTile * staged_row(C, K, 4) <= kStagedMost;
  static constexpr bool ALIGNED = K % NP == 0;
  static constexpr int UNITS = C * K * (int)sizeof(S) / 16;  // 16-byte units of a row
  static constexpr int U = (kTile * UNITS + 64 * WAVES - 1) / (64 * WAVES);  // of a tile, for a thread
  typedef typename Op::V B[NS][NP];
  typedef typename Run<S, NP>::R Held[CTW][4];
  typedef f4 Total[CTW][NP];
};

// A wave's operands: B[s][q] holds component q of the group of this node's channels of step s.  row: the node's
// features from the group's first component on.
template <class S, int C, int L, bool ALIGNED>
__device__ __forceinline__ void take_operands(const S* row, int kq, typename ExpertCfg<S, C, L>::B& B) {
  using Cfg = ExpertCfg<S, C, L>;
  using Op = Operand<S>;
  constexpr int K = Cfg::K, NP = Cfg::NP;
  typedef Run<S, NP, ALIGNED> In;
#pragma unroll
  for (int s = 0; s < Cfg::NS; ++s) {
    const int c = s * Cfg::STEP + kq * Op::N;
    if constexpr (NP == 1) {
      B[s][0] = typename Op::V{};
      if (c < C) B[s][0] = *reinterpret_cast<const typename Op::V*>(row + c);  // (rows are 16-byte aligned)
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
}

// The wave's products: total[t][q] = the sum over the tile's experts of the gate times D of output tile ct0 + t and
// component m0 + q.  DOT: also the sums of D times what lies at the same places of `with`, by place of the node's
// list, into dots [kTile][kMaxTopK]; components below dup are another wave's.
template <class S, int C, int L, bool DOT>
__device__ __forceinline__ void multiply(const ExpertArgs& a, const Listed& list, int m0, int dup, int ct0, int i16, int kq,
                                         const typename ExpertCfg<S, C, L>::B& B, const typename ExpertCfg<S, C, L>::Held& held,
                                         typename ExpertCfg<S, C, L>::Total& total, float (*dots)[kMaxTopK]) {
  using Cfg = ExpertCfg<S, C, L>;
  using Op = Operand<S>;
  typedef typename Op::V V;
  constexpr int NP = Cfg::NP, CTW = Cfg::CTW;
#pragma unroll
  for (int t = 0; t < CTW; ++t)
#pragma unroll
    for (int q = 0; q < NP; ++q) total[t][q] = f4{0.f, 0.f, 0.f, 0.f};
  const int lf = degree_of_plane(m0), ll = degree_of_plane(m0 + NP - 1);
  // the wave's weights of one expert and degree
  typedef V Weights[CTW][Cfg::NS];
  auto weights = [&](Weights& wf, int e, int l) {
    const S* We = static_cast<const S*>(a.W) + (int64_t)(e * (L + 1) + l) * (C * C);
#pragma unroll
    for (int t = 0; t < CTW; ++t) {
      const int co = (ct0 + t) * 16 + i16;
#pragma unroll
      for (int s = 0; s < Cfg::NS; ++s) {
        const int c = s * Cfg::STEP + kq * Op::N;
        wf[t][s] = *reinterpret_cast<const V*>(We + (co < C ? co : 0) * C + (c < C ? c : 0));
        if constexpr (C % Cfg::STEP != 0) wf[t][s] = c < C ? wf[t][s] : V{};
      }
    }
  };
  int e = list.after(-1);
  Weights wf;
  weights(wf, min(e, a.X - 1), lf);
  while (e < kMaxExperts) {
    const int then = list.after(e);
    float w;
    const bool has = list.has(e, i16, w);
    float dot = 0.0f;
    for (int l = lf; l <= ll; ++l) {
      // the weights after these are on their way while these are multiplied
      Weights wn;
      weights(wn, l < ll ? e : min(then, a.X - 1), l < ll ? l + 1 : lf);
#pragma unroll
      for (int q = 0; q < NP; ++q) {
        if (degree_of_plane(m0 + q) != l) continue;
#pragma unroll
        for (int t = 0; t < CTW; ++t) {
          f4 acc = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < Cfg::NS; ++s) acc = Op::mul(wf[t][s], B[s][q], acc);
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            total[t][q][v] = has ? fmaf(w, acc[v], total[t][q][v]) : total[t][q][v];
            if constexpr (DOT)
              if (q >= dup && (ct0 + t) * 16 + 4 * kq + v < C) dot = fmaf(acc[v], (float)held[t][v][q], dot);
          }
        }
      }
#pragma unroll
      for (int t = 0; t < CTW; ++t)
#pragma unroll
        for (int s = 0; s < Cfg::NS; ++s) wf[t][s] = wn[t][s];
    }
    if constexpr (DOT) {
      dot = rows_sum(dot);
#pragma unroll
      for (int i = 0; i < kListed; ++i)
        if (list.ex[i] == e) dots[i16][kq + 4 * i] += dot;
    }
    e = then;
  }
}

// What the lane's results meet in the gates' gradient.
template <class S, int C, int L>
__device__ __forceinline__ void take_held(const S* row, int ct0, int kq, typename ExpertCfg<S, C, L>::Held& held) {
  constexpr int K = ExpertCfg<S, C, L>::K, NP = ExpertCfg<S, C, L>::NP, CTW = ExpertCfg<S, C, L>::CTW;
#pragma unroll
  for (int t = 0; t < CTW; ++t)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int c = (ct0 + t) * 16 + 4 * kq + v;
      held[t][v] = Run<S, NP>::load(row + (c < C ? c : 0) * K);
    }
}

// A lane's results of a tile: NP components (K = 1: one) of four channels.
template <class O, int K, int NP, bool ALIGNED>
__device__ __forceinline__ void put_runs(O* o, const f4 (&total)[NP]) {
  if constexpr (NP == 1) {
    typename Run<O, 4, ALIGNED>::R r;
#pragma unroll
    for (int v = 0; v < 4; ++v) r[v] = (O)total[0][v];
    Run<O, 4, ALIGNED>::store(o, r);
  } else {
    constexpr int W = NP * (int)sizeof(O) > 16 ? 16 / (int)sizeof(O) : NP;
#pragma unroll
    for (int v = 0; v < 4; ++v)
#pragma unroll
      for (int q = 0; q < NP; q += W) {
        typename Run<O, W, ALIGNED>::R r;
#pragma unroll
        for (int i = 0; i < W; ++i) r[i] = (O)total[q + i][v];
        Run<O, W, ALIGNED>::store(o + v * K + q, r);
      }
  }
}

template <class S, int C, int L, bool ALIGNED>
__device__ __forceinline__ void put_tiles(const ExpertArgs& a, unsigned char* row, int m0, int ct0, int kq,
                                          const typename ExpertCfg<S, C, L>::Total& total) {
  constexpr int K = ExpertCfg<S, C, L>::K, NP = ExpertCfg<S, C, L>::NP, CTW = ExpertCfg<S, C, L>::CTW;
#pragma unroll
  for (int t = 0; t < CTW; ++t) {
    const int c = (ct0 + t) * 16 + 4 * kq;
    if (c >= C) continue;
    if (a.out_bf16) put_runs<__bf16, K, NP, ALIGNED>(reinterpret_cast<__bf16*>(row) + c * K + m0, total[t]);
    else put_runs<float, K, NP, ALIGNED>(reinterpret_cast<float*>(row) + c * K + m0, total[t]);
  }
}

__device__ __forceinline__ int64_t node_at(const ExpertArgs& a, int64_t p) {
  return a.order ? clamp_index(a.order[p], (int)a.N) : p;
}

// Runs from and to memory: one tile a workgroup, its tasks (group of components, share of the channels) dealt to its waves.
template <class S, int C, int L, bool DOT>
__global__ __launch_bounds__(512) void expert_kernel(ExpertArgs a) {
  using Cfg = ExpertCfg<S, C, L>;
  constexpr int K = Cfg::K, NP = Cfg::NP, CTW = Cfg::CTW, waves = Cfg::WAVES;
  __shared__ float dots[DOT ? 8 : 1][kTile][kMaxTopK];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i16 = lane & 15, kq = lane >> 4;
  const int64_t p0 = (int64_t)blockIdx.x * kTile;
  const int nv = (int)min((int64_t)kTile, a.places - p0);
  const int64_t node = node_at(a, p0 + min(i16, nv - 1));
  Listed list;
  list.load(a, node, i16 < nv, kq);
  if constexpr (DOT) {
    for (int i = lane; i < kTile * kMaxTopK; i += 64) (&dots[wv][0][0])[i] = 0.0f;
    wave_lds_sync();
  }
  for (int task = wv; task < Cfg::TASKS; task += waves) {
    const int g = task / Cfg::CS, ct0 = (task - g * Cfg::CS) * CTW, m0 = group_first(g, K, NP);
    typename Cfg::B B;
    typename Cfg::Held held;
    typename Cfg::Total total;
    take_operands<S, C, L, false>(static_cast<const S*>(a.h) + node * (C * K) + m0, kq, B);
    if constexpr (DOT) take_held<S, C, L>(static_cast<const S*>(a.dot_with) + node * (C * K) + m0, ct0, kq, held);
    multiply<S, C, L, DOT>(a, list, m0, g * NP - m0, ct0, i16, kq, B, held, total, dots[DOT ? wv : 0]);
    if (a.out != nullptr && i16 < nv)
      put_tiles<S, C, L, false>(a, static_cast<unsigned char*>(a.out) + node * (C * K * (a.out_bf16 ? 2 : 4)), m0, ct0, kq, total);
  }
  if constexpr (DOT) {
    __syncthreads();
    for (int i = threadIdx.x; i < nv * a.k; i += blockDim.x) {
      const int r = i / a.k, j = i - r * a.k;
      float v = 0.0f;
      for (int w = 0; w < waves; ++w) v += dots[w][r][j];
      a.gweight[node_at(a, p0 + r) * a.k + j] = v;
    }
  }
}

// Runs from and to LDS, through which a workgroup moves its nodes' whole rows: a task a wave, tile after tile.  While a
// tile is worked on, the next one's rows and lists are on their way into registers, and the order of the one after.
template <class S, int C, int L>
__global__ __launch_bounds__(512, 2) void expert_staged_kernel(ExpertArgs a, int64_t tiles) {
  using Cfg = ExpertCfg<S, C, L>;
  constexpr int K = Cfg::K, NP = Cfg::NP, CTW = Cfg::CTW, waves = Cfg::WAVES, U = Cfg::U, row_in = Cfg::ROW;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  __shared__ int nid[2][kTile];
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i16 = lane & 15, kq = lane >> 4;
  const int row_out = staged_row(C, K, a.out_bf16 ? 2 : 4);
  const int g = wv / Cfg::CS, ct0 = (wv - g * Cfg::CS) * CTW, m0 = group_first(g, K, NP);
  u32x4 rows[U];
  Listed list;
  int ahead = 0;
  auto ask_order = [&](int64_t tile) {  // nodes of a tile (its first one for places past the last)
    if (tid < kTile && tile < tiles) {
      const int64_t p = tile * kTile + tid;
      ahead = (int)node_at(a, p < a.N ? p : tile * kTile);
    }
  };
  auto ask_rows = [&](int64_t tile, const int* n) {
    if (tile >= tiles) return;
    const int nv = (int)min((int64_t)kTile, a.N - tile * kTile);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = tid + j * (64 * waves), r = i / Cfg::UNITS;
      rows[j] = reinterpret_cast<const u32x4*>(a.h)[(int64_t)n[r < nv ? r : 0] * Cfg::UNITS + (i - r * Cfg::UNITS)];
    }
    list.load(a, n[i16], i16 < nv, kq);
  };
  int64_t tile = blockIdx.x;
  ask_order(tile);
  if (tid < kTile) nid[0][tid] = ahead;
  __syncthreads();
  ask_rows(tile, nid[0]);
  ask_order(tile + gridDim.x);
  for (int turn = 0; tile < tiles; tile += gridDim.x, turn ^= 1) {
    const int nv = (int)min((int64_t)kTile, a.N - tile * kTile);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = tid + j * (64 * waves), r = i / Cfg::UNITS;
      if (r < kTile) *reinterpret_cast<u32x4*>(lds + r * row_in + (i - r * Cfg::UNITS) * 16) = rows[j];
    }
    if (tid < kTile) nid[turn ^ 1][tid] = ahead;
    __syncthreads();
    typename Cfg::B B;
    const typename Cfg::Held held = {};  // (of the form with the gates' gradient)
    typename Cfg::Total total;
    take_operands<S, C, L, Cfg::ALIGNED>(reinterpret_cast<const S*>(lds + i16 * row_in) + m0, kq, B);
    const Listed now = list;
    ask_rows(tile + gridDim.x, nid[turn ^ 1]);
    ask_order(tile + 2 * gridDim.x);
    multiply<S, C, L, false>(a, now, m0, 0, ct0, i16, kq, B, held, total, nullptr);
    __syncthreads();  // every wave has its operands: the place takes the results
    put_tiles<S, C, L, Cfg::ALIGNED>(a, lds + i16 * row_out, m0, ct0, kq, total);
    __syncthreads();
    const int out_units = row_out / 16 - 1;
    for (int r = wv; r < nv; r += waves) {
      u32x4* to = reinterpret_cast<u32x4*>(static_cast<unsigned char*>(a.out) + (int64_t)nid[turn][r] * (row_out - 16));
      const u32x4* from = reinterpret_cast<const u32x4*>(lds + r * row_out);
#pragma unroll 4
      for (int i = lane; i < out_units; i += 64) to[i] = from[i];
    }
    __syncthreads();  // the next tile's rows come into the same place
  }
}

// fp32: a tile a workgroup, its rows in LDS; a wave reads its operands from there 16 input channels at a time, just
// before their products.
// ONE: a node has one expert at most and no gate, so a tile of one expert needs no totals beside its products.  Where it
// meets several, each one's products are written to its nodes' rows right away -- a node keeps
// nothing of the other experts', whatever their weights hold -- and the call returns true.
template <int C, int L, bool DOT, bool ONE>
__device__ __forceinline__ bool multiply_steps(const ExpertArgs& a, const Listed& list, const float* row, int m0, int dup, int ct0,
                                               int i16, int kq, const typename ExpertCfg<float, C, L>::Held& held,
                                               typename ExpertCfg<float, C, L>::Total& total, float (*dots)[kMaxTopK],
                                               int64_t p0, int nv) {
  using Cfg = ExpertCfg<float, C, L>;
  typedef Run<float, Cfg::NP, Cfg::ALIGNED> In;
  constexpr int K = Cfg::K, NP = Cfg::NP, CTW = Cfg::CTW, NL = NP == 1 ? 1 : 2;  // (four components: two degrees at most)
  const int lf = degree_of_plane(m0), ll = degree_of_plane(m0 + NP - 1);
  typedef f4 Weights[NL][CTW];
  auto weights = [&](Weights& wf, int e, int s) {
    const int c = s * 16 + kq * 4;
#pragma unroll
    for (int d = 0; d < NL; ++d) {
      const float* We = static_cast<const float*>(a.W) + (int64_t)(e * (L + 1) + (d == 0 ? lf : ll)) * (C * C) + (c < C ? c : 0);
#pragma unroll
      for (int t = 0; t < CTW; ++t) {
        const int co = (ct0 + t) * 16 + i16;
        wf[d][t] = *reinterpret_cast<const f4*>(We + (co < C ? co : 0) * C);
        if constexpr (C % 16 != 0) wf[d][t] = c < C ? wf[d][t] : f4{0.f, 0.f, 0.f, 0.f};
      }
    }
  };
#pragma unroll
  for (int t = 0; t < CTW; ++t)
#pragma unroll
    for (int q = 0; q < NP; ++q) total[t][q] = f4{0.f, 0.f, 0.f, 0.f};
  int e = list.after(-1);
  Weights wf;
  weights(wf, min(e, a.X - 1), 0);
  bool several = false, done = false;
  auto put = [&] {  // (the row's place is looked up again: held over the products, it would take their registers)
    unsigned char* o = static_cast<unsigned char*>(a.out) + node_at(a, p0 + i16) * (C * K * (a.out_bf16 ? 2 : 4));
    put_tiles<float, C, L, Cfg::ALIGNED>(a, o, m0, ct0, kq, total);
  };
  while (e < kMaxExperts) {
    const int then = list.after(e);
    several |= then < kMaxExperts;
    float w;
    const bool has = list.has(e, i16, w);
    typename Cfg::Total apart;
    if constexpr (!ONE) {
#pragma unroll
      for (int t = 0; t < CTW; ++t)
#pragma unroll
        for (int q = 0; q < NP; ++q) apart[t][q] = f4{0.f, 0.f, 0.f, 0.f};
    }
    typename Cfg::Total& into = ONE ? total : apart;
#pragma unroll 2
    for (int s = 0; s < Cfg::NS; ++s) {
      Weights wn;  // on their way while these are multiplied
      weights(wn, s + 1 < Cfg::NS ? e : min(then, a.X - 1), s + 1 < Cfg::NS ? s + 1 : 0);
      const int c = s * 16 + kq * 4;
      float x[4][NP];
      if constexpr (NP == 1) {
        const f4 r = *reinterpret_cast<const f4*>(row + (c < C ? c : 0));
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i][0] = r[i];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const typename In::R r = In::load(row + (c < C ? c + i : 0) * K);
#pragma unroll
          for (int q = 0; q < NP; ++q) x[i][q] = r[q];
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int q = 0; q < NP; ++q) {
          if constexpr (C % 16 != 0) x[i][q] = c < C ? x[i][q] : 0.0f;
        }
#pragma unroll
      for (int q = 0; q < NP; ++q) {
        if (NL == 1 || degree_of_plane(m0 + q) == lf) {
#pragma unroll
          for (int t = 0; t < CTW; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) into[t][q] = __builtin_amdgcn_mfma_f32_16x16x4f32(wf[0][t][i], x[i][q], into[t][q], 0, 0, 0);
        } else {
#pragma unroll
          for (int t = 0; t < CTW; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              into[t][q] = __builtin_amdgcn_mfma_f32_16x16x4f32(wf[NL - 1][t][i], x[i][q], into[t][q], 0, 0, 0);
        }
      }
#pragma unroll
      for (int d = 0; d < NL; ++d)
#pragma unroll
        for (int t = 0; t < CTW; ++t) wf[d][t] = wn[d][t];
    }
    if constexpr (ONE) {
      if (several && has) put();
      done |= has;
      const bool keep = has && !several;
#pragma unroll
      for (int t = 0; t < CTW; ++t)
#pragma unroll
        for (int q = 0; q < NP; ++q)
#pragma unroll
          for (int v = 0; v < 4; ++v) total[t][q][v] = keep ? total[t][q][v] : 0.0f;
    }
    float dot = 0.0f;
#pragma unroll
    for (int t = 0; t < CTW; ++t)
#pragma unroll
      for (int q = 0; q < NP; ++q)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          if constexpr (!ONE) total[t][q][v] = has ? fmaf(w, apart[t][q][v], total[t][q][v]) : total[t][q][v];
          if constexpr (DOT)
            if (q >= dup && (ct0 + t) * 16 + 4 * kq + v < C) dot = fmaf(apart[t][q][v], held[t][v][q], dot);
        }
    if constexpr (DOT) {
      dot = rows_sum(dot);
#pragma unroll
      for (int i = 0; i < kListed; ++i)
        if (list.ex[i] == e) dots[i16][kq + 4 * i] += dot;
    }
    e = then;
  }
  if (ONE && several && !done && i16 < nv) put();  // zeros
  return ONE && several;
}

// (ONE: registers for two workgroups of eight waves a compute unit where the LDS holds two, 37 us; with eight registers
// more and one workgroup 42: 10k nodes of 64 x 16.  With 128 channels a wave has twice the products, which half of the
// registers do not hold: 10k nodes at lmax 1 and 2, 48 and 176 us against 39 and 95.)
constexpr int f32_waves(int C, int L, bool one) {
  return one && C < 128 && 2 * kTile * staged_row(C, num_comp(L), 4) <= (160 << 10) ? 4 : 2;
}

template <int C, int L, bool DOT, bool ONE>
__global__ __launch_bounds__(512, f32_waves(C, L, ONE)) void expert_f32_kernel(ExpertArgs a) {
  using Cfg = ExpertCfg<float, C, L>;
  constexpr int K = Cfg::K, NP = Cfg::NP, CTW = Cfg::CTW, waves = Cfg::WAVES, U = Cfg::U, row_in = Cfg::ROW;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  __shared__ float dots[DOT ? waves : 1][kTile][kMaxTopK];
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i16 = lane & 15, kq = lane >> 4;
  const int g = wv / Cfg::CS, ct0 = (wv - g * Cfg::CS) * CTW, m0 = group_first(g, K, NP);
  const int64_t p0 = (int64_t)blockIdx.x * kTile;
  const int nv = (int)min((int64_t)kTile, a.places - p0);
  {
    u32x4 rows[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = tid + j * (64 * waves), r = i / Cfg::UNITS;
      rows[j] = reinterpret_cast<const u32x4*>(a.h)[node_at(a, p0 + (r < nv ? r : 0)) * Cfg::UNITS + (i - r * Cfg::UNITS)];
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = tid + j * (64 * waves), r = i / Cfg::UNITS;
      if (r < kTile) *reinterpret_cast<u32x4*>(lds + r * row_in + (i - r * Cfg::UNITS) * 16) = rows[j];
    }
  }
  const int64_t node = node_at(a, p0 + min(i16, nv - 1));
  Listed list;
  list.load(a, node, i16 < nv, kq);
  if constexpr (DOT)
    for (int i = lane; i < kTile * kMaxTopK; i += 64) (&dots[wv][0][0])[i] = 0.0f;
  typename Cfg::Held held;
  typename Cfg::Total total;
  if constexpr (DOT) take_held<float, C, L>(static_cast<const float*>(a.dot_with) + node * (C * K) + m0, ct0, kq, held);
  __syncthreads();
  // (whether a tile meets several experts is the same in all its waves)
  if (multiply_steps<C, L, DOT, ONE>(a, list, reinterpret_cast<const float*>(lds + i16 * row_in) + m0, m0, g * NP - m0, ct0, i16, kq,
                                     held, total, dots[DOT ? wv : 0], p0, nv))
    return;
  __syncthreads();  // every wave has read its operands: the place takes the results
  if (a.out != nullptr) {
    const int row_out = staged_row(C, K, a.out_bf16 ? 2 : 4), units = row_out / 16 - 1;
    put_tiles<float, C, L, Cfg::ALIGNED>(a, lds + i16 * row_out, m0, ct0, kq, total);
    __syncthreads();
    for (int r = wv; r < nv; r += waves) {
      u32x4* to = reinterpret_cast<u32x4*>(static_cast<unsigned char*>(a.out) + node_at(a, p0 + r) * (row_out - 16));
      const u32x4* from = reinterpret_cast<const u32x4*>(lds + r * row_out);
#pragma unroll 4
      for (int i = lane; i < units; i += 64) to[i] = from[i];
    }
  }
  if constexpr (DOT)
    for (int i = tid; i < nv * a.k; i += blockDim.x) {
      const int r = i / a.k, j = i - r * a.k;
      float v = 0.0f;
      for (int w = 0; w < waves; ++w) v += dots[w][r][j];
      a.gweight[node_at(a, p0 + r) * a.k + j] = v;
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

// Launches of a tile a workgroup: a launch holds less than 2^32 threads (more wrap round, without an error), so the tiles
// beyond go to further ones, which begin at their own part of the order, or of the rows (a first place held in the
// kernel would cost it registers: 37.6 us instead of 37.2 for 10k x 64 x 16).
constexpr int64_t kLaunchThreads = int64_t(1) << 31;
template <class F>
static hipError_t over_tiles(const ExpertArgs& a, int64_t tiles, int threads, F launch) {
  const int64_t most = kLaunchThreads / threads, row = (int64_t)a.C * num_comp(a.lmax);
  for (int64_t t = 0; t < tiles; t += most) {
    ExpertArgs part = a;
    const int64_t first = t * kTile;
    part.places = a.N - first;
    if (a.order) {
      part.order += first;
    } else {
      auto on = [&](const void* p, int64_t bytes) { return p ? static_cast<const char*>(p) + first * bytes : nullptr; };
      part.N = part.places;
      part.h = on(a.h, row * (a.bf16 ? 2 : 4));
      part.dot_with = on(a.dot_with, row * (a.bf16 ? 2 : 4));
      part.out = const_cast<char*>(on(a.out, row * (a.out_bf16 ? 2 : 4)));
      part.idx = a.idx + first * a.k;
      part.weight = a.weight ? a.weight + first * a.k : nullptr;
      part.gweight = a.gweight ? a.gweight + first * a.k : nullptr;
    }
    launch(part, dim3((unsigned)(tiles - t < most ? tiles - t : most)), dim3(threads));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <class S, int C, int L, bool DOT>
static hipError_t expert_launch(const ExpertArgs& a) {
  using Cfg = ExpertCfg<S, C, L>;
  const int64_t tiles = (a.N + kTile - 1) / kTile;
  if constexpr (Cfg::STAGED && !Cfg::BF16) {
    constexpr int lds = kTile * Cfg::ROW;
    if constexpr (!DOT) {
      if (a.k == 1 && a.weight == nullptr)
        return over_tiles(a, tiles, 64 * Cfg::WAVES, [](const ExpertArgs& part, dim3 grid, dim3 block) {
          expert_f32_kernel<C, L, DOT, true><<<grid, block, lds, part.stream>>>(part);
        });
    }
    return over_tiles(a, tiles, 64 * Cfg::WAVES, [](const ExpertArgs& part, dim3 grid, dim3 block) {
      expert_f32_kernel<C, L, DOT, false><<<grid, block, lds, part.stream>>>(part);
    });
  } else if constexpr (Cfg::STAGED && !DOT) {
    const int bytes = kTile * (a.out_bf16 ? Cfg::ROW : staged_row(C, Cfg::K, 4));
    static std::atomic<int> known[2];  // workgroups that a compute unit holds
    std::atomic<int>& held = known[a.out_bf16];
    int n = held.load(std::memory_order_relaxed);
    if (n == 0) {
      if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, expert_staged_kernel<S, C, L>, 64 * Cfg::WAVES, bytes) != hipSuccess ||
          n < 1)
        n = 1;
      held.store(n, std::memory_order_relaxed);
    }
    // as many workgroups as the card holds, all with the same number of tiles
    const int64_t most = (int64_t)num_cus() * n, each = (tiles + most - 1) / most;
    expert_staged_kernel<S, C, L>
        <<<dim3((unsigned)((tiles + each - 1) / each)), dim3(64 * Cfg::WAVES), bytes, a.stream>>>(a, tiles);
    return hipGetLastError();
  } else {
    return over_tiles(a, tiles, 64 * Cfg::WAVES, [](const ExpertArgs& part, dim3 grid, dim3 block) {
      expert_kernel<S, C, L, DOT><<<grid, block, 0, part.stream>>>(part);
    });
  }
}

template <class S, int L, bool DOT>
static hipError_t expert_c(const ExpertArgs& a) {
  switch (a.C) {
    case 8: return expert_launch<S, 8, L, DOT>(a);
    case 16: return expert_launch<S, 16, L, DOT>(a);
    case 32: return expert_launch<S, 32, L, DOT>(a);
    case 64: return expert_launch<S, 64, L, DOT>(a);
    case 128: return expert_launch<S, 128, L, DOT>(a);
    default: return hipErrorInvalidValue;
  }
}

template <class S, bool DOT>
static hipError_t expert_l(const ExpertArgs& a) {
  switch (a.lmax) {
    case 0: return expert_c<S, 0, DOT>(a);
    case 1: return expert_c<S, 1, DOT>(a);
    case 2: return expert_c<S, 2, DOT>(a);
    case 3: return expert_c<S, 3, DOT>(a);
    case 4: return expert_c<S, 4, DOT>(a);
    case 5: return expert_c<S, 5, DOT>(a);
    case 6: return expert_c<S, 6, DOT>(a);
    default: return hipErrorInvalidValue;
  }
}

// ---------------------------------------------------------------------------
// Few nodes: a tile of 16 columns would multiply mostly nothing, and one wave
// after the other would wait for weights.  A workgroup takes CB output channels of one node, its features in
// LDS; a thread one output component at a time, with vector-ALU products.
// For very few nodes the backward pass reads the weights as they are (no transposed copy).
// ---------------------------------------------------------------------------
constexpr int kFewThreads = 256;

template <class S, bool DOT, bool TRANS>
__global__ __launch_bounds__(kFewThreads) void expert_few_kernel(ExpertArgs a, int CB) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  __shared__ float sums[kFewThreads / 64][kMaxTopK];
  float* h = reinterpret_cast<float*>(lds);  // [C][K]
  const int C = a.C, K = num_comp(a.lmax), tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int64_t n = blockIdx.x;
  const int c0 = blockIdx.y * CB;
  const S* src = static_cast<const S*>(a.h) + n * C * K;
  for (int i = tid; i < C * K; i += kFewThreads) h[i] = (float)src[i];
  if constexpr (DOT)
    for (int i = tid; i < kFewThreads / 64 * kMaxTopK; i += kFewThreads) (&sums[0][0])[i] = 0.0f;
  __syncthreads();
  for (int o0 = 0; o0 < CB * K; o0 += kFewThreads) {
    const bool on = o0 + tid < CB * K;
    const int o = on ? o0 + tid : 0, co = c0 + o / K, m = o - o / K * K, l = degree_of_plane(m);
    float total = 0.0f;
    const float with = DOT && on ? (float)static_cast<const S*>(a.dot_with)[(n * C + co) * K + m] : 0.0f;
    for (int j = 0; j < a.k; ++j) {
      const int e = a.idx[n * a.k + j];
      if (e < 0 || e >= a.X) continue;
      const S* W = static_cast<const S*>(a.W) + (int64_t)(e * (a.lmax + 1) + l) * C * C + (TRANS ? co : co * C);
      float acc = 0.0f;
#pragma unroll 8
      for (int c = 0; c < C; ++c) acc = fmaf((float)W[TRANS ? c * C : c], h[c * K + m], acc);
      total = fmaf(a.weight ? a.weight[n * a.k + j] : 1.0f, acc, total);
      if constexpr (DOT) {
        const float d = lane_sum<64>(on ? acc * with : 0.0f);
        if (lane == 0) sums[wv][j] += d;
      }
    }
    if (on && a.out != nullptr) {
      const int64_t at = (n * C + co) * K + m;
      if (a.out_bf16) static_cast<__bf16*>(a.out)[at] = (__bf16)total;
      else static_cast<float*>(a.out)[at] = total;
    }
  }
  if constexpr (DOT) {
    __syncthreads();
    if (tid < a.k) a.part[(n * a.k + tid) * gridDim.y + blockIdx.y] = (sums[0][tid] + sums[1][tid]) + (sums[2][tid] + sums[3][tid]);
  }
}
// the workgroups' sums of each place, in order
__global__ __launch_bounds__(256) void expert_few_gates_kernel(int64_t places, int parts, const float* __restrict__ part,
                                                               float* __restrict__ gweight) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= places) return;
  float v = 0.0f;
  for (int j = 0; j < parts; ++j) v += part[i * parts + j];
  gweight[i] = v;
}

// Up to 512 nodes.  Forward, us, against the tiles: fp32, two experts of a node: 64 channels at lmax 3, 128, 256 and 512
// nodes 6 / 33, 9 / 29 and 16 / 25 (1024 nodes 28 / 28); 128 channels at lmax 6, 512 nodes 194 / 1052, at lmax 0 12 / 12.
// bf16: 64 channels at lmax 3, one expert 4 / 8, 5 / 8 and 8 / 8, two 6 / 13, 7 / 12 and 12 / 11.  The gradients of h
// and gates are as near.  A node's work here grows with its experts, and the tiles' hardly: from 8 of them on the tiles
// would be faster (fp32, 64 channels at lmax 3, 256 and 512 nodes 27 / 43 and 53 / 44; bf16 19 / 15 and 40 / 16; bf16, 128
// channels at lmax 0, 32 nodes 22 / 10).
static bool expert_few(int64_t N) { return N <= 512; }
// The other way round the weights are read an element at a time (us, gradients of 128 channels at lmax 3: 32 nodes 27, with
// the transposed copy 20; one node 17, 20).
bool expert_as_is(int64_t N) { return N <= 16; }
// a workgroup's outputs: a thread each
static int few_channels(int C, int K) {
  int CB = kFewThreads / K < C ? kFewThreads / K : C;
  while (C % CB != 0) --CB;
  return CB;
}
int64_t expert_gate_floats(int64_t N, int C, int lmax, int k) {
  return expert_few(N) ? N * k * (C / few_channels(C, num_comp(lmax))) : 0;
}

template <class S>
static hipError_t few_launch(const ExpertArgs& a) {
  const int K = num_comp(a.lmax), bytes = a.C * K * 4, CB = few_channels(a.C, K);
  const dim3 grid((unsigned)a.N, a.C / CB);
  if (a.gweight) {
    if (a.as_is) expert_few_kernel<S, true, true><<<grid, dim3(kFewThreads), bytes, a.stream>>>(a, CB);
    else expert_few_kernel<S, true, false><<<grid, dim3(kFewThreads), bytes, a.stream>>>(a, CB);
    expert_few_gates_kernel<<<dim3((unsigned)((a.N * a.k + 255) / 256)), dim3(256), 0, a.stream>>>(a.N * a.k, a.C / CB, a.part,
                                                                                                 a.gweight);
  } else if (a.as_is) {
    expert_few_kernel<S, false, true><<<grid, dim3(kFewThreads), bytes, a.stream>>>(a, CB);
  } else {
    expert_few_kernel<S, false, false><<<grid, dim3(kFewThreads), bytes, a.stream>>>(a, CB);
  }
  return hipGetLastError();
}

hipError_t launch_expert(const ExpertArgs& a) {
  if (a.N == 0) return hipSuccess;
  if (expert_few(a.N)) return a.bf16 ? few_launch<__bf16>(a) : few_launch<float>(a);
  if (a.gweight) return a.bf16 ? expert_l<__bf16, true>(a) : expert_l<float, true>(a);
  return a.bf16 ? expert_l<__bf16, false>(a) : expert_l<float, false>(a);
}

}  // namespace eqtp
