// norm.hip -- layer norm by degree of features [N, C, K] (gradients are in
// norm_grad.hip), with the residual branch's dropout and sum in the same pass:
//   z = x, or residual + keep x / (1 - p);
//   zc = z - [l = 0] mean_c z;  r_l = 1 / sqrt(mean_{c, m of l} zc^2 + eps);
//   out = zc r_l weight[l, c] + [l = 0] bias[c].
//
// Each element is read and written once: bound by HBM where the tensors are
// large, by the vector ALUs (a row's fixed work) where they stay in the 256 MB
// cache or the rows have many degrees and few channels.  A group of T threads
// (8 to 512) holds a node's row of D = C K elements in registers, NV quads of
// four consecutive elements a thread, so the row is read once for both the
// statistics and the result.  Only the first A threads of a group take quads,
// A a multiple of K / gcd(K, 4): quad j of thread t begins at 4 (t + A j), so a
// thread's four slots keep their components m, degrees and factors for every j
// and every row, whatever K is, and loads stay coalesced.  Groups walk over
// the rows, as many as the card holds at once; weights stay in registers.
// Sums by degree are folded over the lanes together (register moves, no LDS),
// then over a group's waves through LDS.
// 100k nodes, 32 channels, lmax 3, with dropout and residual: 146 us (819 MB,
// 5.6 TB/s; a large copy reaches 5.4), vector ALUs busy 29% of it; 10k x 64 x
// 16 to bf16: 13 us (61 MB), 66%; 266k x 64 bf16: 16 us (68 MB), 74%; 5003 x 33
// x 25 with dropout: 19 us (66 MB), 73%; 66k x 10 x 49 bf16: 54 us (129 MB), 96%.
#include "norm_device.hpp"

namespace eqtp {

template <class E, class O, int T, int NV, int KT, bool ADD>
__global__ __launch_bounds__(norm_threads(T)) void norm_kernel(NormArgs a, int A, NormInv inv) {
  constexpr int R = norm_threads(T) / T;  // rows at a time in a workgroup
  __shared__ float red[T > 64 ? 2 * (T / 64) * (kMaxDeg + 1) : 1];
  __shared__ uint8_t nib[ADD ? R * (T * NV + 2) : 1];
  const int C = a.C, D = C * a.K, deg = KT == 0 ? 1 : a.lmax + 1;
  Slots<T, KT> sl(a.K, A);
  const int g = T < 64 ? threadIdx.x / T : __builtin_amdgcn_readfirstlane(threadIdx.x / T);
  const bool tail = KT != 1 && (D & 3) != 0;
  int turn = 0;
  constexpr int G = T < 64 ? T : 64;
  const float inv_mine = 1.0f / (float)(C * (2 * sum8_index<G>() + 1));
  constexpr int NB = KT == 0 ? 4 : 1;  // component 0 fills every slot (K = 1), or at most one of a quad
  float w[NV][4], b[NV][NB];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = sl.channel(q, j);
      w[j][q] = a.weight && sl.on && c < C ? a.weight[sl.l(q) * C + c] : 1.0f;
      if (KT == 0 || q == 0) b[j][KT == 0 ? q : 0] = 0.0f;
      if (a.bias && sl.on && c < C && sl.zero(q)) b[j][KT == 0 ? q : 0] = a.bias[c];
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int q = 0; q < 4; ++q) arrived(w[j][q]);
#pragma unroll
    for (int q = 0; q < NB; ++q) arrived(b[j][q]);
  }
  const bool full = A == T && D == 4 * T * NV;
  DropState ds = {};
  if constexpr (ADD)
    if (a.rng) ds = drop_state(a.rng, a.thr, a.scale);
  for (int64_t n = (int64_t)blockIdx.x * R + g; n < a.N; n += (int64_t)gridDim.x * R) {
    sl.row();
    forget_keys(ds);
    const E* x = (const E*)a.x + n * D;
    float z[NV][4];
    RowQuads<E, NV> rows;
    rows.load(x, sl, A, D);
    if constexpr (ADD) {
      float res[NV][4];
      RowQuads<E, NV> more;
      more.load((const E*)a.residual + n * D, sl, A, D);
      KeepBits<T, KT> kb;
      if (a.rng) kb.begin(ds, n, C, sl.t, nib + g * (T * NV + 2));
      rows.values(sl, A, D, full, tail, z);
      more.values(sl, A, D, full, tail, res);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int i = 4 * (sl.t + A * j);
        if (sl.on && i < D) {
          int c[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) c[q] = min(sl.channel(q, j), C - 1);
          const uint32_t keep = a.rng ? kb.quad(ds, c) : 15u;
#pragma unroll
          for (int q = 0; q < 4; ++q)  // the norm is that of the sum as it is written
            z[j][q] = (float)(E)drop_add<E>(keep, q, z[j][q], a.scale, res[j][q]);
          store4((E*)a.total + n * D + i, D - i, tail, z[j]);
        }
      }
    } else {
      rows.values(sl, A, D, full, tail, z);
    }
    float slot[4] = {};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) slot[q] += z[j][q];
    float mu[1] = {sl.on ? sl.scalars(slot) : 0.0f};
    group_sums<T, 1>(mu, 1, red, turn);
    mu[0] *= inv.v[0];
    float sq[4] = {};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = 4 * (sl.t + A * j);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        // (places past the row hold 0 and stay 0)
        if (KT != 1 || q == 0) z[j][q] -= sl.zero(q) && (KT == 1 ? i < D : i + q < D) ? mu[0] : 0.0f;
        sq[q] = fmaf(z[j][q], z[j][q], sq[q]);
      }
    }
    if (!sl.on)
#pragma unroll
      for (int q = 0; q < 4; ++q) sq[q] = 0.0f;
    float rq[4], r;
    if constexpr (KT == 0) {
      float v[1] = {(sq[0] + sq[1]) + (sq[2] + sq[3])};
      group_sums<T, 1>(v, 1, red, turn);
      r = rsqrtf(fmaf(v[0], inv.v[0], a.eps));
#pragma unroll
      for (int q = 0; q < 4; ++q) rq[q] = r;
    } else {
      float v[8] = {};
      sl.by_degree(sq, deg, v);
      r = rsqrtf(fmaf(group_sums8<T>(v, red, turn), inv_mine, a.eps));
      sl.of_degree(r, 0, rq);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = 4 * (sl.t + A * j);
      float o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        o[q] = fmaf(z[j][q] * rq[q], w[j][q], KT == 0 ? b[j][q % NB] : (KT == 1 ? (q == 0 ? b[j][0] : 0.0f) : (sl.zero(q) ? b[j][0] : 0.0f)));
      if (sl.on) store4((O*)a.out + n * D + i, D - i, tail, o);
    }
    if (a.stats) {
      float* st = a.stats + n * (a.lmax + 2);
      if (sl.t == 0) st[0] = mu[0];
      if constexpr (KT == 0) {
        if (sl.t == 0) st[1] = r;
      } else {
        if (T > 64 ? sl.t < 64 && sl.t % 8 == 0 : sl.t % (T / 8) == 0)  // a thread that has a degree's sum first
          if (const int d = sum8_index<G>(); d < deg) st[1 + d] = r;
      }
    }
  }
}

template <auto kernel, int T>
static hipError_t norm_launch(const NormArgs& a, int A) {
  kernel<<<dim3(norm_grid<kernel, T>(a.N)), dim3(norm_threads(T)), 0, a.stream>>>(a, A, norm_inv(a.C));
  return hipGetLastError();
}

template <class E, class O, int KT, bool ADD>
static hipError_t norm_t(const NormArgs& a) {
  const NormShape s = norm_shape(a.C, a.K);
#define EQTP_NORM(T_, NV_) norm_launch<norm_kernel<E, O, T_, NV_, KT, ADD>, T_>(a, s.A)
  return EQTP_NORM_SHAPES(s, EQTP_NORM);
#undef EQTP_NORM
}

template <class E, class O>
static hipError_t norm_k(const NormArgs& a) {
  if (a.total) return a.K == 1 ? norm_t<E, O, 0, true>(a) : (a.K % 4 == 0 ? norm_t<E, O, 1, true>(a) : norm_t<E, O, 2, true>(a));
  return a.K == 1 ? norm_t<E, O, 0, false>(a) : (a.K % 4 == 0 ? norm_t<E, O, 1, false>(a) : norm_t<E, O, 2, false>(a));
}

hipError_t launch_norm(const NormArgs& a) {
  if (a.N == 0) return hipSuccess;
  if (a.x_bf16) return a.out_bf16 ? norm_k<__bf16, __bf16>(a) : norm_k<__bf16, float>(a);
  return a.out_bf16 ? norm_k<float, __bf16>(a) : norm_k<float, float>(a);
}

}  // namespace eqtp
