// norm_grad.hip -- gradients of the layer norm by degree (and of the residual
// sum and dropout before it):
//   a = weight g,  zhat = zc r_l,
//   gz = r_l (a - [l = 0] mean_c a - zhat mean_l(a zhat)) (+ grad_total),
//   gx = keep gz / (1 - p),  gweight[l, c] = sum g zhat,  gbias[c] = sum g[0].
// Bound as the forward pass is: z, g (and grad_total) are read once, the
// gradients written once.  Rows lie in groups of threads as there.  The sums
// over nodes are kept at each thread's own places while its group walks over
// the rows; at the end a workgroup adds its groups and the components of a
// degree through LDS, in a fixed order, into its line of part
// [workgroups][(lmax+2) C], and a second kernel adds the lines.  Both add in
// 64 bits and round once: at 1000 nodes of 32 x 16 the results are 6e-8 off
// the exact sums (fp32 additions one after the other: 1.9e-7; a pairwise fp32
// sum: 1.3e-7), in the same time.  A thread's own sum, over the rows of its
// group, is fp32.
// 100k nodes, 32 channels, lmax 3, five tensors of 205 MB: 192 us (5.3 TB/s)
// and 5 for the lines, vector ALUs busy 26%; 266k rows of 64 bf16: 23 and 4.3
// us (102 MB), 71%; 66k x 10 x 49 bf16: 70 us (194 MB), 90%.  Dropout makes
// kernels of its own: its words cost registers, and with them waves (bf16 rows
// of 64: 34 us with, 24 without).
#include "norm_device.hpp"

namespace eqtp {

template <class E, class O, int T, int NV, int KT, bool DROP>
__global__ __launch_bounds__(norm_threads(T)) void norm_grad_kernel(NormGradArgs a, int A, NormInv inv, float* part) {
  constexpr int TH = norm_threads(T), R = TH / T;
  constexpr bool HOLD = NV < 9;  // weights in registers
  __shared__ float red[T > 64 ? 2 * (T / 64) * (kMaxDeg + 1) : 1];
  __shared__ uint8_t nib[DROP ? R * (T * NV + 2) : 1];
  __shared__ float pos[R * T * NV * 4];  // per group: a value for each place of a row
  const int C = a.C, D = C * a.K, deg = KT == 0 ? 1 : a.lmax + 1;
  Slots<T, KT> sl(a.K, A);
  const int g = T < 64 ? threadIdx.x / T : __builtin_amdgcn_readfirstlane(threadIdx.x / T);
  const bool tail = KT != 1 && (D & 3) != 0;
  int turn = 0;
  constexpr int G = T < 64 ? T : 64;
  const int place = sum8_index<G>();  // of eight sums: the scalars', then the degrees'
  const float inv_mine = 1.0f / (float)(C * (place == 0 ? 1 : 2 * place - 1));
  constexpr int NB = KT == 0 ? 4 : 1;  // component 0 fills every slot (K = 1), or at most one of a quad
  float w[NV][4], aw[NV][4] = {}, ab[NV][NB] = {};
  auto weights = [&]() {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = sl.channel(q, j);
        w[j][q] = a.weight && sl.on && c < C ? a.weight[sl.l(q) * C + c] : 1.0f;
      }
  };
  if constexpr (HOLD) {
    weights();
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) arrived(w[j][q]);
  }
  const bool full = A == T && D == 4 * T * NV;
  DropState ds = {};
  if constexpr (DROP) ds = drop_state(a.rng, a.thr, a.scale);
  for (int64_t n = (int64_t)blockIdx.x * R + g; n < a.N; n += (int64_t)gridDim.x * R) {
    sl.row();
    if constexpr (DROP) forget_keys(ds);
    if constexpr (!HOLD) weights();
    float z[NV][4], go[NV][4], gt[NV][4] = {};
    RowQuads<E, NV> rz, rt;
    RowQuads<O, NV> rg;
    rz.load((const E*)a.total + n * D, sl, A, D);
    rg.load((const O*)a.gout + n * D, sl, A, D);
    if (a.gtotal) rt.load((const E*)a.gtotal + n * D, sl, A, D);
    const float* st = a.stats + n * (a.lmax + 2);
    const float mu = st[0];
    float rq[4], sq[4] = {}, slot[4] = {}, v[8] = {};
#pragma unroll
    for (int q = 0; q < 4; ++q) rq[q] = st[1 + sl.l(q)];
    rz.values(sl, A, D, full, tail, z);
    rg.values(sl, A, D, full, tail, go);
    if (a.gtotal) rt.values(sl, A, D, full, tail, gt);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = 4 * (sl.t + A * j);
      float av[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        // (places past the row hold 0 and stay 0)
        if (KT != 1 || q == 0) z[j][q] -= sl.zero(q) && (KT == 1 ? i < D : i + q < D) ? mu : 0.0f;
        z[j][q] *= rq[q];
        aw[j][q] = fmaf(go[j][q], z[j][q], aw[j][q]);
        av[q] = go[j][q] * w[j][q];
        sq[q] = fmaf(av[q], z[j][q], sq[q]);
        slot[q] += av[q];
      }
      if constexpr (KT == 0) {
#pragma unroll
        for (int q = 0; q < 4; ++q) ab[j][q] += go[j][q];
      } else {
        ab[j][0] += KT == 1 ? go[j][0] : sl.scalars(go[j]);
      }
    }
    if (a.gres || a.gx) {
      if (!sl.on)
#pragma unroll
        for (int q = 0; q < 4; ++q) sq[q] = 0.0f;
      v[0] = sl.on ? sl.scalars(slot) : 0.0f;
      float am, mq[4];
      if constexpr (KT == 0) {
        float two[2] = {v[0], (sq[0] + sq[1]) + (sq[2] + sq[3])};
        group_sums<T, 2>(two, 2, red, turn);
        am = two[0] * inv.v[0];
#pragma unroll
        for (int q = 0; q < 4; ++q) mq[q] = two[1] * inv.v[0];
      } else {
        sl.by_degree(sq, deg, v + 1);
        const float mean = group_sums8<T>(v, red, turn) * inv_mine;
        am = sum8_of<G>(mean, 0);
        sl.of_degree(mean, 1, mq);
      }
      KeepBits<T, KT> kb;
      if constexpr (DROP) kb.begin(ds, n, C, sl.t, nib + g * (T * NV + 2));
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int i = 4 * (sl.t + A * j);
        if (sl.on && i < D) {
          float gz[4];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            gz[q] = fmaf(rq[q], (go[j][q] * w[j][q] - (sl.zero(q) ? am : 0.0f)) - z[j][q] * mq[q], gt[j][q]);
          if (a.gres) store4((E*)a.gres + n * D + i, D - i, tail, gz);
          if (a.gx) {
            if constexpr (DROP) {
              int c[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) c[q] = min(sl.channel(q, j), C - 1);
              const uint32_t keep = kb.quad(ds, c);
#pragma unroll
              for (int q = 0; q < 4; ++q) gz[q] = drop(keep, q, gz[q], a.scale);
            }
            store4((E*)a.gx + n * D + i, D - i, tail, gz);
          }
        }
      }
    }
  }
  if (part == nullptr) return;
  const int cols = (a.lmax + 2) * C, wcols = cols - C;
  part += (int64_t)blockIdx.x * cols;
  float* mine = pos + g * (T * NV * 4);
  if (sl.on)
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) mine[4 * (sl.t + A * j) + q] = aw[j][q];
  __syncthreads();
  for (int col = threadIdx.x; col < wcols; col += TH) {
    const int l = col / C, c = col - l * C;
    double s = 0.0;
    for (int k = 0; k < R; ++k)
      for (int m = l * l; m < (l + 1) * (l + 1); ++m) s += pos[k * (T * NV * 4) + c * a.K + m];
    part[col] = (float)s;
  }
  __syncthreads();
  if (sl.on)
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (sl.zero(q) && sl.channel(q, j) < C) mine[sl.channel(q, j)] = ab[j][KT == 0 ? q : 0];
  __syncthreads();
  for (int c = threadIdx.x; c < C; c += TH) {
    double s = 0.0;
    for (int k = 0; k < R; ++k) s += pos[k * (T * NV * 4) + c];
    part[wcols + c] = (float)s;
  }
}

// Sums of the lines of part: 16 columns and 64 stretches of lines a workgroup.
__global__ __launch_bounds__(1024) void norm_weight_sum_kernel(int cols, int wcols, int parts,
                                                               const float* __restrict__ part, float* gw, float* gb) {
  __shared__ double red[64][17];
  const int cc = threadIdx.x & 15, k = threadIdx.x >> 4, col = blockIdx.x * 16 + cc;
  double s = 0.0;
  if (col < cols) {
#pragma unroll 8
    for (int p = k; p < parts; p += 64) s += part[(int64_t)p * cols + col];
  }
  red[k][cc] = s;
  __syncthreads();
  if (k == 0 && col < cols) {
    s = 0.0;
#pragma unroll
    for (int i = 0; i < 64; ++i) s += red[i][cc];
    if (col < wcols) {
      if (gw) gw[col] = (float)s;
    } else if (gb) {
      gb[col - wcols] = (float)s;
    }
  }
}

// The same for one or two sets of lines at once (blockIdx.y).
__global__ __launch_bounds__(1024) void line_sums_kernel(LineSums a, LineSums b) {
  const LineSums& l = blockIdx.y ? b : a;
  __shared__ double red[64][17];
  const int cc = threadIdx.x & 15, k = threadIdx.x >> 4, col = blockIdx.x * 16 + cc;
  if (blockIdx.x * 16 >= (unsigned)l.cols) return;
  double s = 0.0;
  if (col < l.cols) {
#pragma unroll 8
    for (int p = k; p < l.parts; p += 64) s += l.part[(int64_t)p * l.cols + col];
  }
  red[k][cc] = s;
  __syncthreads();
  if (k == 0 && col < l.cols) {
    s = 0.0;
#pragma unroll
    for (int i = 0; i < 64; ++i) s += red[i][cc];
    l.out[col] = (float)s;
  }
}

hipError_t launch_line_sums(const LineSums& a, const LineSums& b, hipStream_t stream) {
  const int cols = a.cols > b.cols ? a.cols : b.cols;
  if (cols == 0) return hipSuccess;
  hipLaunchKernelGGL(line_sums_kernel, dim3((cols + 15) / 16, b.cols > 0 ? 2 : 1), dim3(1024), 0, stream, a, b);
  return hipGetLastError();
}

constexpr int kMaxParts = 2048;

int64_t norm_workspace_floats(int64_t N, int C, int lmax) {
  // a line for each workgroup of the gradient kernel: at most kMaxParts, and one a node
  return (N < kMaxParts ? (N > 0 ? N : 1) : kMaxParts) * (lmax + 2) * C;
}

template <auto kernel, int T>
static hipError_t norm_grad_launch(const NormGradArgs& a, int A, float* part, int& parts) {
  parts = norm_grid<kernel, T>(a.N);
  if (parts > kMaxParts) parts = kMaxParts;
  kernel<<<dim3(parts), dim3(norm_threads(T)), 0, a.stream>>>(a, A, norm_inv(a.C), part);
  return hipGetLastError();
}

template <class E, class O, int KT, bool DROP>
static hipError_t norm_grad_t(const NormGradArgs& a) {
  const bool sums = a.gw || a.gb;
  int parts = 0;
  if (a.N > 0) {
    const NormShape s = norm_shape(a.C, a.K);
    float* part = sums ? a.ws : nullptr;
#define EQTP_NORM(T_, NV_) norm_grad_launch<norm_grad_kernel<E, O, T_, NV_, KT, DROP>, T_>(a, s.A, part, parts)
    const hipError_t e = EQTP_NORM_SHAPES(s, EQTP_NORM);
#undef EQTP_NORM
    if (e != hipSuccess) return e;
  }
  if (sums) {
    const int cols = (a.lmax + 2) * a.C;
    hipLaunchKernelGGL(norm_weight_sum_kernel, dim3((cols + 15) / 16), dim3(1024), 0, a.stream, cols, cols - a.C, parts,
                       a.ws, a.gw, a.gb);
    return hipGetLastError();
  }
  return hipSuccess;
}

template <class E, class O>
static hipError_t norm_grad_k(const NormGradArgs& a) {
  if (a.rng) return a.K == 1 ? norm_grad_t<E, O, 0, true>(a) : (a.K % 4 == 0 ? norm_grad_t<E, O, 1, true>(a) : norm_grad_t<E, O, 2, true>(a));
  return a.K == 1 ? norm_grad_t<E, O, 0, false>(a) : (a.K % 4 == 0 ? norm_grad_t<E, O, 1, false>(a) : norm_grad_t<E, O, 2, false>(a));
}

hipError_t launch_norm_grad(const NormGradArgs& a) {
  if (a.x_bf16) return a.out_bf16 ? norm_grad_k<__bf16, __bf16>(a) : norm_grad_k<__bf16, float>(a);
  return a.out_bf16 ? norm_grad_k<float, __bf16>(a) : norm_grad_k<float, float>(a);
}

}  // namespace eqtp
