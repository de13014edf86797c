// head_norm.hip -- norm of queries and keys by head and degree, and the
// rotation of channel pairs by position, in one pass over both tensors, and
// the gradients.  A head's row has d channels of K components:
//   r_l = 1 / sqrt(mean_{c, m of l} x^2 + eps),  y = x r_l weight[l, c],
//   theta[j] = sum_a pos[a] freq[a, j],
//   out[j] = y[j] cos theta[j] - y[j + d/2] sin theta[j]        (j < R),
//   out[j + d/2] = y[j] sin theta[j] + y[j + d/2] cos theta[j],
// every component m of a channel by the same angle, so rotations of space
// commute with it where they leave the angles as they are (freq turned with
// pos, or positions along something that space does not turn).  Backward, with u the gradient turned back and a = weight u:
//   gx = r_l a - r_l^3 x mean_l(a x),  gweight[l, c] = sum u x r_l,
//   gtheta[j] = sum_{heads, m} y[j] u[j + d/2] - y[j + d/2] u[j]
// (the cross product of a pair is the same before and after the turn),
//   gpos[a] = sum_j freq[a, j] gtheta[j].
//
// Each element is read and written once; what a long row takes is the cache's
// and HBM's time, a short one its fixed work.  Forward: 10k nodes x 64 channels
// x 16, q and k, 33 us (5.0 TB/s); 100k x (32 + 16) x 16 bf16 70 us (4.4 TB/s);
// 100k rows of 128 + 32 bf16 22 us (2.9 TB/s: a thread's sixteen elements carry
// a norm and eight angles), of fp32 40 us.  Backward, with the weights'
// gradients: the first 74 us (3.3 TB/s, vector ALUs some 40 of them), the second
// 185, the rows 51 (fp32 60); 5 us for the lines' sums.
//
// A group of T threads
// holds a head's row in registers as pairs: quad i of the row's first half
// beside quad i of its second half, NV pairs of quads a thread, so both ends of
// a rotation are in one thread.  As in the layer norm, A threads of a group take quads and a
// thread's slots keep their components and weights from row to row.  A workgroup
// makes the angles of its rows' nodes together, once for all heads of a node.
// Angles are summed and reduced to a fraction of a turn in 64 bits (a position
// of 10^5 times a frequency of 1 loses 4e-3 rad in fp32), their sine and cosine
// are fp32.
#include "norm_device.hpp"

namespace eqtp {

// What a thread's pairs of quads are: Slots of the first half; the second half's slots are the same ones, half a head on.
template <int KT>
constexpr int kTrig = KT == 0 ? 4 : (KT == 1 ? 1 : 2);  // channels of a quad

constexpr int kMaxAxes = 3;

struct HeadShape {
  int T, NV, A;
};

// cosine and sine of a node's angle j
__device__ __forceinline__ void turn_of(const float* pos, const float* freq, int axes, int R, int j, float& c, float& s) {
  double t = 0.0;
  for (int a = 0; a < axes; ++a) t = fma((double)pos[a], (double)freq[a * R + j], t);
  t *= 0.15915494309189533577;  // turns
  t -= rint(t);
  sincospif(2.0f * (float)t, &s, &c);
}

template <int T, int NV, int KT>
struct Turns {
  static constexpr int NC = kTrig<KT>;
  float c[NV][NC], s[NV][NC];
  bool turned[NV][4];  // of the slots' channels: the same in every row
  template <class S>
  __device__ __forceinline__ void begin(const S& sl, int R) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int q = 0; q < NC; ++q) c[j][q] = 1.0f, s[j][q] = 0.0f;
#pragma unroll
      for (int q = 0; q < 4; ++q) turned[j][q] = sl.channel(q, j) < R;
    }
  }
  template <class S>
  static __device__ __forceinline__ int channel(const S& sl, int j, int q) {
    return KT == 0 ? sl.channel(q, j) : sl.channel(0, j) + q;
  }
  template <class S>
  __device__ __forceinline__ void make(const S& sl, const float* pos, const float* freq, int axes, int R) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int q = 0; q < NC; ++q) {
        const int ch = channel(sl, j, q);
        c[j][q] = 1.0f;
        s[j][q] = 0.0f;
        if (sl.on && ch < R) turn_of(pos, freq, axes, R, ch, c[j][q], s[j][q]);
      }
  }
  // from a table of a node's angles [R]
  template <class S>
  __device__ __forceinline__ void read(const S& sl, const float2* table, int R) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int q = 0; q < NC; ++q) {
        const int ch = channel(sl, j, q);
        const float2 t = table[min(ch, R - 1)];
        c[j][q] = ch < R ? t.x : 1.0f;
        s[j][q] = ch < R ? t.y : 0.0f;
      }
  }
  // of slot q
  template <class S>
  __device__ __forceinline__ float cs(const S& sl, int j, int q) const {
    return KT == 0 ? c[j][q % NC] : (KT == 1 ? c[j][0] : (q >= sl.wrap ? c[j][NC - 1] : c[j][0]));
  }
  template <class S>
  __device__ __forceinline__ float sn(const S& sl, int j, int q) const {
    return KT == 0 ? s[j][q % NC] : (KT == 1 ? s[j][0] : (q >= sl.wrap ? s[j][NC - 1] : s[j][0]));
  }
  // A pair, turned; the other way round where SIGN is -1.  Of channels that are not turned both stay as they are, and
  // neither meets the other: a product with sine 0 would make NaN of an infinity half a head away.
  template <int SIGN, class S>
  __device__ __forceinline__ void turn(const S& sl, int j, int q, float& a, float& b) const {
    const float co = cs(sl, j, q), si = sn(sl, j, q);
    const float ta = SIGN > 0 ? fmaf(a, co, -b * si) : fmaf(a, co, b * si);
    const float tb = SIGN > 0 ? fmaf(a, si, b * co) : fmaf(b, co, -a * si);
    a = turned[j][q] ? ta : a;
    b = turned[j][q] ? tb : b;
  }
};

// A workgroup's side (queries or keys) and the first of its groups' items: heads of nodes one after the other, or,
// where a group takes whole nodes, nodes.
struct HeadPlace {
  int64_t first, step, items;
  int side;
};
__device__ __forceinline__ HeadPlace head_place(const HeadNormArgs& a, int R) {
  HeadPlace p;
  p.side = (int)blockIdx.x >= a.blocks_q;
  const int b = blockIdx.x - (p.side ? a.blocks_q : 0);
  const int blocks = p.side ? gridDim.x - a.blocks_q : a.blocks_q;
  p.first = (int64_t)b * R;
  p.step = (int64_t)blocks * R;
  p.items = a.side[p.side].rows * (a.side[p.side].whole ? 1 : a.side[p.side].heads);
  return p;
}
__device__ __forceinline__ int64_t node_of(int64_t item, int64_t items, int heads) {
  return items < 0x80000000 ? (int64_t)((uint32_t)item / (uint32_t)heads) : item / heads;
}

// The angles of the nodes that a workgroup's R items from `first` on belong to, made together: each once for all the
// heads of a node.  tables: two, used in turn.
template <int R>
__device__ __forceinline__ const float2* head_turns(const HeadNormArgs& a, const HeadSide& s, const HeadPlace& p, int64_t first,
                                                    int64_t n0, float2* tables, int size, int& turn) {
  float2* tab = tables + turn * size;
  turn ^= 1;
  const int64_t last = min(first + R, p.items) - 1;
  const int count = (int)(node_of(last, p.items, s.heads) - n0 + 1) * a.R;
  for (int i = threadIdx.x; i < count; i += 256) {
    const int n = i / a.R;
    float2 t;
    turn_of(s.pos + (n0 + n) * a.axes, a.freq, a.axes, a.R, i - n * a.R, t.x, t.y);
    tab[i] = t;
  }
  __syncthreads();
  return tab;
}

template <int T, int NV, int KT>
__device__ __forceinline__ void head_weights(const HeadSide& s, const Slots<T, KT>& sl, int d, int half, float (&w0)[NV][4],
                                             float (&w1)[NV][4]) {
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = sl.channel(q, j);
      w0[j][q] = s.weight && sl.on && c < half ? s.weight[sl.l(q) * d + c] : 1.0f;
      w1[j][q] = s.weight && sl.on && c + half < d ? s.weight[sl.l(q) * d + c + half] : 1.0f;
    }
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      arrived(w0[j][q]);
      arrived(w1[j][q]);
    }
}

// Sums over the group by degree of slot values, the slots' own means: value times 1 / (d (2l + 1)).
template <int T, int KT>
__device__ __forceinline__ void degree_means(const Slots<T, KT>& sl, float (&sq)[4], int deg, float inv_mine, float (&m)[4]) {
  int turn = 0;
  if (!sl.on)
#pragma unroll
    for (int q = 0; q < 4; ++q) sq[q] = 0.0f;
  if constexpr (KT == 0) {
    float v[1] = {(sq[0] + sq[1]) + (sq[2] + sq[3])};
    group_sums<T, 1>(v, 1, nullptr, turn);
#pragma unroll
    for (int q = 0; q < 4; ++q) m[q] = v[0] * inv_mine;
  } else {
    float v[8] = {};
    sl.by_degree(sq, deg, v);
    const float mine = group_sums8<T>(v, nullptr, turn) * inv_mine;
    sl.of_degree(mine, 0, m);
  }
}

template <class E, int T, int NV, int KT>
__global__ __launch_bounds__(256) void head_norm_kernel(HeadNormArgs a, int A) {
  constexpr int R = 256 / T;
  const int d = a.d, K = a.K, half = (d + 1) / 2, D0 = half * K, D1 = (d - half) * K, deg = KT == 0 ? 1 : a.lmax + 1;
  Slots<T, KT> sl(K, A);
  const int g = threadIdx.x / T;
  const HeadPlace p = head_place(a, R);
  const HeadSide s = a.side[p.side];
  const bool tail0 = (D0 & 3) != 0, tail1 = (D1 & 3) != 0;
  const float inv_mine = 1.0f / (float)(d * (KT == 0 ? 1 : 2 * (int)sum8_index<(T < 8 ? 8 : T)>() + 1));
  float w0[NV][4], w1[NV][4];
  head_weights(s, sl, d, half, w0, w1);
  Turns<T, NV, KT> tr;
  tr.begin(sl, a.R);
  extern __shared__ __attribute__((aligned(8))) float2 tables[];
  int turn = 0;
  RowQuads<E, NV> r0, r1;
  auto ask = [&](int64_t at) {
    r0.load((const E*)s.x + at, sl, A, D0);
    r1.load((const E*)s.x + at + D0, sl, A, D1);
  };
  for (int64_t first = p.first; first < p.items; first += p.step) {
    const int64_t item = first + g;
    const bool live = item < p.items;
    int64_t n = min(item, p.items - 1);
    const int64_t at = n * (int64_t)(D0 + D1);
    ask(at);  // (before the angles, which take their time)
    if (a.axes) {
      const int64_t n0 = node_of(first, p.items, s.heads);
      n = node_of(n, p.items, s.heads);
      tr.read(sl, head_turns<R>(a, s, p, first, n0, tables, a.turns, turn) + (n - n0) * a.R, a.R);
    }
    sl.row();
    float x0[NV][4], x1[NV][4], sq[4] = {}, m[4];
    r0.values(sl, A, D0, false, tail0, x0);
    r1.values(sl, A, D1, false, tail1, x1);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) sq[q] = fmaf(x1[j][q], x1[j][q], fmaf(x0[j][q], x0[j][q], sq[q]));
    degree_means<T, KT>(sl, sq, deg, inv_mine, m);
#pragma unroll
    for (int q = 0; q < 4; ++q) m[q] = rsqrtf(m[q] + a.eps);
    E* o = (E*)s.out + at;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = 4 * (sl.t + A * j);
      float o0[4], o1[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        o0[q] = x0[j][q] * m[q] * w0[j][q];
        o1[q] = x1[j][q] * m[q] * w1[j][q];
        tr.template turn<1>(sl, j, q, o0[q], o1[q]);
      }
      if (sl.on && live) {
        store4(o + i, D0 - i, tail0, o0);
        store4(o + D0 + i, D1 - i, tail1, o1);
      }
    }
  }
}

template <class E, int T, int NV, int KT>
__global__ __launch_bounds__(256) void head_norm_grad_kernel(HeadNormArgs a, int A) {
  constexpr int R = 256 / T;
  __shared__ float pos[R * T * NV * 4];  // per group: a value for each place of a half
  __shared__ float head_sums[2][R * kMaxAxes];
  const int d = a.d, K = a.K, half = (d + 1) / 2, D0 = half * K, D1 = (d - half) * K, deg = KT == 0 ? 1 : a.lmax + 1;
  Slots<T, KT> sl(K, A);
  const int g = threadIdx.x / T;
  const HeadPlace p = head_place(a, R);
  const HeadSide s = a.side[p.side];
  const bool tail0 = (D0 & 3) != 0, tail1 = (D1 & 3) != 0;
  const float inv_mine = 1.0f / (float)(d * (KT == 0 ? 1 : 2 * (int)sum8_index<(T < 8 ? 8 : T)>() + 1));
  float w0[NV][4], w1[NV][4], aw0[NV][4] = {}, aw1[NV][4] = {};
  head_weights(s, sl, d, half, w0, w1);
  Turns<T, NV, KT> tr;
  tr.begin(sl, a.R);
  extern __shared__ __attribute__((aligned(8))) float2 tables[];
  int turn = 0;
  RowQuads<E, NV> r0, r1, q0, q1;
  auto ask = [&](int64_t at) {
    r0.load((const E*)s.x + at, sl, A, D0);
    r1.load((const E*)s.x + at + D0, sl, A, D1);
    q0.load((const E*)s.gout + at, sl, A, D0);
    q1.load((const E*)s.gout + at + D0, sl, A, D1);
  };
  for (int64_t first = p.first; first < p.items; first += p.step) {
    const int64_t item = first + g;
    const bool live = item < p.items;
    int64_t n = min(item, p.items - 1);
    int64_t at = n * (s.whole ? s.heads : 1) * (int64_t)(D0 + D1);
    if (!s.whole) {
      const int64_t n0 = node_of(first, p.items, s.heads);
      n = node_of(n, p.items, s.heads);
      if (a.axes) tr.read(sl, head_turns<R>(a, s, p, first, n0, tables, a.turns, turn) + (n - n0) * a.R, a.R);
    } else if (a.axes) {
      tr.make(sl, s.pos + n * a.axes, a.freq, a.axes, a.R);
    }
    const int hn = !live ? 0 : (s.whole ? s.heads : 1);
    float gt[NV][Turns<T, NV, KT>::NC] = {};
    for (int h = 0; h < hn; ++h, at += D0 + D1) {
      sl.row();
      ask(at);
      float x0[NV][4], x1[NV][4], u0[NV][4], u1[NV][4], sq[4] = {}, sa[4] = {}, m[4], ma[4];
      r0.values(sl, A, D0, false, tail0, x0);
      r1.values(sl, A, D1, false, tail1, x1);
      q0.values(sl, A, D0, false, tail0, u0);
      q1.values(sl, A, D1, false, tail1, u1);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          tr.template turn<-1>(sl, j, q, u0[j][q], u1[j][q]);
          sq[q] = fmaf(x1[j][q], x1[j][q], fmaf(x0[j][q], x0[j][q], sq[q]));
          sa[q] = fmaf(u1[j][q] * w1[j][q], x1[j][q], fmaf(u0[j][q] * w0[j][q], x0[j][q], sa[q]));
        }
      degree_means<T, KT>(sl, sq, deg, inv_mine, m);
      degree_means<T, KT>(sl, sa, deg, inv_mine, ma);
      float r[4], r3[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        r[q] = rsqrtf(m[q] + a.eps);
        r3[q] = r[q] * r[q] * ma[q];
      }
      E* o = (E*)s.gx + at;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int i = 4 * (sl.t + A * j);
        float g0[4], g1[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float z0 = x0[j][q] * r[q], z1 = x1[j][q] * r[q];
          aw0[j][q] = fmaf(u0[j][q], z0, aw0[j][q]);
          aw1[j][q] = fmaf(u1[j][q], z1, aw1[j][q]);
          g0[q] = r[q] * fmaf(-x0[j][q], r3[q], u0[j][q] * w0[j][q]);
          g1[q] = r[q] * fmaf(-x1[j][q], r3[q], u1[j][q] * w1[j][q]);
          if (s.gpos) {
            const float cross = fmaf(z0 * w0[j][q], u1[j][q], -z1 * w1[j][q] * u0[j][q]);
            constexpr int NC = Turns<T, NV, KT>::NC;
            if constexpr (KT == 2) {
              gt[j][0] += q >= sl.wrap ? 0.0f : cross;
              gt[j][NC - 1] += q >= sl.wrap ? cross : 0.0f;
            } else {
              gt[j][KT == 0 ? q % NC : 0] += cross;
            }
          }
        }
        if (s.gx && sl.on) {
          store4(o + i, D0 - i, tail0, g0);
          store4(o + D0 + i, D1 - i, tail1, g1);
        }
      }
    }
    if (s.gpos) {  // over the heads: the group's own, or groups beside each other
      float* sums = head_sums[turn] + g * kMaxAxes;
      for (int ax = 0; ax < a.axes; ++ax) {
        float v = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int q = 0; q < Turns<T, NV, KT>::NC; ++q) {
            const int ch = Turns<T, NV, KT>::channel(sl, j, q);
            if (sl.on && ch < a.R) v = fmaf(a.freq[ax * a.R + ch], gt[j][q], v);
          }
        v = lane_sum<T>(v);
        if (sl.t == 0 && live) {
          if (s.whole) s.gpos[n * a.axes + ax] = v;
          else sums[ax] = v;
        }
      }
      if (!s.whole) {
        __syncthreads();
        const int64_t n0 = node_of(first, p.items, s.heads);
        for (int i = threadIdx.x; i < R / s.heads * a.axes; i += 256) {
          const int k = i / a.axes, ax = i - k * a.axes;
          if (n0 + k >= s.rows) continue;
          float v = 0.0f;
          for (int h = 0; h < s.heads; ++h) v += head_sums[turn][(k * s.heads + h) * kMaxAxes + ax];
          s.gpos[(n0 + k) * a.axes + ax] = v;
        }
      }
    }
  }
  if (s.part == nullptr) return;
  // the workgroup's line of the weight gradient [degrees][d]: a half at a time through LDS
  float* line = s.part + (int64_t)(blockIdx.x - (p.side ? a.blocks_q : 0)) * deg * d;
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    const int cn = hf ? d - half : half;
    __syncthreads();
    if (sl.on)
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) pos[g * (T * NV * 4) + 4 * (sl.t + A * j) + q] = hf ? aw1[j][q] : aw0[j][q];
    __syncthreads();
    for (int i = threadIdx.x; i < deg * cn; i += 256) {
      const int l = i / cn, c = i - l * cn;
      double v = 0.0;
      for (int k = 0; k < R; ++k)
        for (int mm = l * l; mm < (l + 1) * (l + 1); ++mm) v += pos[k * (T * NV * 4) + c * K + mm];
      line[l * d + hf * half + c] = (float)v;
    }
  }
}

// The smallest group whose threads hold half a head's row in two quads or fewer, in the gradients, which hold four
// tensors' quads, one (100k rows of 128 bf16: 51 us, with two 52; 10k x 64 x 16 71, with two 70: nearly even, and half
// the registers); beyond 64 threads' worth, four or six (a head's row has up to 2048 elements).  Rows at lmax 1 and above take 8 threads at least, which the sums by
// degree are dealt over.
static HeadShape head_shape(int d, int K, bool grad) {
  const int D0 = (d + 1) / 2 * K, Q = (D0 + 3) / 4;
  const int P = K % 4 == 0 ? K / 4 : K;
  HeadShape s = {64, 0, 64 / P * P};
  for (int T : {1, 2, 4, 8, 16, 32}) {
    if (T < (K > 1 ? 8 : (grad ? 2 : 1))) continue;
    const int A = T / P * P;
    if (A > 0 && (Q + A - 1) / A <= (grad ? 1 : 2)) {
      s = {T, 0, A};
      break;
    }
  }
  s.NV = (Q + s.A - 1) / s.A;
  return s;
}

constexpr int kHeadParts = 2048;  // workgroups of the gradient kernel at most
// Workgroups of a compute unit at most.  100k x (32 + 16) x 16 bf16, forward: 83 us with seven, 70 with six, although
// the registers are for seven; the other sizes that were timed differ by 2 % at most.
constexpr int kHeadHeld = 6;

// How the items of both sides are dealt: workgroups in the ratio of the sides' elements, at most what the card holds.
// A group takes one head at a time, its neighbours the next ones, so that a workgroup reads rows in a stretch; whole
// nodes only for the gradient of positions where a workgroup's groups are no whole number of nodes: it sums over heads.
static void head_deal(HeadNormArgs& a, int T, int held) {
  const int R = 256 / T;
  const int64_t most = (int64_t)num_cus() * held;
  int64_t want[2];
  a.turns = 0;
  for (int i = 0; i < 2; ++i) {
    HeadSide& s = a.side[i];
    s.whole = s.gpos != nullptr && R % s.heads != 0;
    want[i] = (s.rows * (s.whole ? 1 : s.heads) + R - 1) / R;
    // R heads in a row belong to as many nodes at most
    const int nodes = R / s.heads + 2 < R ? R / s.heads + 2 : R;
    if (!s.whole && nodes * a.R > a.turns) a.turns = nodes * a.R;
  }
  const int64_t e0 = a.side[0].rows * a.side[0].heads, e1 = a.side[1].rows * a.side[1].heads;
  int64_t b0 = e0 + e1 > 0 ? (int64_t)((double)most * e0 / (e0 + e1) + 0.5) : 0, b1 = most - b0;
  if (e0 > 0 && b0 < 1) b0 = 1;
  if (e1 > 0 && b1 < 1) b1 = 1;
  a.blocks_q = (int)(want[0] < b0 ? want[0] : b0);
  a.blocks_k = (int)(want[1] < b1 ? want[1] : b1);
}

template <auto kernel, int T>
static hipError_t head_launch(HeadNormArgs a, int A, bool grad, int* blocks) {
  static const int held = [] {
    int n = 0;
    return hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, 256, 0) == hipSuccess && n > 0 ? n : 1;
  }();
  head_deal(a, T, held < kHeadHeld ? held : kHeadHeld);
  if (grad) {
    // a line for each workgroup: as many as the workspace holds for the side
    for (int i = 0; i < 2; ++i) {
      int& b = i ? a.blocks_k : a.blocks_q;
      const int64_t most = a.side[i].rows * a.side[i].heads < kHeadParts ? a.side[i].rows * a.side[i].heads : kHeadParts;
      if (b > most) b = (int)most;
    }
    blocks[0] = a.blocks_q;
    blocks[1] = a.blocks_k;
  }
  if (a.blocks_q + a.blocks_k == 0) return hipSuccess;
  kernel<<<dim3(a.blocks_q + a.blocks_k), dim3(256), 2 * sizeof(float2) * a.turns, a.stream>>>(a, A);
  return hipGetLastError();
}

// Calls F(T, NV): the next of the built sizes.
#define EQTP_HEAD_SHAPES0(s, F)                                                              \
  ((s).T == 1    ? ((s).NV <= 1 ? F(1, 1) : F(1, 2))                                         \
   : (s).T == 2  ? ((s).NV <= 1 ? F(2, 1) : F(2, 2))                                                                   \
   : (s).T == 4  ? F(4, 2)                                                                   \
   : (s).T == 8  ? F(8, 2)                                                                   \
   : (s).T == 16 ? F(16, 2)                                                                  \
   : (s).T == 32 ? F(32, 2)                                                                  \
                 : ((s).NV <= 2 ? F(64, 2) : F(64, 4)))
#define EQTP_HEAD_SHAPES1(s, F)                                                              \
  ((s).T == 8    ? ((s).NV <= 1 ? F(8, 1) : F(8, 2))                                         \
   : (s).T == 16 ? ((s).NV <= 1 ? F(16, 1) : F(16, 2))                                       \
   : (s).T == 32 ? ((s).NV <= 1 ? F(32, 1) : F(32, 2))                                       \
                 : ((s).NV <= 2 ? F(64, 2) : ((s).NV <= 4 ? F(64, 4) : F(64, 6))))

#define EQTP_HEAD_GRAD_SHAPES0(s, F)                                                         \
  ((s).T == 2    ? F(2, 1)                                                                   \
   : (s).T == 4  ? F(4, 1)                                                                   \
   : (s).T == 8  ? F(8, 1)                                                                   \
   : (s).T == 16 ? F(16, 1)                                                                  \
   : (s).T == 32 ? F(32, 1)                                                                  \
                 : ((s).NV <= 1 ? F(64, 1) : ((s).NV <= 2 ? F(64, 2) : F(64, 4))))
#define EQTP_HEAD_GRAD_SHAPES1(s, F)                                                         \
  ((s).T == 8    ? F(8, 1)                                                                   \
   : (s).T == 16 ? F(16, 1)                                                                  \
   : (s).T == 32 ? F(32, 1)                                                                  \
                 : ((s).NV <= 1 ? F(64, 1)                                                   \
                                : ((s).NV <= 2 ? F(64, 2) : ((s).NV <= 4 ? F(64, 4) : F(64, 6)))))

template <class E, int KT>
static hipError_t head_norm_t(const HeadNormArgs& a) {
  const HeadShape s = head_shape(a.d, a.K, false);
#define EQTP_HEAD(T_, NV_) head_launch<head_norm_kernel<E, T_, NV_, KT>, T_>(a, s.A, false, nullptr)
  if constexpr (KT == 0) return EQTP_HEAD_SHAPES0(s, EQTP_HEAD);
  else return EQTP_HEAD_SHAPES1(s, EQTP_HEAD);
#undef EQTP_HEAD
}

template <class E, int KT>
static hipError_t head_norm_grad_t(const HeadNormArgs& a, int* blocks) {
  const HeadShape s = head_shape(a.d, a.K, true);
#define EQTP_HEAD(T_, NV_) head_launch<head_norm_grad_kernel<E, T_, NV_, KT>, T_>(a, s.A, true, blocks)
  if constexpr (KT == 0) return EQTP_HEAD_GRAD_SHAPES0(s, EQTP_HEAD);
  else return EQTP_HEAD_GRAD_SHAPES1(s, EQTP_HEAD);
#undef EQTP_HEAD
}

int64_t head_norm_workspace_floats(int64_t rows, int heads, int d, int lmax) {
  const int64_t lines = rows * heads < kHeadParts ? rows * heads : kHeadParts;
  return lines * (lmax + 1) * d;
}

hipError_t launch_head_norm(const HeadNormArgs& a) {
  if (a.side[0].rows == 0 && a.side[1].rows == 0) return hipSuccess;
  if (a.bf16) return a.K == 1 ? head_norm_t<__bf16, 0>(a) : (a.K % 4 == 0 ? head_norm_t<__bf16, 1>(a) : head_norm_t<__bf16, 2>(a));
  return a.K == 1 ? head_norm_t<float, 0>(a) : (a.K % 4 == 0 ? head_norm_t<float, 1>(a) : head_norm_t<float, 2>(a));
}

hipError_t launch_head_norm_grad(const HeadNormArgs& a, float* const (&gw)[2]) {
  int blocks[2] = {0, 0};
  if (a.side[0].rows > 0 || a.side[1].rows > 0) {
    hipError_t e;
    if (a.bf16) e = a.K == 1 ? head_norm_grad_t<__bf16, 0>(a, blocks) : (a.K % 4 == 0 ? head_norm_grad_t<__bf16, 1>(a, blocks) : head_norm_grad_t<__bf16, 2>(a, blocks));
    else e = a.K == 1 ? head_norm_grad_t<float, 0>(a, blocks) : (a.K % 4 == 0 ? head_norm_grad_t<float, 1>(a, blocks) : head_norm_grad_t<float, 2>(a, blocks));
    if (e != hipSuccess) return e;
  }
  LineSums l[2] = {};
  int n = 0;
  for (int i = 0; i < 2; ++i)
    if (gw[i]) l[n++] = {(a.lmax + 1) * a.d, blocks[i], a.side[i].part, gw[i]};
  return launch_line_sums(l[0], l[1], a.stream);
}

}  // namespace eqtp
