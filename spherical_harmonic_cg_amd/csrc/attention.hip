// attention.hip -- attention over the edges of a graph (CSR rows), forward and
// backward; no per-edge vectors are formed in memory.
//   s = scale q[dst] . k[src] + bias,  w = softmax of s over the row,
//   out[n] = sum w v[src].
//
// Every edge reads a row of k and one of v by its source (backward: by rows k
// and v again, by sources q and the output's gradient), 2 E C K elements each
// time.  A query meets each of them once, so the products stay on the vector
// ALUs and the gathers bound the kernels: rows outside an XCD's L2 (4 MiB)
// arrive at 7.4 to 8.2 TB/s, whatever holds them.  10k atoms, 266k edges,
// 4 heads of 256 fp32 elements: 2.18 GB a pass, forward 250, by rows 267, by
// sources 285 us (8.7, 8.2, 7.7 TB/s, a fifth of it L2 hits; vector ALUs busy
// 36, 47 and 43% of the time); 100k atoms, 5.2M edges, bf16, 2 key and value
// heads of 128: 5.37 GB, 718 us (7.5 TB/s).
//
// A head's row of D elements is a line of 16-byte units.  G lanes hold it, NU
// units each (unit lig + G j), beside the q and sums of the same places; dot
// products are added over the G lanes by register moves.  A wave takes HW
// heads of a row side by side and, where they do not fill it, ES edges at a
// time (their partial results are joined at the row's end).  EU edges are
// loaded together, with the next ones' indexes and biases on the way.  The
// softmax runs along the row in one pass: a running maximum and sum, one
// rescaling for each EU edges.
//
// Few long rows (a readout) are cut into S pieces of about equal length, whose
// partial results go through the workspace and are added by a second kernel.
#include <type_traits>

#include "eqtp_device.hpp"
#include "eqtp_kernels.hpp"
#include "lane_ops.hpp"

namespace eqtp {

constexpr float kLog2E = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLog2ELow = (float)(1.4426950408889634 - (double)kLog2E);
// exp(v) / 2^down for a difference of logits (taken before the change to base 2: biases of the type's lowest value
// would overflow in it).  The hardware's exponential is of base 2; of its argument v log2 e the whole part is taken off
// first and the rest, at most 1/2, formed with log2 e in two parts.  Rounded as one product the argument would cost |v|
// half steps of the result (57 of them measured at v = -57, against 2.6 at most); the cases' times are the same, a
// single wave's long row takes a tenth longer.  Below -300 the result is 0 in any case (|down| < 100), and no infinity
// enters the differences; NaN stays NaN.
__device__ __forceinline__ float exp_of(float v, int down = 0) {
  v = v < -300.0f ? -300.0f : v;
  const float whole = __builtin_rintf(v * kLog2E);
  const float rest = fmaf(v, kLog2ELow, fmaf(v, kLog2E, -whole));
  return __builtin_ldexpf(__builtin_amdgcn_exp2f(rest), (int)whole - down);
}

// ---- 16 bytes of a row --------------------------------------------------------
typedef uint32_t u4u __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

template <class T>
struct El;
template <>
struct El<float> {
  static constexpr int VE = 4;
  static __device__ __forceinline__ float at(const u4& r, int i) {
    const uint32_t w = r[i];  // a value: the cast of a vector's element itself takes element 0
    return __builtin_bit_cast(float, w);
  }
  static __device__ __forceinline__ float dot(const u4& a, const u4& b, float c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = fmaf(at(a, i), at(b, i), c);
    return c;
  }
};
template <>
struct El<__bf16> {
  static constexpr int VE = 8;
  static __device__ __forceinline__ float at(const u4& r, int i) {
    return __builtin_bit_cast(float, i & 1 ? r[i >> 1] & 0xffff0000u : r[i >> 1] << 16);
  }
  // Pairs of exact products, added to the running sum by one instruction with one rounding; what lies below the
  // largest of the three by more than a few bits of an fp32 value is cut off first, as separate fp32 additions would
  // round it off.  Subnormals are kept; a product past fp32's range is infinite.
  static __device__ __forceinline__ float dot(const u4& a, const u4& b, float c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = a[i], y = b[i];
      c = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, x), __builtin_bit_cast(bf16x2, y), c, false);
    }
    return c;
  }
};

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
// Piece s of S of it.
__device__ __forceinline__ RowRange piece(RowRange r, int s, int S) {
  const int64_t len = r.e - r.b;
  return {r.b + len * s / S, r.b + len * (s + 1) / S};
}

// How a wave's lanes lie over (edge, head, place in the head's row).  MODE 0:
// the units fill the G lanes and rows are whole units; 1: units past the row
// are masked and the row's last unit ends at its end (its first elements, which
// the unit before holds, are masked); 2: rows shorter than a unit.
template <class T, int G, int NU, int MODE>
struct Lanes {
  static constexpr int VE = El<T>::VE;
  int lig, hs, es;
  int off[NU];               // first element of each unit
  u4 mask[MODE == 1 ? NU : 1];
  __device__ __forceinline__ Lanes(int D, int HW) {
    const int lane = threadIdx.x & 63;
    lig = lane & (G - 1);
    hs = lane / G & (HW - 1);
    es = lane / (G * HW);
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      off[j] = VE * (lig + G * j);
      if constexpr (MODE == 1) {
        const int at = min(off[j], D - VE), lo = off[j] < D ? off[j] - at : VE;  // elements below lo are not this unit's
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (VE == 4) mask[j][i] = i >= lo ? ~0u : 0u;
          else mask[j][i] = (2 * i >= lo ? 0xffffu : 0u) | (2 * i + 1 >= lo ? 0xffff0000u : 0u);
        }
        off[j] = at;
      }
    }
  }
  __device__ __forceinline__ u4 load(const T* row, int j, int D) const {
    if constexpr (MODE == 2) {
      u4 r = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < VE; ++i)
        if (i < D) {
          if constexpr (VE == 4) r[i] = __builtin_bit_cast(uint32_t, row[i]);
          else r[i >> 1] |= (uint32_t)__builtin_bit_cast(uint16_t, row[i]) << (16 * (i & 1));
        }
      return r;
    } else {
      u4 r = *reinterpret_cast<const u4u*>(row + off[j]);
      if constexpr (MODE == 1) r &= mask[j];
      return r;
    }
  }
  // stores f(i) at the unit's own elements
  template <class F>
  __device__ __forceinline__ void store(T* row, int j, int D, F f) const {
    if constexpr (MODE == 0) {
      u4 r = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const T t = (T)f(i);
        if constexpr (VE == 4) r[i] = __builtin_bit_cast(uint32_t, t);
        else r[i >> 1] |= (uint32_t)__builtin_bit_cast(uint16_t, t) << (16 * (i & 1));
      }
      *reinterpret_cast<u4u*>(row + off[j]) = r;
    } else {
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const bool own = MODE == 2 ? i < D : (VE == 4 ? mask[MODE == 1 ? j : 0][i & 3] != 0u
                                                      : (mask[MODE == 1 ? j : 0][i >> 1] >> (16 * (i & 1)) & 1u) != 0u);
        if (own) row[off[j] + i] = (T)f(i);
      }
    }
  }
  template <class F>
  __device__ __forceinline__ void store_f32(float* row, int j, int D, F f) const {
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const bool own = MODE == 0 || (MODE == 2 ? i < D : (VE == 4 ? mask[MODE == 1 ? j : 0][i & 3] != 0u
                                                                  : (mask[MODE == 1 ? j : 0][i >> 1] >> (16 * (i & 1)) & 1u) != 0u));
      if (own) row[off[j] + i] = f(i);
    }
  }
};

// What a launch fixes for its waves.
struct Tiling {
  int HW, ES;       // heads and edges (or, SHORT, rows) of a wave side by side (powers of two)
  int blocks;       // of HW heads
  int S;            // pieces of a row
  int step;         // distance of a lane's next edge: ES, or 1 where lanes side by side have rows of their own
  int spread;       // head blocks are dealt to the XCDs: 8 / blocks of them for each; 0: not
  int64_t first;    // task of the launch's first wave, and the end of the tasks (one head block's, where spread)
  int64_t end;
  float* part;      // S > 1: partial results
};

// A wave's task: its row, piece and head block, the same for all lanes, but the row where lanes have their own.
struct Task {
  int64_t row, n;  // row S + piece, row
  int sp, hb;
  bool in;         // a row of the graph (a wave's last rows may lie past the end)
};
__device__ __forceinline__ bool find_task(const Tiling& t, int64_t rows, int es, Task& k) {
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t task;
  if (t.spread) {
    // workgroups go to the XCDs in turn: an XCD sees one block of heads only, and keeps more of its rows in its L2
    const int x = blockIdx.x & 7;
    k.hb = x / t.spread;
    task = (((int64_t)(blockIdx.x >> 3) * t.spread) + (x & (t.spread - 1))) * 4 + wv;
    if (task >= t.end) return false;
  } else {
    task = t.first + (int64_t)blockIdx.x * 4 + wv;
    if (task >= t.end) return false;
    if (t.blocks == 1) {
      k.hb = 0;
    } else {
      const int64_t r = task / t.blocks;
      k.hb = (int)(task - r * t.blocks);
      task = r;
    }
  }
  k.in = true;
  k.sp = 0;
  if (t.S > 1) {
    k.row = task;
    k.n = task / t.S;
    k.sp = (int)(task - k.n * t.S);
  } else if (t.step != t.ES) {
    k.n = task * t.ES + es;
    k.in = k.n < rows;
    k.n = k.in ? k.n : rows - 1;
    k.row = k.n;
  } else {
    k.row = k.n = task;
  }
  return true;
}

__device__ __forceinline__ u4 keep_if(const u4& v, bool keep) {
  const uint32_t m = keep ? ~0u : 0u;
  return v & u4{m, m, m, m};
}

// Waves a SIMD that the compiler is held to where it comes to a few registers more than three leave it (168): whole
// units, and fp32 rows of four units a lane.  Masked units take 178 and more; those are left to it.
template <class T, int NU, int MODE>
constexpr int attn_waves() {
  return MODE == 0 || (El<T>::VE == 4 && NU == 4) ? 3 : 1;
}

// One wave: heads hb HW .. of row n, piece s.
template <class T, int G, int NU, int MODE, int EU>
__global__ __launch_bounds__(256, (attn_waves<T, NU, MODE>())) void attn_kernel(AttnArgs a, Tiling t) {
  constexpr int VE = El<T>::VE;
  const int D = a.D, H = a.heads;
  const Lanes<T, G, NU, MODE> ln(D, t.HW);
  Task task;
  if (!find_task(t, a.N, ln.es, task)) return;
  const int64_t row = task.row, n = task.n;
  const int hb = task.hb;
  const int h = min(hb * t.HW + ln.hs, H - 1), R = H / a.kv_heads;
  const bool mine = hb * t.HW + ln.hs < H;
  const int64_t rowlen = (int64_t)a.kv_heads * D;
  const T* kb = (const T*)a.k + (int64_t)(h / R) * D;
  const T* vb = (const T*)a.v + (int64_t)(h / R) * D;
  u4 q[NU];
  float acc[NU][VE] = {};
#pragma unroll
  for (int j = 0; j < NU; ++j) q[j] = ln.load((const T*)a.q + (n * H + h) * D, j, D);
  RowRange r = piece(row_range(a.row_ptr, n, a.E), task.sp, t.S);
  if (!task.in) r.e = r.b;
  const int es = t.step == t.ES ? ln.es : 0;
  float top = -INFINITY, sum = 0.0f;
  int idx[EU];
  float bias[EU];
  auto fetch = [&](int64_t e0) {
#pragma unroll
    for (int i = 0; i < EU; ++i) {
      int64_t e = e0 + i * t.step + es;
      e = e < r.e ? e : (r.e > 0 ? r.e - 1 : 0);  // (r.e = 0: a row of its own beside others that have edges)
      idx[i] = a.src[e];
      bias[i] = a.bias ? a.bias[e * H + h] : 0.0f;
    }
  };
  if (__any(r.b < r.e)) fetch(r.b);
  for (int64_t e0 = r.b; __any(e0 < r.e); e0 += EU * t.step) {
    u4 k[EU][NU], v[EU][NU];
    float s[EU];
    bool live[EU], all = true;
#pragma unroll
    for (int i = 0; i < EU; ++i) {
      const int64_t at = (int64_t)clamp_index(idx[i], (int)a.M) * rowlen;
#pragma unroll
      for (int j = 0; j < NU; ++j) k[i][j] = ln.load(kb + at, j, D);
#pragma unroll
      for (int j = 0; j < NU; ++j) v[i][j] = ln.load(vb + at, j, D);
      s[i] = bias[i];
      live[i] = bias[i] != -INFINITY && e0 + i * t.step + es < r.e;
      all = all && live[i];
    }
    if (__any(e0 + EU * t.step < r.e)) fetch(e0 + EU * t.step);
    float m = top;
#pragma unroll
    for (int i = 0; i < EU; ++i) {
      float d = 0.0f;
#pragma unroll
      for (int j = 0; j < NU; ++j) d = El<T>::dot(q[j], k[i][j], d);
      s[i] = fmaf(a.scale, lane_sum<G>(d), s[i]);
    }
    if (!__all(all)) {  // masked edges and places past the row take no part, whatever they hold
#pragma unroll
      for (int i = 0; i < EU; ++i) {
        s[i] = live[i] ? s[i] : -INFINITY;
#pragma unroll
        for (int j = 0; j < NU; ++j) v[i][j] = keep_if(v[i][j], live[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < EU; ++i) m = fmaxf(m, s[i]);
    const float base = m == -INFINITY ? 0.0f : m;
    const float down = exp_of(top - base);
    top = m;
    sum *= down;
#pragma unroll
    for (int j = 0; j < NU; ++j)
#pragma unroll
      for (int x = 0; x < VE; ++x) acc[j][x] *= down;
#pragma unroll
    for (int i = 0; i < EU; ++i) {
      const float w = exp_of(s[i] - base);
      sum += w;
#pragma unroll
      for (int j = 0; j < NU; ++j)
#pragma unroll
        for (int x = 0; x < VE; ++x) acc[j][x] = fmaf(w, El<T>::at(v[i][j], x), acc[j][x]);
    }
  }
  // join the edges that ran side by side
  for (int d = t.step == t.ES ? G * t.HW : 64; d < 64; d <<= 1) {
    const float other = __shfl_xor(top, d, 64), m = fmaxf(top, other), base = m == -INFINITY ? 0.0f : m;
    const float down = exp_of(top - base), od = exp_of(other - base);
    top = m;
    sum = fmaf(sum, down, __shfl_xor(sum, d, 64) * od);
#pragma unroll
    for (int j = 0; j < NU; ++j)
#pragma unroll
      for (int x = 0; x < VE; ++x) acc[j][x] = fmaf(acc[j][x], down, __shfl_xor(acc[j][x], d, 64) * od);
  }
  if (!mine || !task.in || es != 0) return;
  if (t.S > 1) {
    float* ml = t.part + (int64_t)a.N * t.S * H * D;
#pragma unroll
    for (int j = 0; j < NU; ++j) ln.store_f32(t.part + (row * H + h) * D, j, D, [&](int x) { return acc[j][x]; });
    if (ln.lig == 0) {
      ml[(row * H + h) * 2] = top;
      ml[(row * H + h) * 2 + 1] = sum;
    }
    return;
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int j = 0; j < NU; ++j) ln.store((T*)a.out + (n * H + h) * D, j, D, [&](int x) { return acc[j][x] * inv; });
  if (a.lse && ln.lig == 0) a.lse[n * H + h] = sum == 0.0f ? -INFINITY : top + __builtin_amdgcn_logf(sum) * kLn2;
}

constexpr int kMaxPieces = 1024, kJoin = 1024;  // pieces of a row; threads of a workgroup that joins them

// Sums of v over a workgroup of kJoin threads, or the largest, the same in every thread.
template <bool MAX>
__device__ __forceinline__ float over_group(float v, float* red) {
  for (int d = 32; d; d >>= 1) {
    const float o = __shfl_xor(v, d, 64);
    v = MAX ? fmaxf(v, o) : v + o;
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < kJoin / 64; ++i) v = MAX ? fmaxf(v, red[i]) : v + red[i];
  return v;
}

// sum over the pieces k, k + W, .. of f(piece), then over the W threads of a place; the result in the threads with
// k = 0.
template <class F>
__device__ __forceinline__ float over_pieces(int S, int k, int W, int L, float* red, F f) {
  float acc = 0.0f;
#pragma unroll 4
  for (int s = k; s < S; s += W) acc += f(s);
  __syncthreads();
  red[threadIdx.x] = acc;
  for (int w = W; w > 1; w >>= 1) {
    __syncthreads();
    if (k < w / 2) red[threadIdx.x] += red[threadIdx.x + w / 2 * L];
  }
  return red[threadIdx.x];
}

// Joins the pieces of the rows: a workgroup a (row, head) and L places; its threads lie over the pieces and the places.
template <class T>
__global__ __launch_bounds__(kJoin) void attn_join_kernel(AttnArgs a, Tiling t, int L) {
  __shared__ float red[kJoin], w[kMaxPieces], few[kJoin / 64];
  const int H = a.heads, D = a.D, S = t.S;
  const int64_t n = blockIdx.x / H;
  const int h = (int)(blockIdx.x - n * H), d = blockIdx.y * L + (threadIdx.x & (L - 1)), k = threadIdx.x / L, W = kJoin / L;
  const float* part = t.part + (n * S * H + h) * D;
  const float* ml = t.part + a.N * S * H * (int64_t)D + (n * S * H + h) * 2;
  float top = -INFINITY, sum = 0.0f;
  for (int s = threadIdx.x; s < S; s += kJoin) {
    w[s] = ml[(int64_t)s * H * 2];
    top = fmaxf(top, w[s]);
  }
  top = over_group<true>(top, few);
  const float base = top == -INFINITY ? 0.0f : top;
  for (int s = threadIdx.x; s < S; s += kJoin) {
    w[s] = exp_of(w[s] - base);
    sum = fmaf(ml[(int64_t)s * H * 2 + 1], w[s], sum);
  }
  sum = over_group<false>(sum, few);
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const float acc = over_pieces(S, k, W, L, red, [&](int s) { return d < D ? part[(int64_t)s * H * D + d] * w[s] : 0.0f; });
  if (k == 0 && d < D) ((T*)a.out)[(n * H + h) * D + d] = (T)(acc * inv);
  if (a.lse && threadIdx.x == 0 && blockIdx.y == 0) a.lse[n * H + h] = sum == 0.0f ? -INFINITY : top + __builtin_amdgcn_logf(sum) * kLn2;
}

// ---- gradients ------------------------------------------------------------------
// Row pass: grad_q, and per edge and head the weight w and u = w (a - t),
// a = g . v, which the source pass reads.  t = sum w a is known only at the
// row's end, so sum u k is formed as sum w a k - t sum w k, and a waits in u's
// place until then.  (Two sums that partly cancel; against fp32 operations with
// t at hand grad_q is 0.75 to 0.9 times as far off on rows of 20 edges over
// several lanes, k and v with or without a common mean of up to 16 times their
// spread, 1.26 times where one lane adds a row, 1.1 on rows of 7000.)  The
// weights exp(s - lse) are summed and divided by their sum again: it is 1 but
// for lse's rounding, which counts where the logits are so large that the sum's
// logarithm is lost in lse (biases of the lowest value).  It allows any other
// factor near 1 too: a moderate lse is taken off as a whole power of two instead
// of in the difference, which would round (8 half steps of a weight in a row of
// 4096 edges).
//
// Both lie in tables of E heads numbers, edge by edge, or head by head where
// heads are dealt to the XCDs: each then writes and reads stretches of its own
// (edge by edge, four of them wrote to every line: 120 MB written instead of
// 85, of which the bias's gradient, the caller's and edge by edge, is a part,
// and 8.5 MB of tables beside the gathered rows in each L2 instead of 2).
struct EdgeTables {
  float* w;
  float* u;
  float* gbias;    // u also goes here, edge by edge; or nullptr (u is the caller's, or not asked for)
  int64_t se, sh;  // distance of edges and of heads
  __device__ __forceinline__ int64_t at(int64_t e, int h) const { return e * se + h * sh; }
  __device__ __forceinline__ void finish(int64_t e, int h, int H, float t, float inv) const {
    const int64_t i = at(e, h);
    const float weight = w[i] * inv, v = weight == 0.0f ? 0.0f : weight * (u[i] - t);
    w[i] = weight;
    u[i] = v;
    if (gbias) gbias[e * H + h] = v;
  }
};

template <class T, int G, int NU, int MODE, int EU>
__global__ __launch_bounds__(256) void attn_grad_row_kernel(AttnGradArgs a, Tiling t, EdgeTables tab) {
  constexpr int VE = El<T>::VE;
  const int D = a.D, H = a.heads;
  const Lanes<T, G, NU, MODE> ln(D, t.HW);
  Task task;
  if (!find_task(t, a.N, ln.es, task)) return;
  const int64_t row = task.row, n = task.n;
  const int hb = task.hb;
  const int h = min(hb * t.HW + ln.hs, H - 1), R = H / a.kv_heads;
  const bool mine = hb * t.HW + ln.hs < H;
  const int64_t rowlen = (int64_t)a.kv_heads * D;
  const T* kb = (const T*)a.k + (int64_t)(h / R) * D;
  const T* vb = (const T*)a.v + (int64_t)(h / R) * D;
  u4 q[NU], g[NU];
  float wak[NU][VE] = {}, wk[NU][VE] = {}, tt = 0.0f, total = 0.0f;
#pragma unroll
  for (int j = 0; j < NU; ++j) {
    q[j] = ln.load((const T*)a.q + (n * H + h) * D, j, D);
    g[j] = ln.load((const T*)a.gout + (n * H + h) * D, j, D);
  }
  const float lse = a.lse[n * H + h];
  const bool moderate = fabsf(lse) < 64.0f;
  const float from = moderate ? 0.0f : lse;
  const int down = moderate ? (int)__builtin_rintf(lse * kLog2E) : 0;
  RowRange r = piece(row_range(a.row_ptr, n, a.E), task.sp, t.S);
  if (!task.in) r.e = r.b;
  const int es = t.step == t.ES ? ln.es : 0;
  int idx[EU];
  float bias[EU];
  auto fetch = [&](int64_t e0) {
#pragma unroll
    for (int i = 0; i < EU; ++i) {
      int64_t e = e0 + i * t.step + es;
      e = e < r.e ? e : (r.e > 0 ? r.e - 1 : 0);  // (r.e = 0: a row of its own beside others that have edges)
      idx[i] = a.src[e];
      bias[i] = a.bias ? a.bias[e * H + h] : 0.0f;
    }
  };
  if (__any(r.b < r.e)) fetch(r.b);
  for (int64_t e0 = r.b; __any(e0 < r.e); e0 += EU * t.step) {
    u4 k[EU][NU], v[EU][NU];
    float s[EU];
    bool live[EU], in[EU], all = true;
#pragma unroll
    for (int i = 0; i < EU; ++i) {
      const int64_t at = (int64_t)clamp_index(idx[i], (int)a.M) * rowlen;
#pragma unroll
      for (int j = 0; j < NU; ++j) k[i][j] = ln.load(kb + at, j, D);
#pragma unroll
      for (int j = 0; j < NU; ++j) v[i][j] = ln.load(vb + at, j, D);
      s[i] = bias[i];
      in[i] = e0 + i * t.step + es < r.e;
      live[i] = bias[i] != -INFINITY && in[i];
      all = all && live[i];
    }
    if (__any(e0 + EU * t.step < r.e)) fetch(e0 + EU * t.step);
    if (!__all(all)) {
#pragma unroll
      for (int i = 0; i < EU; ++i) {
        s[i] = live[i] ? s[i] : -INFINITY;
#pragma unroll
        for (int j = 0; j < NU; ++j) {
          k[i][j] = keep_if(k[i][j], live[i]);
          v[i][j] = keep_if(v[i][j], live[i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < EU; ++i) {
      float d = 0.0f, av = 0.0f;
#pragma unroll
      for (int j = 0; j < NU; ++j) {
        d = El<T>::dot(q[j], k[i][j], d);
        av = El<T>::dot(g[j], v[i][j], av);
      }
      s[i] = s[i] == -INFINITY ? s[i] : fmaf(a.scale, lane_sum<G>(d), s[i]);
      av = lane_sum<G>(av);
      const bool none = s[i] == -INFINITY;
      const float w = none ? 0.0f : exp_of(s[i] - from, down), wa = none ? 0.0f : w * av;
      tt += wa;
      total += w;
#pragma unroll
      for (int j = 0; j < NU; ++j)
#pragma unroll
        for (int x = 0; x < VE; ++x) {
          const float kx = El<T>::at(k[i][j], x);
          wak[j][x] = fmaf(wa, kx, wak[j][x]);
          wk[j][x] = fmaf(w, kx, wk[j][x]);
        }
      if (mine && in[i] && ln.lig == 0) {
        const int64_t at = tab.at(e0 + i * t.step + es, h);
        tab.w[at] = w;
        tab.u[at] = none ? 0.0f : av;
      }
    }
  }
  for (int d = t.step == t.ES ? G * t.HW : 64; d < 64; d <<= 1) {
    tt += __shfl_xor(tt, d, 64);
    total += __shfl_xor(total, d, 64);
#pragma unroll
    for (int j = 0; j < NU; ++j)
#pragma unroll
      for (int x = 0; x < VE; ++x) {
        wak[j][x] += __shfl_xor(wak[j][x], d, 64);
        wk[j][x] += __shfl_xor(wk[j][x], d, 64);
      }
  }
  if (t.S > 1) {
    if (!mine || es != 0) return;
    const int64_t all = a.N * t.S * H * (int64_t)D;
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      ln.store_f32(t.part + (row * H + h) * D, j, D, [&](int x) { return wak[j][x]; });
      ln.store_f32(t.part + all + (row * H + h) * D, j, D, [&](int x) { return wk[j][x]; });
    }
    if (ln.lig == 0) {
      t.part[2 * all + (row * H + h) * 2] = tt;
      t.part[2 * all + (row * H + h) * 2 + 1] = total;
    }
    return;
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  tt *= inv;
  if (a.gq && mine && task.in && es == 0)
#pragma unroll
    for (int j = 0; j < NU; ++j)
      ln.store((T*)a.gq + (n * H + h) * D, j, D, [&](int x) { return fmaf(-tt, wk[j][x], wak[j][x]) * (inv * a.scale); });
  // w and u of the row's edges: lanes over (edge, head), once the wave's own stores above are done
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
  if (t.step == t.ES) {
    const int hh = (threadIdx.x & 63) & (t.HW - 1);
    const float th = __shfl(tt, hh * G, 64), ih = __shfl(inv, hh * G, 64);
    if (hb * t.HW + hh < H)
      for (int64_t e = r.b + (threadIdx.x & 63) / t.HW; e < r.e; e += 64 / t.HW) tab.finish(e, hb * t.HW + hh, H, th, ih);
  } else if (mine) {
    for (int64_t e = r.b + ln.lig; e < r.e; e += G) tab.finish(e, h, H, tt, inv);
  }
}

// Joins the pieces of the row pass: t and the weights' sum, then grad_q.
template <class T>
__global__ __launch_bounds__(kJoin) void attn_grad_join_kernel(AttnGradArgs a, Tiling t, int L) {
  __shared__ float red[kJoin], few[kJoin / 64];
  const int H = a.heads, D = a.D, S = t.S;
  const int64_t n = blockIdx.x / H, all = a.N * S * H * (int64_t)D;
  const int h = (int)(blockIdx.x - n * H), d = blockIdx.y * L + (threadIdx.x & (L - 1)), k = threadIdx.x / L, W = kJoin / L;
  const float* tp = t.part + 2 * all + (n * S * H + h) * 2;
  float tt = 0.0f, total = 0.0f;
  for (int s = threadIdx.x; s < S; s += kJoin) {
    tt += tp[(int64_t)s * H * 2];
    total += tp[(int64_t)s * H * 2 + 1];
  }
  tt = over_group<false>(tt, few);
  total = over_group<false>(total, few);
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  tt *= inv;
  if (threadIdx.x == 0 && blockIdx.y == 0) {
    float* o = t.part + 2 * all + (a.N * S * H + n * H + h) * 2;
    o[0] = tt;
    o[1] = inv;
  }
  if (a.gq) {
    const float* p = t.part + (n * S * H + h) * D + d;
    const float x = over_pieces(S, k, W, L, red, [&](int s) { return d < D ? p[(int64_t)s * H * D] : 0.0f; });
    const float y = over_pieces(S, k, W, L, red, [&](int s) { return d < D ? p[all + (int64_t)s * H * D] : 0.0f; });
    if (k == 0 && d < D) ((T*)a.gq)[(n * H + h) * D + d] = (T)(fmaf(-tt, y, x) * (inv * a.scale));
  }
}

// w and u of every edge of the pieces, from their rows' joined sums: a workgroup a (row, piece).  (By the joining
// workgroups themselves, one head each, it took 15 us more for a readout of 50k items and 8 heads: 4 of 32 bytes.)
__global__ __launch_bounds__(256) void attn_grad_fix_kernel(AttnGradArgs a, Tiling t, EdgeTables tab) {
  const int H = a.heads;
  const int64_t n = blockIdx.x / t.S;
  const RowRange r = piece(row_range(a.row_ptr, n, a.E), (int)(blockIdx.x - n * t.S), t.S);
  const float* tt = t.part + 2 * (a.N * t.S * H * (int64_t)a.D) + (a.N * t.S + n) * H * 2;
  for (int64_t i = threadIdx.x; i < (r.e - r.b) * H; i += 256) {
    const int h = (int)(i % H);
    tab.finish(r.b + i / H, h, H, tt[h * 2], tt[h * 2 + 1]);
  }
}

// Source pass: grad_k = scale sum u q, grad_v = sum w g over a source's edges
// (and the heads that share a key and value head).
template <class T, int G, int NU, int MODE, int EU>
__global__ __launch_bounds__(256) void attn_grad_source_kernel(AttnGradArgs a, Tiling t, EdgeTables tab) {
  constexpr int VE = El<T>::VE;
  const int D = a.D, H = a.heads, HK = a.kv_heads;
  const Lanes<T, G, NU, MODE> ln(D, t.HW);
  Task task;
  if (!find_task(t, a.M, ln.es, task)) return;
  const int64_t row = task.row, m = task.n;
  const int hb = task.hb;
  const int hk = min(hb * t.HW + ln.hs, HK - 1), R = H / HK;
  const bool mine = hb * t.HW + ln.hs < HK;
  float ka[NU][VE] = {}, va[NU][VE] = {};
  RowRange r = piece(row_range(a.src_ptr, m, a.E), task.sp, t.S);
  if (!task.in) r.e = r.b;
  const int es = t.step == t.ES ? ln.es : 0;
  int edge[EU], dst[EU];
  auto fetch = [&](int64_t i0) {
#pragma unroll
    for (int i = 0; i < EU; ++i) {
      int64_t e = i0 + i * t.step + es;
      e = e < r.e ? e : (r.e > 0 ? r.e - 1 : 0);
      edge[i] = a.perm[e];
      dst[i] = a.dst_s[e];
    }
  };
  if (__any(r.b < r.e)) fetch(r.b);
  for (int64_t i0 = r.b; __any(i0 < r.e); i0 += EU * t.step) {
    int64_t eh[EU], nh[EU];
#pragma unroll
    for (int i = 0; i < EU; ++i) {
      eh[i] = tab.at(clamp_index(edge[i], (int)a.E), hk * R);
      nh[i] = ((int64_t)clamp_index(dst[i], (int)a.N) * H + hk * R) * D;
    }
    if (__any(i0 + EU * t.step < r.e)) fetch(i0 + EU * t.step);
    for (int h = 0; h < R; ++h) {
      u4 q[EU][NU], g[EU][NU];
      float w[EU], u[EU];
      bool all = true;
#pragma unroll
      for (int i = 0; i < EU; ++i) {
        const bool in = i0 + i * t.step + es < r.e;
        w[i] = in ? tab.w[eh[i] + h * tab.sh] : 0.0f;
        u[i] = in ? tab.u[eh[i] + h * tab.sh] : 0.0f;
#pragma unroll
        for (int j = 0; j < NU; ++j) q[i][j] = ln.load((const T*)a.q + nh[i] + (int64_t)h * D, j, D);
#pragma unroll
        for (int j = 0; j < NU; ++j) g[i][j] = ln.load((const T*)a.gout + nh[i] + (int64_t)h * D, j, D);
      }
#pragma unroll
      for (int i = 0; i < EU; ++i) all = all && (w[i] != 0.0f || u[i] != 0.0f);
      if (!__all(all)) {  // masked edges and places past the row: whatever the rows hold
#pragma unroll
        for (int i = 0; i < EU; ++i)
#pragma unroll
          for (int j = 0; j < NU; ++j) {
            q[i][j] = keep_if(q[i][j], w[i] != 0.0f || u[i] != 0.0f);
            g[i][j] = keep_if(g[i][j], w[i] != 0.0f || u[i] != 0.0f);
          }
      }
#pragma unroll
      for (int i = 0; i < EU; ++i)
#pragma unroll
        for (int j = 0; j < NU; ++j)
#pragma unroll
          for (int x = 0; x < VE; ++x) {
            ka[j][x] = fmaf(u[i], El<T>::at(q[i][j], x), ka[j][x]);
            va[j][x] = fmaf(w[i], El<T>::at(g[i][j], x), va[j][x]);
          }
    }
  }
  for (int d = t.step == t.ES ? G * t.HW : 64; d < 64; d <<= 1)
#pragma unroll
    for (int j = 0; j < NU; ++j)
#pragma unroll
      for (int x = 0; x < VE; ++x) {
        ka[j][x] += __shfl_xor(ka[j][x], d, 64);
        va[j][x] += __shfl_xor(va[j][x], d, 64);
      }
  if (!mine || !task.in || es != 0) return;
  if (t.S > 1) {
    const int64_t all = a.M * t.S * HK * (int64_t)D;
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      ln.store_f32(t.part + (row * HK + hk) * D, j, D, [&](int x) { return ka[j][x]; });
      ln.store_f32(t.part + all + (row * HK + hk) * D, j, D, [&](int x) { return va[j][x]; });
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < NU; ++j) {
    if (a.gk) ln.store((T*)a.gk + (m * HK + hk) * D, j, D, [&](int x) { return ka[j][x] * a.scale; });
    if (a.gv) ln.store((T*)a.gv + (m * HK + hk) * D, j, D, [&](int x) { return va[j][x]; });
  }
}

template <class T>
__global__ __launch_bounds__(kJoin) void attn_source_join_kernel(AttnGradArgs a, Tiling t, int L) {
  __shared__ float red[kJoin];
  const int HK = a.kv_heads, D = a.D, S = t.S;
  const int64_t m = blockIdx.x / HK, all = a.M * S * HK * (int64_t)D;
  const int h = (int)(blockIdx.x - m * HK), d = blockIdx.y * L + (threadIdx.x & (L - 1)), k = threadIdx.x / L, W = kJoin / L;
  const float* p = t.part + (m * S * HK + h) * D + d;
  const float x = over_pieces(S, k, W, L, red, [&](int s) { return d < D ? p[(int64_t)s * HK * D] : 0.0f; });
  const float y = over_pieces(S, k, W, L, red, [&](int s) { return d < D ? p[all + (int64_t)s * HK * D] : 0.0f; });
  if (k == 0 && d < D) {
    if (a.gk) ((T*)a.gk)[(m * HK + h) * D + d] = (T)(x * a.scale);
    if (a.gv) ((T*)a.gv)[(m * HK + h) * D + d] = (T)y;
  }
}

// ---- launch ---------------------------------------------------------------------
static int pow2_from(int v) {
  int p = 1;
  while (p < v) p <<= 1;
  return p;
}

// Pieces of a row: where the rows alone give fewer than kMinWaves waves, as many as bring them there, of kMinPiece
// edges on average or more (7 rows over 50k items, 8 heads of 16: one wave a row 15 ms, 292 pieces 14 us and 6 to join).
// (1024 waves of 64 edges or more: 15 and 19 us forward and by rows; 2048 of 32: 14 and 15; 4096: the same.)
// The rule knows the rows' number and their mean length, not the longest: among kMinWaves rows and more a row is one
// wave's (or, beside short ones, one lane group's) however long it is.  10k rows, 300k edges, 4 heads of 16, trained: 84
// us with even rows, 14 ms with 100k of the edges in one row, 6 ms with 100k at one source.
constexpr int64_t kMinWaves = 2048, kMinPiece = 32;
// (a join's grid is a workgroup of kJoin threads for each of fewer than kMinWaves rows and each head)
static_assert((kMinWaves - 1) * kMaxAttnHeads * kJoin < ((int64_t)1 << 32), "a grid holds fewer than 2^32 threads");
static int pieces(int64_t rows, int64_t E) {
  if (rows <= 0 || rows >= kMinWaves) return 1;
  int64_t s = (kMinWaves + rows - 1) / rows;
  const int64_t by_length = E / rows / kMinPiece;
  s = s < by_length ? s : by_length;
  s = s < kMaxPieces ? s : kMaxPieces;
  return s < 2 ? 1 : (int)s;
}

int64_t attn_workspace_bytes(int64_t N, int64_t, int64_t E, int D, int heads, int) {
  const int S = pieces(N, E);
  return S == 1 ? 0 : 4 * N * S * heads * ((int64_t)D + 2);
}

static int64_t grad_tables(int64_t E, int heads) { return (2 * 4 * E * heads + 15) / 16 * 16; }

int64_t attn_grad_workspace_bytes(int64_t N, int64_t M, int64_t E, int D, int heads, int kv_heads) {
  const int S = pieces(N, E), Z = pieces(M, E);
  const int64_t rows = S == 1 ? 0 : 4 * N * heads * (S * (2 * (int64_t)D + 2) + 2);
  const int64_t sources = Z == 1 ? 0 : 4 * M * Z * kv_heads * 2 * (int64_t)D;
  return grad_tables(E, heads) + (rows > sources ? rows : sources);
}

constexpr int64_t kSpreadLine = 512, kSpreadBytes = (int64_t)8 << 20, kSpreadMost = (int64_t)32 << 20, kShortRow = 8,
                  kShortPlaces = 4;

// Lanes and units of a head's row: up to 8 units one a lane, then two, four, eight a lane.
struct HeadShape {
  int G, NU, mode;
};
static HeadShape head_shape(int D, int VE) {
  const int U = (D + VE - 1) / VE;
  HeadShape s;
  s.NU = U <= 8 ? 1 : (U <= 32 ? 2 : (U <= 256 ? 4 : 8));
  s.G = pow2_from((U + s.NU - 1) / s.NU);
  s.mode = D < VE ? 2 : (D == s.G * s.NU * VE ? 0 : 1);
  return s;
}
static bool is_pow2(int v) { return (v & (v - 1)) == 0; }

// heads of the pass (of q, or of k and v), share of them that read the same rows, rows and edges of the pass, bytes
// of the two gathered tensors and of a head's row in them.
static Tiling tiling(const HeadShape& s, int heads, int share, int64_t rows, int64_t E, int64_t gathered,
                     int row_bytes, float* part) {
  Tiling t;
  const int room = 64 / s.G, kv = heads / share;
  t.S = pieces(rows, E);
  t.HW = pow2_from(heads) < room ? pow2_from(heads) : room;
  // Heads dealt to the XCDs: each L2 then sees one slice of the gathered tensors and finds more of it (10k atoms,
  // 4 heads, 82 MB: slices of 20 MB, a fifth of the reads; 308 -> 250 us forward).  Not up to 8 MB, where much is
  // found by whatever XCD (10k rows of 27 edges, 4 heads of 256; 4 MB: fp32 forward 99 us, 104 if dealt, bf16 66 and 90;
  // 6 MB: 132 and 104, trained 838 and 838, bf16 75 and 91; 8 MB: 171 and 105, trained 959 and 880, bf16 92 and 91), nor
  // where a slice is so large that hardly anything is found (51 MB: 718 -> 726 us), nor with slices of less than some
  // cache lines a row (64-byte pieces of 512-byte rows: 69 -> 250 us).
  t.spread = 0;
  int nb = kv < 8 ? kv : 8;
  while (nb > 1 && kv / nb * row_bytes < kSpreadLine) nb >>= 1;
  if (t.S == 1 && nb > 1 && gathered > kSpreadBytes && gathered / nb <= kSpreadMost && is_pow2(kv) && is_pow2(share) &&
      heads / nb <= room &&
      rows < ((int64_t)1 << 22)) {  // (eight workgroups for four rows: below 2^32 threads)
    t.HW = heads / nb;
    t.spread = 8 / nb;
  }
  t.ES = room / t.HW;
  t.blocks = (heads + t.HW - 1) / t.HW;
  // Rows of few edges beside the places for edges (ES by EU): lanes side by side take rows of their own.  50k rows of
  // 20 edges, 4 heads of one element (ES 16): forward 77 -> 25 us; 50k sources of one edge: 46 -> 27 us.
  const bool few = E < rows * kShortRow || (E < rows * t.ES * kShortPlaces && rows / t.ES >= kMinWaves / 4);
  t.step = t.S == 1 && t.ES > 1 && few ? 1 : t.ES;
  t.first = t.end = 0;
  t.part = part;
  return t;
}
static int64_t wave_tasks(const Tiling& t, int64_t rows) {
  if (t.S > 1) return rows * t.S;
  return t.step != t.ES ? (rows + t.ES - 1) / t.ES : rows;
}

// Launches over all tasks; a launch holds at most 2^24 waves (2^32 threads is the
// grid's limit).
template <class L>
static hipError_t over_tasks(int64_t rows, Tiling& t, L launch) {
  constexpr int64_t kMost = (int64_t)1 << 24;
  const int64_t tasks = wave_tasks(t, rows);
  if (t.spread) {
    t.end = tasks;
    const int64_t groups = (tasks + 3) / 4;
    launch(dim3((unsigned)((groups + t.spread - 1) / t.spread * 8)));
    return hipGetLastError();
  }
  t.end = tasks * t.blocks;
  for (t.first = 0; t.first < t.end; t.first += kMost) {
    const int64_t n = t.end - t.first < kMost ? t.end - t.first : kMost;
    launch(dim3((unsigned)((n + 3) / 4)));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
// Calls f(G, NU, MODE) as constants.  Of eight units a lane there are fp32 rows only (2048 bf16 elements fill 64
// lanes of four); a single unit a row is whole or short.
template <class T, class F>
static void with_shape(const HeadShape& s, F f) {
  auto modes = [&](auto G, auto NU) {
    if (s.mode == 0) f(G, NU, std::integral_constant<int, 0>());
    else f(G, NU, std::integral_constant<int, 1>());
  };
  typedef std::integral_constant<int, 1> I1;
  typedef std::integral_constant<int, 2> I2;
  typedef std::integral_constant<int, 4> I4;
  typedef std::integral_constant<int, 8> I8;
  typedef std::integral_constant<int, 16> I16;
  typedef std::integral_constant<int, 32> I32;
  typedef std::integral_constant<int, 64> I64;
  if (s.mode == 2) f(I1(), I1(), I2());
  else if (s.NU == 1 && s.G == 1) f(I1(), I1(), std::integral_constant<int, 0>());
  else if (s.NU == 1 && s.G == 2) modes(I2(), I1());
  else if (s.NU == 1 && s.G == 4) modes(I4(), I1());
  else if (s.NU == 1) modes(I8(), I1());
  else if (s.NU == 2 && s.G == 8) modes(I8(), I2());
  else if (s.NU == 2) modes(I16(), I2());
  else if (s.NU == 4 && s.G == 16) modes(I16(), I4());
  else if (s.NU == 4 && s.G == 32) modes(I32(), I4());
  else if (s.NU == 4) modes(I64(), I4());
  else if constexpr (El<T>::VE == 4) modes(I64(), I8());
}

// places of a row that a joining workgroup takes: 64 bytes, so that 64 threads share each place's pieces
static int join_lanes(int D) { return pow2_from(D) < 16 ? pow2_from(D) : 16; }
static dim3 join_grid(int64_t rows, int D) { return dim3((unsigned)rows, (unsigned)((D + join_lanes(D) - 1) / join_lanes(D))); }

template <class T>
static hipError_t attn_t(const AttnArgs& a) {
  const HeadShape s = head_shape(a.D, El<T>::VE);
  Tiling t = tiling(s, a.heads, a.heads / a.kv_heads, a.N, a.E, 2 * a.M * a.kv_heads * a.D * (int64_t)sizeof(T), a.D * (int)sizeof(T), (float*)a.ws);
  const hipError_t e = over_tasks(a.N, t, [&](dim3 grid) {
    with_shape<T>(s, [&](auto G, auto NU, auto MODE) {
      attn_kernel<T, G(), NU(), MODE(), 8 / NU()><<<grid, dim3(256), 0, a.stream>>>(a, t);
    });
  });
  if (e != hipSuccess || t.S == 1) return e;
  attn_join_kernel<T><<<join_grid(a.N * a.heads, a.D), dim3(kJoin), 0, a.stream>>>(a, t, join_lanes(a.D));
  return hipGetLastError();
}

template <class T>
static hipError_t attn_grad_t(const AttnGradArgs& a) {
  EdgeTables tab = {(float*)a.ws, a.gbias ? a.gbias : (float*)a.ws + a.E * a.heads, nullptr, a.heads, 1};
  float* part = (float*)((unsigned char*)a.ws + grad_tables(a.E, a.heads));
  const HeadShape s = head_shape(a.D, El<T>::VE);
  if (a.N > 0) {
    Tiling t = tiling(s, a.heads, a.heads / a.kv_heads, a.N, a.E, 2 * a.M * a.kv_heads * a.D * (int64_t)sizeof(T), a.D * (int)sizeof(T), part);
    if (t.spread) tab = {tab.w, tab.w + a.E * a.heads, a.gbias, 1, a.E};
    hipError_t e = over_tasks(a.N, t, [&](dim3 grid) {
      with_shape<T>(s, [&](auto G, auto NU, auto MODE) {
        attn_grad_row_kernel<T, G(), NU(), MODE(), (NU() >= 4 ? 1 : 4 / NU())><<<grid, dim3(256), 0, a.stream>>>(a, t, tab);
      });
    });
    if (e != hipSuccess) return e;
    if (t.S > 1) {
      attn_grad_join_kernel<T><<<join_grid(a.N * a.heads, a.D), dim3(kJoin), 0, a.stream>>>(a, t, join_lanes(a.D));
      e = hipGetLastError();
      if (e != hipSuccess) return e;
      attn_grad_fix_kernel<<<dim3((unsigned)(a.N * t.S)), dim3(256), 0, a.stream>>>(a, t, tab);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  if (a.M == 0 || (!a.gk && !a.gv)) return hipSuccess;
  Tiling t = tiling(s, a.kv_heads, 1, a.M, a.E, 2 * a.N * a.heads * a.D * (int64_t)sizeof(T), a.D * (int)sizeof(T), part);
  // sources of one or two edges (a readout's items have one): places for four would stay empty and cost the registers
  // that more waves need (50k sources of one edge: 27 against 15 us)
  const bool one = a.E <= 2 * a.M;
  const hipError_t e = over_tasks(a.M, t, [&](dim3 grid) {
    with_shape<T>(s, [&](auto G, auto NU, auto MODE) {
      if (one)
        attn_grad_source_kernel<T, G(), NU(), MODE(), 1><<<grid, dim3(256), 0, a.stream>>>(a, t, tab);
      else
        attn_grad_source_kernel<T, G(), NU(), MODE(), (NU() >= 4 ? 1 : 4 / NU())><<<grid, dim3(256), 0, a.stream>>>(a, t, tab);
    });
  });
  if (e != hipSuccess || t.S == 1) return e;
  attn_source_join_kernel<T><<<join_grid(a.M * a.kv_heads, a.D), dim3(kJoin), 0, a.stream>>>(a, t, join_lanes(a.D));
  return hipGetLastError();
}

hipError_t launch_attention(const AttnArgs& a) { return a.bf16 ? attn_t<__bf16>(a) : attn_t<float>(a); }

hipError_t launch_attention_grad(const AttnGradArgs& a) {
  return a.bf16 ? attn_grad_t<__bf16>(a) : attn_grad_t<float>(a);
}

}  // namespace eqtp
