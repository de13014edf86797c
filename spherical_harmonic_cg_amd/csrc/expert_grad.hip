// expert_grad.hip -- gradient of the experts' weights,
//   grad_W[x, l, c', c] = sum over the places (n, j) of expert x of
//                         weight[n, j] sum_m grad_out[n, c', l m] h[n, c, l m].
//
// Places come grouped by expert (expert_plan.hip).  A wave takes a chunk of one
// expert's places and RT x CTC tiles of 16x16 channels, of degrees 0 to 3
// together or of one degree above, and goes over the chunk four places at a
// time: lane (channel i, k) reads all of those components of channel i of place
// k, of the gradient and of h.  In fp32 a component of each is the operand of
// one product over the four places; in bf16 a degree's components are packed as
// they lie in memory, so one product sums 4 places and up to 8 components.  The
// four waves of a workgroup take turns with a chunk's fours and add their sums
// through LDS in the end, which quarters the lines.
// Bound by the gathered runs' latency: 10k nodes x 64 x 16 fp32, 10 experts, 26
// us (3.1 TB/s) and 6 for the lines' sums; 100k nodes x 32 x 16 bf16, 2 of 8,
// 68 us (410 MB, 6.1 TB/s, half of it found in the L2s) and 7.
// fp32: the products' operands are fp32.  bf16: a gate's product with the
// gradient is held in three bf16 parts, all multiplied, so it keeps its 24 bits
// (two parts would lose 2^-18 of a term, as much as a sum of few terms in all;
// they took 69 us, three 70 to 71).  Where an infinity meets them (inf - inf is
// the second part of an infinite product, and an infinity times a part that is 0
// is NaN) a sum comes out as NaN: the wave then goes over its places again,
// carefully, and what is still NaN is one by the formula.
// Chunks go to lines of part, which a second kernel adds in a fixed
// order: no atomics, the same bits from call to call.
#include <type_traits>

#include "expert_device.hpp"

namespace eqtp {

// Stretches of components that a wave holds at once: degrees 0 to 3 (or up to lmax), then 4, 5 and 6 one at a time.
__host__ __device__ constexpr int stretches_of(int lmax) { return lmax <= 3 ? 1 : lmax - 2; }

struct ChunkOf {
  int x;            // expert, or -1
  int64_t s0, s1;   // its places
};
// Chunk b of the experts' places, `per` places at most each; a whole wave calls it.
__device__ __forceinline__ ChunkOf chunk_of(const int32_t* ptr, int X, int64_t places, int per, int b) {
  const int lane = threadIdx.x & 63;
  ChunkOf r = {-1, 0, 0};
  int before = 0;
  for (int x0 = 0; x0 < X && r.x < 0; x0 += 64) {
    const int x = x0 + lane;
    int64_t lo = 0, hi = 0;
    if (x < X) {
      lo = min(max((int64_t)ptr[x], (int64_t)0), places);
      hi = min(max((int64_t)ptr[x + 1], lo), places);
    }
    const int n = (int)((hi - lo + per - 1) / per);
    int incl = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(incl, o, 64);
      if (lane >= o) incl += u;
    }
    const uint64_t past = __ballot(before + incl > b);
    if (past) {
      const int src = __builtin_ctzll(past);
      const int first = before + __shfl(incl - n, src, 64);
      r.x = __builtin_amdgcn_readfirstlane(x0 + src);
      r.s0 = __shfl((long long)lo, src, 64) + (int64_t)(b - first) * per;
      r.s1 = min(r.s0 + per, (int64_t)__shfl((long long)hi, src, 64));
    }
    before += __shfl(incl, 63, 64);
  }
  return r;
}

// Up to 16 components of a channel in registers, and products of them by degree.
template <class S, bool GATES>
struct Comps;

template <bool GATES>
struct Comps<float, GATES> {
  float x[16];
  __device__ __forceinline__ void load(const float* p, int np) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (4 * w + 4 <= np) {
        const f4 t = Run<float, 4>::load(p + 4 * w);
#pragma unroll
        for (int q = 0; q < 4; ++q) x[4 * w + q] = t[q];
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) x[4 * w + q] = 4 * w + q < np ? p[4 * w + q] : 0.0f;
      }
    }
  }
  template <bool CAREFUL>
  __device__ __forceinline__ void gate(float w, bool live) {
#pragma unroll
    for (int q = 0; q < 16; ++q) x[q] = live ? (GATES ? x[q] * w : x[q]) : 0.0f;
  }
  __device__ __forceinline__ void clear(bool live) {
#pragma unroll
    for (int q = 0; q < 16; ++q) x[q] = live ? x[q] : 0.0f;
  }
  // acc += this (rows) times b (columns) over components first .. first + n - 1 (constants once unrolled)
  template <bool CAREFUL>
  __device__ __forceinline__ void add(const Comps& b, int first, int n, f4& acc) const {
#pragma unroll
    for (int q = 0; q < 16; ++q)
      if (q >= first && q < first + n) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(x[q], b.x[q], acc, 0, 0, 0);
  }
};

// where a pair of bf16 is infinite or NaN: the halves' bits set
__device__ __forceinline__ uint32_t not_finite(uint32_t v) {
  return ((v & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) | ((v & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}

template <bool GATES>
struct Comps<__bf16, GATES> {
  // pairs of components; what the first part of a product leaves, in two parts
  uint32_t x[8], lo[GATES ? 8 : 1], lo2[GATES ? 8 : 1];
  __device__ __forceinline__ void load(const __bf16* p, int np) {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      if (8 * w + 8 <= np) {
        const uint4 t = __builtin_bit_cast(uint4, Run<__bf16, 8>::load(p + 8 * w));
        x[4 * w] = t.x;
        x[4 * w + 1] = t.y;
        x[4 * w + 2] = t.z;
        x[4 * w + 3] = t.w;
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int m = 8 * w + 2 * q;
          x[4 * w + q] = (m < np ? (uint32_t)h[m] : 0u) | (m + 1 < np ? (uint32_t)h[m + 1] << 16 : 0u);
        }
      }
    }
  }
  // The 24 bits of a product in three parts of 8, cut, not rounded: nothing is lost, and a finite one has finite parts.
  // CAREFUL: an infinite one has a first part only.  (Parts of places past the chunk are cleared where there are any:
  // 70 us, in every step 73; in fp32 and without gates that is slower, 33 us instead of 26.)
  template <bool CAREFUL>
  __device__ __forceinline__ void gate(float w, bool live) {
    auto high = [](float a) { return __uint_as_float(__float_as_uint(a) & 0xffff0000u); };
    auto pair = [](float a, float b) { return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u); };
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if constexpr (GATES) {
        const float a = w * __uint_as_float(x[q] << 16), b = w * __uint_as_float(x[q] & 0xffff0000u);
        const float a1 = a - high(a), b1 = b - high(b), a2 = a1 - high(a1), b2 = b1 - high(b1);
        x[q] = pair(a, b);
        lo[q] = pair(a1, b1);
        lo2[q] = pair(a2, b2);
        if constexpr (CAREFUL) {
          lo[q] &= ~not_finite(x[q]);
          lo2[q] &= ~not_finite(x[q]);
        }
      } else {
        x[q] = live ? x[q] : 0u;
      }
    }
  }
  __device__ __forceinline__ void clear(bool live) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      x[q] = live ? x[q] : 0u;
      if constexpr (GATES) {
        lo[q] = live ? lo[q] : 0u;
        lo2[q] = live ? lo2[q] : 0u;
      }
    }
  }
  // word `at` of v, its components outside first .. first + n - 1 cleared
  static __device__ __forceinline__ uint32_t word(const uint32_t (&v)[8], int at, int first, int n) {
    const int m = 2 * at;
    return v[at] & ((m >= first && m < first + n ? 0xffffu : 0u) | (m + 1 >= first && m + 1 < first + n ? 0xffff0000u : 0u));
  }
  // Four words of components are one product's operand; where a degree has one or two, its parts stand beside each other
  // in them.  CAREFUL: an infinity of b meets the first parts only.
  template <bool CAREFUL>
  __device__ __forceinline__ void add(const Comps& b, int first, int n, f4& acc) const {
    constexpr int PARTS = GATES ? 3 : 1;
    const int end = (first + n + 1) / 2;
#pragma unroll
    for (int at = first / 2; at < end; at += 4) {
      const int words = end - at < 4 ? end - at : 4, beside = 4 / words;
#pragma unroll
      for (int p0 = 0; p0 < PARTS; p0 += beside) {
        uint32_t u[4], v[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int p = p0 + s / words, w = at + s % words;
          const bool is = s < beside * words && p < PARTS;
          u[s] = v[s] = 0u;
          if (!is) continue;
          if constexpr (GATES) u[s] = p == 0 ? word(x, w, first, n) : (p == 1 ? word(lo, w, first, n) : word(lo2, w, first, n));
          else u[s] = word(x, w, first, n);
          v[s] = word(b.x, w, first, n);
          if (CAREFUL && p > 0) v[s] &= ~not_finite(v[s]);
        }
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, uint4{u[0], u[1], u[2], u[3]}),
                                                      __builtin_bit_cast(bf16x8, uint4{v[0], v[1], v[2], v[3]}), acc, 0, 0, 0);
      }
    }
  }
};

template <int C>
struct ExpertGradCfg {
  static constexpr int CT = (C + 15) / 16;
  static constexpr int RT = CT < 2 ? CT : 2, CTC = CT < 2 ? CT : 2;  // tiles of a wave: rows, columns
  static constexpr int SPLITS = (CT / RT) * (CT / CTC);
};

constexpr int kGradWaves = 4;  // of a workgroup: they share a chunk

// LMAX: 0 to 3, the degrees of the first stretch; 4 to 6, one degree
template <class S, int C, bool GATES, int LMAX>
__device__ __forceinline__ void expert_grad_walk(const ExpertGradArgs& a, const ChunkOf& ch, int split, float* line, float* lds) {
  using Cfg = ExpertGradCfg<C>;
  constexpr int RT = Cfg::RT, CTC = Cfg::CTC;
  constexpr int L0 = LMAX <= 3 ? 0 : LMAX, LN = LMAX - L0 + 1, NPL = LMAX <= 3 ? (LMAX + 1) * (LMAX + 1) : 2 * LMAX + 1;
  const int K = num_comp(a.lmax), lane = threadIdx.x & 63, wv = threadIdx.x >> 6, i16 = lane & 15, kq = lane >> 4;
  const int rt = split / (Cfg::CT / CTC) * RT, cc = split % (Cfg::CT / CTC) * CTC;
  f4 acc[LN][RT][CTC];
  const int last = (int)min(a.N * a.k, (int64_t)0x7fffffff);
  auto walk = [&](auto careful) {
    constexpr bool CAREFUL = careful;
#pragma unroll
    for (int l = 0; l < LN; ++l)
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < CTC; ++t) acc[l][r][t] = f4{0.f, 0.f, 0.f, 0.f};
    for (int64_t s0 = ch.s0; s0 < ch.s1; s0 += 64) {
      // 64 places, one a lane: node and gate; the waves take turns with the fours of them
      const int64_t mine = min(s0 + lane, ch.s1 - 1);
      const int slot = clamp_index(a.slots[mine], last);
      const int my_node = slot / a.k;
      const float my_gate = GATES ? a.weight[slot] : 1.0f;
      const int steps = (int)min((int64_t)16, (ch.s1 - s0 + 3) / 4);
      for (int st = wv; st < steps; st += kGradWaves) {
        const int from = 4 * st + kq;
        const int64_t node = __shfl(my_node, from, 64);
        const float w = __shfl(my_gate, from, 64);
        const bool live = s0 + from < ch.s1;
        Comps<S, GATES> g[RT], h[CTC];
        const int64_t base = node * C * K + L0 * L0;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const int c = (rt + r) * 16 + i16;
          g[r].load(static_cast<const S*>(a.gout) + base + (c < C ? c : 0) * K, NPL);
        }
#pragma unroll
        for (int t = 0; t < CTC; ++t) {
          const int c = (cc + t) * 16 + i16;
          h[t].load(static_cast<const S*>(a.h) + base + (c < C ? c : 0) * K, NPL);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) g[r].template gate<CAREFUL>(w, live);
        if (s0 + 4 * st + 4 > ch.s1) {  // places past the chunk read its last one's rows: none of it, infinities neither
          if constexpr (GATES && !std::is_same<S, float>::value)
#pragma unroll
            for (int r = 0; r < RT; ++r) g[r].clear(live);
#pragma unroll
          for (int t = 0; t < CTC; ++t) h[t].clear(live);
        }
#pragma unroll
        for (int l = 0; l < LN; ++l)
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < CTC; ++t) {
              if constexpr (LMAX <= 3) g[r].template add<CAREFUL>(h[t], l * l, 2 * l + 1, acc[l][r][t]);
              else g[r].template add<CAREFUL>(h[t], 0, NPL, acc[l][r][t]);
            }
      }
    }
  };
  walk(std::false_type{});
  if constexpr (GATES && std::is_same<S, __bf16>::value) {
    bool nan = false;
#pragma unroll
    for (int l = 0; l < LN; ++l)
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < CTC; ++t)
#pragma unroll
          for (int v = 0; v < 4; ++v) nan |= acc[l][r][t][v] != acc[l][r][t][v];
    if (__any(nan)) walk(std::true_type{});
  }
  // the waves' sums, one wave after the other (in order) into the first one's, a degree at a time
#pragma unroll
  for (int l = 0; l < LN; ++l) {
    constexpr int REGS = RT * CTC * 4;
    __syncthreads();
    if (wv > 0)
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < CTC; ++t)
#pragma unroll
          for (int v = 0; v < 4; ++v) lds[((wv - 1) * REGS + (r * CTC + t) * 4 + v) * 64 + lane] = acc[l][r][t][v];
    __syncthreads();
    if (wv == 0)
#pragma unroll
      for (int w = 0; w < kGradWaves - 1; ++w)
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int t = 0; t < CTC; ++t)
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[l][r][t][v] += lds[(w * REGS + (r * CTC + t) * 4 + v) * 64 + lane];
  }
  if (wv > 0) return;
  // lane (i16, kq) holds D[c' = 4 kq + v][c = i16] of each tile
#pragma unroll
  for (int l = 0; l < LN; ++l)
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < CTC; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int row = (rt + r) * 16 + 4 * kq + v, col = (cc + t) * 16 + i16;
          if (row < C && col < C) line[((int64_t)(L0 + l) * C + row) * C + col] = acc[l][r][t][v];
        }
}

// The splits of a chunk beside each other, on one XCD (workgroups go round the eight).
template <class S, int C, bool GATES>
__global__ __launch_bounds__(64 * kGradWaves) void expert_grad_kernel(ExpertGradArgs a, int per, int lines) {
  constexpr int SPLITS = ExpertGradCfg<C>::SPLITS;
  __shared__ float lds[(kGradWaves - 1) * ExpertGradCfg<C>::RT * ExpertGradCfg<C>::CTC * 4 * 64];
  const int round = blockIdx.x / (8 * SPLITS), in = blockIdx.x % (8 * SPLITS);
  const int chunk = round * 8 + in % 8, split = in / 8;
  if (chunk >= lines) return;
  const ChunkOf ch = chunk_of(a.ptr, a.X, a.N * a.k, per, chunk);
  if (ch.x < 0) return;
  float* line = a.part + (int64_t)chunk * (a.lmax + 1) * C * C;
  switch (blockIdx.y == 0 ? min(a.lmax, 3) : blockIdx.y + 3) {
    case 0: expert_grad_walk<S, C, GATES, 0>(a, ch, split, line, lds); break;
    case 1: expert_grad_walk<S, C, GATES, 1>(a, ch, split, line, lds); break;
    case 2: expert_grad_walk<S, C, GATES, 2>(a, ch, split, line, lds); break;
    case 3: expert_grad_walk<S, C, GATES, 3>(a, ch, split, line, lds); break;
    case 4: expert_grad_walk<S, C, GATES, 4>(a, ch, split, line, lds); break;
    case 5: expert_grad_walk<S, C, GATES, 5>(a, ch, split, line, lds); break;
    default: expert_grad_walk<S, C, GATES, 6>(a, ch, split, line, lds); break;
  }
}

// grad_W[x] = the sum of its chunks' lines, in order, in 64 bits (zeros without one); blockIdx.y: the expert
__global__ __launch_bounds__(256) void expert_grad_sum_kernel(ExpertGradArgs a, int per, int64_t size, int lines) {
  __shared__ int begin, count;
  if (threadIdx.x < 64) {
    // chunks of the experts before this one, and its own
    const int64_t places = a.N * a.k;
    int before = 0, own = 0;
    for (int x = threadIdx.x; x <= (int)blockIdx.y; x += 64) {
      const int64_t lo = min(max((int64_t)a.ptr[x], (int64_t)0), places), hi = min(max((int64_t)a.ptr[x + 1], lo), places);
      const int n = (int)((hi - lo + per - 1) / per);
      if (x < (int)blockIdx.y) before += n;
      else own = n;
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      before += __shfl_xor(before, o, 64);
      own += __shfl_xor(own, o, 64);
    }
    if (threadIdx.x == 0) {
      begin = min(before, lines);
      count = min(own, lines - begin);
    }
  }
  __syncthreads();
  // 64 columns and four stretches of lines a workgroup
  __shared__ double part[4][64];
  const int c = threadIdx.x & 63, k = threadIdx.x >> 6;
  const int64_t i = (int64_t)blockIdx.x * 64 + c;  // (the lines' length is a multiple of 64)
  const float* p = a.part + begin * size + i;
  double s = 0.0;
#pragma unroll 8
  for (int j = k; j < count; j += 4) s += p[j * size];
  part[k][c] = s;
  __syncthreads();
  if (k == 0) a.gW[blockIdx.y * size + i] = (float)((part[0][c] + part[1][c]) + (part[2][c] + part[3][c]));
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
  const int per = chunk_places(a.N, a.C, a.lmax, a.k, a.bf16);
  const int64_t chunks = chunks_at_most(a.N, a.C, a.lmax, a.X, a.k, a.bf16), size = (int64_t)(a.lmax + 1) * C * C;
  if (chunks > 0)
    expert_grad_kernel<S, C, GATES><<<dim3((unsigned)((chunks + 7) / 8 * 8 * ExpertGradCfg<C>::SPLITS), stretches_of(a.lmax)),
                                      dim3(64 * kGradWaves), 0, a.stream>>>(a, per, (int)chunks);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  expert_grad_sum_kernel<<<dim3((unsigned)(size / 64), a.X), dim3(256), 0, a.stream>>>(a, per, size, (int)chunks);
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
