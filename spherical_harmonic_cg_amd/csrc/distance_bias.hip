// distance_bias.hip -- a learned bias of the attention's logits by distance:
//   b(e) = #{j : bounds[j] <= |vec_e|},  bias[e, h] = table[b(e), h],
//   -inf where |vec_e| >= r_cut;  grad_table[b, h] = sum of grad_bias over the
//   edges of bucket b within r_cut.
//
// Lengths are compared as squares in 64 bits: a component squared is exact
// there, so the bucket of an edge next to a bound is the formula's.
//
// Both passes read 12 bytes an edge and write or read 4 H.  Forward: 5.24M edges
// x 8 heads, 64 buckets, 41 us, 5.7 TB/s, a copy's rate; 266k x 4, 33 buckets
// 4.6 us; 20k x 4 3.4 us, a launch.
// Backward: the same cases 88 to 93 us (2.6 TB/s: vector ALUs and LDS) and 12 us,
// and 4 to 5 us for the lines' sums.  A lane adds its own edges of a bucket in
// fp32 (E / (64 waves) of them and a few times as many with many heads), all that
// follows is in 64 bits.
#include "eqtp_device.hpp"
#include "eqtp_kernels.hpp"

namespace eqtp {

typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));

constexpr int kBeyond = -1, kNoLength = -2;  // codes of edges without a bucket

__device__ __forceinline__ float bias_without_bucket(int code) {
  return code == kBeyond ? -__builtin_inff() : __builtin_nanf("");
}

// squares of the bounds; one below 0 lies under every length
__device__ __forceinline__ void load_bounds(const BiasArgs& a, double* b2) {
  for (int i = threadIdx.x; i < a.B - 1; i += blockDim.x) {
    const double b = a.bounds[i];
    b2[i] = b < 0.0 ? -1.0 : b * b;
  }
}

// bucket of an edge: how many bounds are at most its length.  Branch-free search over the ascending bounds, four parts
// at a time: three comparisons beside each other, and half the rounds of a bisection, which wait for each other.
__device__ __forceinline__ int bucket_of(const BiasArgs& a, const double* b2, const float* v) {
  const double x = v[0], y = v[1], z = v[2];
  const double r2 = x * x + y * y + z * z;
  int pos = 0;
  for (int s = a.first_step; s > 0; s >>= 2) {
    int n = 0;
#pragma unroll
    for (int k = 1; k <= 3; ++k) n += pos + k * s < a.B && b2[min(pos + k * s - 1, a.B - 1)] <= r2;
    pos += n * s;
  }
  return r2 >= a.cut2 ? kBeyond : (r2 == r2 ? pos : kNoLength);
}

// Forward (table in LDS up to 48 KB, so that three workgroups share a compute unit; larger ones are read through the
// caches): a wave finds the buckets of 64 edges, one a lane, and then writes
// their 64 H consecutive values together, V a lane and step (V = 4 where H is
// a multiple of 4), each from its edge's row of the table.
template <int V, bool LDS>
__global__ __launch_bounds__(256) void distance_bias_kernel(BiasArgs a) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  double* b2 = reinterpret_cast<double*>(lds);
  float* tab = reinterpret_cast<float*>(b2 + a.B);
  load_bounds(a, b2);
  if constexpr (LDS)
    for (int i = threadIdx.x; i < a.B * a.H; i += 256) tab[i] = a.table[i];
  __syncthreads();
  const float* t = LDS ? tab : a.table;
  const int lane = threadIdx.x & 63;
  const int per = a.H / V;
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t e0 = (int64_t)blockIdx.x * 256 + (threadIdx.x & ~63); e0 < a.E; e0 += step) {
    const int left = (int)min((int64_t)64, a.E - e0);
    const int code = lane < left ? bucket_of(a, b2, a.vec + 3 * (e0 + lane)) : 0;
    float* out = a.bias + e0 * a.H;
    int e = lane / per, h = (lane - e * per) * V;
    const int de = 64 / per, dh = (64 - de * per) * V;
    for (int i = lane; i < 64 * per; i += 64) {
      const int c = __shfl(code, e, 64);
      if (e < left) {
        const float* row = t + max(c, 0) * a.H + h;
        float v[V];
#pragma unroll
        for (int q = 0; q < V; ++q) v[q] = c >= 0 ? row[q] : bias_without_bucket(c);
        if constexpr (V == 4) *reinterpret_cast<f4u*>(out + (int64_t)i * 4) = f4u{v[0], v[1], v[2], v[3]};
        else out[i] = v[0];
      }
      e += de;
      h += dh;
      if (h >= a.H) {
        h -= a.H;
        ++e;
      }
    }
  }
}

// Backward: the 64 lanes of a wave stand for S = 64 / heads edges side by side
// (heads: up to 64 of H), and each lane adds into a table of its own in LDS,
// [bucket][lane]: no two lanes share an address, so there are no atomics (64
// lanes' LDS additions take 190 cycles, a read and a write a few), every bank
// serves one lane, and the sums are the same from call to call.  A workgroup
// then adds its lanes and waves in 64 bits into a line of part, and the lines
// are added by a second kernel, in 64 bits too.
// A wave's next edges, and the first eight steps' values of them, are on their
// way while it adds: with 8 waves a compute unit (their tables fill the LDS)
// little else hides the memory.
__global__ __launch_bounds__(256) void distance_bias_grad_kernel(BiasArgs a, int waves, int h0, int hn) {
  constexpr int T = 8;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  double* b2 = reinterpret_cast<double*>(lds);
  const int rows = a.B + 1;  // the last one takes what no bucket does: masked edges, and places past the last edge
  float* acc = reinterpret_cast<float*>(b2 + a.B);
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  load_bounds(a, b2);
  for (int i = threadIdx.x; i < waves * rows * 64; i += blockDim.x) acc[i] = 0.0f;
  __syncthreads();
  float* mine = acc + wv * rows * 64 + lane;
  const int S = 64 / hn;
  const bool used = lane < S * hn;
  const int slot = used ? lane / hn : 0, h = used ? lane - slot * hn : 0;
  const int64_t step = (int64_t)gridDim.x * waves * 64;
  float v[3], g[T];
  auto ask_edge = [&](int64_t e0) {  // (places past the last edge read the last one's)
    const float* p = a.vec + 3 * e0;
    const int at = 3 * min(lane, (int)min((int64_t)63, a.E - 1 - e0));
#pragma unroll
    for (int q = 0; q < 3; ++q) v[q] = p[at + q];
  };
  auto ask = [&](int64_t e0, int t0) {
    const float* p = a.gbias + e0 * a.H + h0;
    const int last = (int)min((int64_t)63, a.E - 1 - e0);
#pragma unroll
    for (int t = 0; t < T; ++t) g[t] = p[min((t0 + t) * S + slot, last) * a.H + h];
  };
  int64_t e0 = ((int64_t)blockIdx.x * waves + wv) * 64;
  if (e0 < a.E) {
    ask_edge(e0);
    ask(e0, 0);
  }
  for (; e0 < a.E; e0 += step) {
    int code = bucket_of(a, b2, v);
    if (code < 0 || lane >= a.E - e0) code = a.B;
    code *= 64;
    if (e0 + step < a.E) ask_edge(e0 + step);
    for (int t0 = 0; t0 * S < 64; t0 += T) {
      float now[T];
#pragma unroll
      for (int t = 0; t < T; ++t) now[t] = g[t];
      if ((t0 + T) * S < 64) ask(e0, t0 + T);
      else if (e0 + step < a.E) ask(e0 + step, 0);
      int c[T];
#pragma unroll
      for (int t = 0; t < T; ++t) {  // (all lanes take part in every step: they hold each other's buckets)
        const int e = (t0 + t) * S + slot;
        c[t] = __shfl(code, e & 63, 64);
        if (e > 63 || !used) c[t] = a.B * 64;
      }
      // four at a time: read, add one after the other (two of the same bucket follow each other), write in order
#pragma unroll
      for (int t = 0; t < T; t += 4) {
        float s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = mine[c[t + i]];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int k = 0; k < i; ++k) s[i] = c[t + i] == c[t + k] ? s[k] : s[i];
          s[i] += now[t + i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) mine[c[t + i]] = s[i];
      }
    }
  }
  __syncthreads();
  float* line = a.part + (int64_t)blockIdx.x * a.B * a.H;
  for (int i = threadIdx.x; i < a.B * hn; i += blockDim.x) {
    const int b = i / hn, hh = i - b * hn;
    double s = 0.0;
    for (int w = 0; w < waves; ++w)
      for (int k = 0; k < S; ++k) s += acc[(w * rows + b) * 64 + k * hn + hh];
    line[b * a.H + h0 + hh] = (float)s;
  }
}

constexpr int kBiasParts = 2048;  // workgroups of the gradient kernel at most
constexpr int kLdsBytes = 160 << 10;

struct BiasShape {
  int waves, blocks;
};
// Waves of a gradient workgroup: their tables take up to 64 KB and a bit, so that two workgroups share a compute unit's LDS; and
// as many workgroups as the card holds at once (each clears its tables and adds them up in the end).
static BiasShape bias_shape(int64_t E, int B) {
  BiasShape s;
  s.waves = (80 << 10) / ((B + 1) * 256 + 8 * B);
  s.waves = s.waves < 1 ? 1 : (s.waves > 4 ? 4 : s.waves);
  int held = kLdsBytes / (s.waves * (B + 1) * 256 + 8 * B);
  held = held < 1 ? 1 : (held > 32 / s.waves ? 32 / s.waves : held);
  const int64_t want = (E + s.waves * 64 - 1) / (s.waves * 64);
  int64_t most = (int64_t)num_cus() * held;
  if (most > kBiasParts) most = kBiasParts;
  s.blocks = (int)(want < most ? (want > 0 ? want : 1) : most);
  return s;
}

int64_t bias_workspace_floats(int64_t E, int B, int H) { return (int64_t)bias_shape(E, B).blocks * B * H; }

template <int V, bool LDS>
static hipError_t bias_launch(const BiasArgs& a) {
  const int64_t want = (a.E + 255) / 256, most = (int64_t)num_cus() * 8;
  const size_t bytes = 8 * (size_t)a.B + (LDS ? 4 * (size_t)a.B * a.H : 0);
  distance_bias_kernel<V, LDS><<<dim3((unsigned)(want < most ? want : most)), dim3(256), bytes, a.stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_distance_bias(const BiasArgs& a) {
  if (a.E == 0) return hipSuccess;
  const bool lds = a.B * a.H <= 12288;
  if (a.H % 4 == 0) return lds ? bias_launch<4, true>(a) : bias_launch<4, false>(a);
  return lds ? bias_launch<1, true>(a) : bias_launch<1, false>(a);
}

hipError_t launch_distance_bias_grad(const BiasArgs& a, float* grad_table) {
  const BiasShape s = bias_shape(a.E, a.B);
  if (a.E > 0) {
    const size_t bytes = 8 * (size_t)a.B + (size_t)s.waves * (a.B + 1) * 256;
    for (int h0 = 0; h0 < a.H; h0 += 64) {
      const int hn = a.H - h0 < 64 ? a.H - h0 : 64;
      distance_bias_grad_kernel<<<dim3(s.blocks), dim3(64 * s.waves), bytes, a.stream>>>(a, s.waves, h0, hn);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  return launch_line_sums({a.B * a.H, a.E > 0 ? s.blocks : 0, a.part, grad_table}, {}, a.stream);
}

}  // namespace eqtp
