// distance_bias.hip -- a learned bias of the attention's logits by distance:
//   b(e) = #{j : bounds[j] <= |vec_e|},  bias[e, h] = table[b(e), h],
//   -inf where |vec_e| >= r_cut;  grad_table[b, h] = sum of grad_bias over the
//   edges of bucket b within r_cut.
//
// Lengths are compared as squares in 64 bits: a component squared is exact
// there, so the bucket of an edge next to a bound is the formula's.
//
// Both passes read 12 bytes an edge and write or read 4 H: bound by HBM.
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

// bucket of an edge: how many bounds are at most its length (branch-free bisection over the ascending bounds)
__device__ __forceinline__ int bucket_of(const BiasArgs& a, const double* b2, const float* v) {
  const double x = v[0], y = v[1], z = v[2];
  const double r2 = x * x + y * y + z * z;
  int pos = 0;
  for (int s = a.first_step; s > 0; s >>= 1)
    if (pos + s < a.B && b2[pos + s - 1] <= r2) pos += s;
  return r2 >= a.cut2 ? kBeyond : (r2 == r2 ? pos : kNoLength);
}

// Forward: a wave finds the buckets of 64 edges, one a lane, and then writes
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
// [bucket][lane]: no two lanes share an address, so LDS additions need no order
// among them, every bank serves one lane, and the sums are the same from call
// to call.  A workgroup then adds its lanes and waves in 64 bits into a line of
// part, and the lines are added by the norm's second kernel.
__global__ void distance_bias_grad_kernel(BiasArgs a, int waves, int h0, int hn) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  double* b2 = reinterpret_cast<double*>(lds);
  float* acc = reinterpret_cast<float*>(b2 + a.B);
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  load_bounds(a, b2);
  for (int i = threadIdx.x; i < waves * a.B * 64; i += blockDim.x) acc[i] = 0.0f;
  __syncthreads();
  float* mine = acc + wv * a.B * 64 + lane;
  const int S = 64 / hn;
  const int slot = lane / hn, h = lane - slot * hn;
  const int64_t step = (int64_t)gridDim.x * waves * 64;
  for (int64_t e0 = ((int64_t)blockIdx.x * waves + wv) * 64; e0 < a.E; e0 += step) {
    const int left = (int)min((int64_t)64, a.E - e0);
    const int code = lane < left ? bucket_of(a, b2, a.vec + 3 * (e0 + lane)) : -1;
    const float* g = a.gbias + (e0 + slot) * a.H + h0 + h;
    for (int t = 0; t < 64; t += S) {  // (all lanes take part in every step: they hold each other's buckets)
      const int e = t + slot;
      const int c = __shfl(code, min(e, 63), 64);
      if (slot < S && e < left && c >= 0)
        __hip_atomic_fetch_add(mine + c * 64, g[(int64_t)t * a.H], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    }
  }
  __syncthreads();
  float* line = a.part + (int64_t)blockIdx.x * a.B * a.H;
  for (int i = threadIdx.x; i < a.B * hn; i += blockDim.x) {
    const int b = i / hn, hh = i - b * hn;
    double s = 0.0;
    for (int w = 0; w < waves; ++w)
      for (int k = 0; k < S; ++k) s += acc[(w * a.B + b) * 64 + k * hn + hh];
    line[b * a.H + h0 + hh] = (float)s;
  }
}

constexpr int kBiasParts = 1024;  // workgroups of the gradient kernel at most

struct BiasShape {
  int waves, blocks;
};
// Waves of a gradient workgroup: their tables take up to 64 KB, so that two workgroups share a compute unit's LDS.
static BiasShape bias_shape(int64_t E, int B) {
  BiasShape s;
  s.waves = 65536 / (B * 256);
  s.waves = s.waves < 1 ? 1 : (s.waves > 4 ? 4 : s.waves);
  const int64_t want = (E + s.waves * 64 - 1) / (s.waves * 64);
  s.blocks = (int)(want < kBiasParts ? (want > 0 ? want : 1) : kBiasParts);
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
    const size_t bytes = 8 * (size_t)a.B + (size_t)s.waves * a.B * 256;
    for (int h0 = 0; h0 < a.H; h0 += 64) {
      const int hn = a.H - h0 < 64 ? a.H - h0 : 64;
      distance_bias_grad_kernel<<<dim3(s.blocks), dim3(64 * s.waves), bytes, a.stream>>>(a, s.waves, h0, hn);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  return launch_line_sums(a.B * a.H, a.E > 0 ? s.blocks : 0, a.part, grad_table, a.stream);
}

}  // namespace eqtp
