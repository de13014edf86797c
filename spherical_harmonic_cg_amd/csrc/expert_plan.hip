// expert_plan.hip -- groups the places (node n, j) of a routing by expert, and
// orders the nodes so that neighbours in the order go to the same experts.
//   slots [N k]: n k + j, by expert, in input order within one (what the weight
//                gradient sums over); places without an expert come last;
//   ptr [X+1]:   where each expert's places begin;
//   order [N]:   the nodes by their two lowest experts.
// Stable counting sorts of both at once: counts of a tile of nodes in LDS, one
// scan, ranks from wave ballots; three launches (100k nodes, 2 of 8 experts: 5 + 7
// + 6 us, each a few dependent steps), or one for few places (one node 5 us).  With many experts the nodes'
// second key is coarsened to 1024 bins in all: order only has to be a good
// one, the linear's results do not depend on it.
#include "eqtp_device.hpp"
#include "eqtp_kernels.hpp"

namespace eqtp {

constexpr int kPlanBins = 1024;
constexpr int kPlanTiles = 256, kPlanCounts = 1 << 16;  // tiles, and counts of the nodes' keys, at most (one workgroup adds them)

struct PlanShape {
  int X, k, b_bins, bins2, rounds, tiles;
  int64_t N;
};
static PlanShape plan_shape(int64_t N, int k, int X) {
  PlanShape p;
  p.N = N;
  p.X = X;
  p.k = k;
  p.b_bins = X + 1 < kPlanBins / (X + 1) ? X + 1 : kPlanBins / (X + 1);
  p.bins2 = (X + 1) * p.b_bins;
  const int64_t most = 256 * (int64_t)(kPlanCounts / p.bins2 < kPlanTiles ? kPlanCounts / p.bins2 : kPlanTiles);
  const int64_t r = (N + most - 1) / most;
  p.rounds = r < 1 ? 1 : (int)r;
  p.tiles = (int)((N + 256 * (int64_t)p.rounds - 1) / (256 * (int64_t)p.rounds));
  if (p.tiles < 1) p.tiles = 1;
  return p;
}

int64_t expert_plan_ints(int64_t N, int k, int X) {
  const PlanShape p = plan_shape(N, k, X);
  return (int64_t)(X + 1 + p.bins2) * p.tiles;
}

__device__ __forceinline__ int expert_of(int v, int X) { return v >= 0 && v < X ? v : X; }

// key of a node: its lowest expert and the lowest of the others (X: none)
__device__ __forceinline__ int node_key(const PlanShape& p, const int32_t* idx, int64_t n) {
  int lo = p.X, next = p.X;
  for (int j = 0; j < p.k; ++j) {
    const int e = expert_of(idx[n * p.k + j], p.X);
    if (e < lo) {
      next = lo;
      lo = e;
    } else if (e > lo && e < next) {
      next = e;
    }
  }
  return lo * p.b_bins + (next * p.b_bins) / (p.X + 1);
}

__global__ __launch_bounds__(256) void plan_count_kernel(PlanShape p, const int32_t* __restrict__ idx, int* __restrict__ hist1,
                                                         int* __restrict__ hist2) {
  __shared__ int c1[kMaxExperts + 1], c2[kPlanBins];
  for (int b = threadIdx.x; b <= p.X; b += 256) c1[b] = 0;
  for (int b = threadIdx.x; b < p.bins2; b += 256) c2[b] = 0;
  __syncthreads();
  const int64_t n0 = (int64_t)blockIdx.x * 256 * p.rounds;
  const int64_t n1 = min(p.N, n0 + 256 * (int64_t)p.rounds);
  for (int64_t s = n0 * p.k + threadIdx.x; s < n1 * p.k; s += 256) atomicAdd(&c1[expert_of(idx[s], p.X)], 1);
  if (hist2)
    for (int64_t n = n0 + threadIdx.x; n < n1; n += 256) atomicAdd(&c2[node_key(p, idx, n)], 1);
  __syncthreads();
  for (int b = threadIdx.x; b <= p.X; b += 256) hist1[b * p.tiles + blockIdx.x] = c1[b];
  if (hist2)
    for (int b = threadIdx.x; b < p.bins2; b += 256) hist2[b * p.tiles + blockIdx.x] = c2[b];
}

// Exclusive scans of both counts (a workgroup each) in place; ptr from the first.  4096 counts at a time through LDS, so
// that memory is read and written along the lanes; the next ones are on their way meanwhile.
__global__ __launch_bounds__(1024) void plan_scan_kernel(PlanShape p, int* __restrict__ hist1, int* __restrict__ hist2,
                                                         int32_t* __restrict__ ptr) {
  __shared__ int wsum[16], part[4096];
  int* a = blockIdx.x ? hist2 : hist1;
  const int len = (blockIdx.x ? p.bins2 : p.X + 1) * p.tiles;
  const int t = threadIdx.x, lane = t & 63, wv = t >> 6;
  int carry = 0, next[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) next[q] = 1024 * q + t < len ? a[1024 * q + t] : 0;
  for (int c0 = 0; c0 < len; c0 += 4096) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      part[1024 * q + t] = next[q];
      const int i = c0 + 4096 + 1024 * q + t;
      next[q] = i < len ? a[i] : 0;
    }
    __syncthreads();
    int v[4], sum = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[q] = part[4 * t + q];
      sum += v[q];
    }
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int u = __shfl_up(incl, off, 64);
      if (lane >= off) incl += u;
    }
    if (lane == 63) wsum[wv] = incl;
    __syncthreads();
    int run = carry + incl - sum, all = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
      run += w < wv ? wsum[w] : 0;
      all += wsum[w];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      part[4 * t + q] = run;
      run += v[q];
    }
    carry += all;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = c0 + 1024 * q + t;
      if (i < len) a[i] = part[1024 * q + t];
    }
    __syncthreads();  // part and wsum are written again
  }
  if (blockIdx.x == 0)
    for (int x = t; x <= p.X; x += 1024) ptr[x] = a[x * p.tiles];
}

// Places of one round's 256 items among those of their keys, in item order: toff [bins] are the keys' next free
// places, wcnt [4][bins] zeros.  Every thread calls it; returns the item's place (-1 without one).
__device__ __forceinline__ int take_places(int key, bool valid, int bits, int bins, int* toff, int* wcnt) {
  const int t = threadIdx.x, lane = t & 63, wv = t >> 6;
  uint64_t same = __ballot(valid);
  for (int b = 0; b < bits; ++b) {
    const bool bit = (key >> b) & 1;
    const uint64_t on = __ballot(bit);
    same &= bit ? on : ~on;
  }
  const int rank = __popcll(same & (lane == 0 ? 0ull : (~0ull >> (64 - lane))));
  if (valid && rank == 0) wcnt[wv * bins + key] = __popcll(same);
  __syncthreads();
  int pos = -1;
  if (valid) {
    pos = toff[key] + rank;
    for (int w = 0; w < wv; ++w) pos += wcnt[w * bins + key];
  }
  __syncthreads();
  for (int b = t; b < bins; b += 256) {
    int sum = 0;
    for (int w = 0; w < 4; ++w) {
      sum += wcnt[w * bins + b];
      wcnt[w * bins + b] = 0;
    }
    toff[b] += sum;
  }
  __syncthreads();
  return pos;
}

__device__ __forceinline__ int bits_for(int bins) { return bins > 1 ? 32 - __clz(bins - 1) : 0; }

// blockIdx.y 0: slots, 1: order
__global__ __launch_bounds__(256) void plan_place_kernel(PlanShape p, const int32_t* __restrict__ idx,
                                                         const int* __restrict__ hist1, const int* __restrict__ hist2,
                                                         int32_t* __restrict__ slots, int32_t* __restrict__ order) {
  __shared__ int toff[kPlanBins], wcnt[4 * kPlanBins];
  const bool nodes = blockIdx.y != 0;
  const int bins = nodes ? p.bins2 : p.X + 1;
  const int* hist = nodes ? hist2 : hist1;
  for (int b = threadIdx.x; b < bins; b += 256) {
    toff[b] = hist[b * p.tiles + blockIdx.x];
    for (int w = 0; w < 4; ++w) wcnt[w * bins + b] = 0;
  }
  __syncthreads();
  const int bits = bits_for(bins);
  const int64_t n0 = (int64_t)blockIdx.x * 256 * p.rounds;
  const int64_t n1 = min(p.N, n0 + 256 * (int64_t)p.rounds);
  const int64_t i0 = nodes ? n0 : n0 * p.k, i1 = nodes ? n1 : n1 * p.k;
  for (int64_t i = i0; i < i1; i += 256) {
    const int64_t mine = i + threadIdx.x;
    const bool valid = mine < i1;
    const int key = !valid ? 0 : (nodes ? node_key(p, idx, mine) : expert_of(idx[mine], p.X));
    const int pos = take_places(key, valid, bits, bins, toff, wcnt);
    if (valid) (nodes ? order : slots)[pos] = (int32_t)mine;
  }
}

// Few places: all three steps by one workgroup, 256 places a round, two groupings.  Up to 1024 of them: 256 nodes of 2
// take 5 us in one launch, 9 in three; a workgroup's rounds grow with the places.
constexpr int kFewPlaces = 1024;
__global__ __launch_bounds__(256) void plan_few_kernel(PlanShape p, const int32_t* __restrict__ idx, int32_t* __restrict__ slots,
                                                       int32_t* __restrict__ order, int32_t* __restrict__ ptr) {
  __shared__ int toff[kPlanBins], wcnt[4 * kPlanBins], wsum[4];
  const int t = threadIdx.x, lane = t & 63, wv = t >> 6;
  for (int nodes = 0; nodes < (order ? 2 : 1); ++nodes) {
    const int bins = nodes ? p.bins2 : p.X + 1, count = (int)(nodes ? p.N : p.N * p.k);
    for (int b = t; b < kPlanBins; b += 256) toff[b] = 0;
    for (int b = t; b < 4 * bins; b += 256) wcnt[b] = 0;
    __syncthreads();
    for (int i = t; i < count; i += 256) atomicAdd(&toff[nodes ? node_key(p, idx, i) : expert_of(idx[i], p.X)], 1);
    __syncthreads();
    // exclusive scan of the 1024 bins, four a thread
    int v[4], sum = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[q] = toff[4 * t + q];
      sum += v[q];
    }
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int u = __shfl_up(incl, off, 64);
      if (lane >= off) incl += u;
    }
    if (lane == 63) wsum[wv] = incl;
    __syncthreads();
    int run = incl - sum;
    for (int w = 0; w < wv; ++w) run += wsum[w];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      toff[4 * t + q] = run;
      if (!nodes && 4 * t + q <= p.X) ptr[4 * t + q] = run;
      run += v[q];
    }
    __syncthreads();
    const int bits = bits_for(bins);
    for (int i = 0; i < count; i += 256) {
      const bool valid = i + t < count;
      const int key = !valid ? 0 : (nodes ? node_key(p, idx, i + t) : expert_of(idx[i + t], p.X));
      const int pos = take_places(key, valid, bits, bins, toff, wcnt);
      if (valid) (nodes ? order : slots)[pos] = i + t;
    }
    __syncthreads();
  }
}

hipError_t launch_expert_plan(int64_t N, int k, int X, const int32_t* idx, int32_t* order, int32_t* slots, int32_t* ptr,
                              int32_t* ws, hipStream_t stream) {
  const PlanShape p = plan_shape(N, k, X);
  if (N * k <= kFewPlaces) {
    hipLaunchKernelGGL(plan_few_kernel, dim3(1), dim3(256), 0, stream, p, idx, slots, order, ptr);
    return hipGetLastError();
  }
  int* hist1 = ws;
  int* hist2 = order ? ws + (int64_t)(X + 1) * p.tiles : nullptr;
  hipLaunchKernelGGL(plan_count_kernel, dim3(p.tiles), dim3(256), 0, stream, p, idx, hist1, hist2);
  hipLaunchKernelGGL(plan_scan_kernel, dim3(order ? 2 : 1), dim3(1024), 0, stream, p, hist1, hist2, ptr);
  if (N > 0)
    hipLaunchKernelGGL(plan_place_kernel, dim3(p.tiles, order ? 2 : 1), dim3(256), 0, stream, p, idx, hist1, hist2, slots,
                       order);
  return hipGetLastError();
}

}  // namespace eqtp
