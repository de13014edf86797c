// eqtp_kernels.hpp -- host-side launch interface between the C ABI and the
// kernels.  Arguments are validated by the ABI layer before these are called.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

namespace eqtp {

struct ConvArgs {
  int64_t N, E;
  int lmax, C, path_set, weight_mode, edge_order;
  int x_bf16 = 0;     // x holds bfloat16 features
  int messages = 0;   // edge-aligned kernel: per-edge messages [E, C, K] into out instead of the sum
  bool out_bf16 = false;  // out holds bfloat16 (edges in any order: packed bf16 atomics)
  float r_cut;
  const float* vec;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* row_ptr;
  const float* x;
  const float* w;
  float* out;
  hipStream_t stream;
  // radial edge-aligned kernel: a per-edge basis [E, 64] (stored [E][4][16], hidden unit 4 i + q at
  // q * 16 + i) in place of the radial functions, with w [64, P*C]; else nullptr
  const float* phi = nullptr;
};

struct ProbeArgs {
  int64_t N, E;
  int C, lmax;
  const int32_t* row_ptr;
  const int32_t* src;
  int32_t* count;
  long long* src_sum;
  hipStream_t stream;
};

struct BwdArgs {
  int64_t N, E;
  int lmax, C, path_set;
  const float* vec;
  const int32_t* src;
  const int32_t* dst;      // unsorted edges (row_ptr == nullptr)
  const int32_t* row_ptr;  // dst-sorted edges
  const float* x;
  const float* w;
  const float* gout;
  float* gx;    // or nullptr
  float* gw;    // or nullptr
  float* gvec;  // or nullptr
  int algo = 0;  // grad_vec of sorted edges: 2 = vector-ALU walk, else matrix cores
  float r_cut = 0.0f;  // radial weights: w is [8, P*C] and gw [8, P*C]
  hipStream_t stream;
  // edges grouped by source: row_ptr is the CSR over sources, dst the destinations in that order,
  // perm[i] the input index of grouped edge i (grad_vec is written there)
  bool by_src = false;
  const int32_t* perm = nullptr;
};

// layer norm by degree; with total: of residual + dropout(x), written there
struct NormArgs {
  int64_t N;
  int C, K, lmax;
  bool x_bf16, out_bf16;
  float eps;
  const void* x;
  const void* residual;   // with total
  const int64_t* rng;     // nullptr: nothing is dropped
  uint32_t thr;           // floor(p 2^32)
  float scale;            // 1 / (1 - p)
  const float* weight;    // or nullptr
  const float* bias;      // or nullptr
  void* total;            // or nullptr
  void* out;
  float* stats;           // or nullptr
  hipStream_t stream;
};

struct NormGradArgs {
  int64_t N;
  int C, K, lmax;
  bool x_bf16, out_bf16;
  const void* total;
  const float* stats;
  const float* weight;    // or nullptr
  const void* gout;
  const void* gtotal;     // or nullptr
  const int64_t* rng;     // nullptr: nothing was dropped
  uint32_t thr;
  float scale;
  void* gres;             // or nullptr
  void* gx;               // or nullptr
  float* gw;              // or nullptr
  float* gb;              // or nullptr
  float* ws;              // norm_workspace_floats floats when gw or gb is given
  hipStream_t stream;
};

struct DropArgs {
  int64_t N;
  int C, K;
  bool bf16;
  const void* x;
  const void* residual;   // or nullptr
  const int64_t* rng;     // nullptr: nothing is dropped
  uint32_t thr;
  float scale;
  void* out;
  hipStream_t stream;
};

constexpr int kMaxAttnHeads = 1024;  // heads of q: bounds the grids of the attention's joins

// attention over a graph; head rows of D = (C / heads) K elements
struct AttnArgs {
  int64_t N, M, E;
  int D, heads, kv_heads;
  bool bf16;
  float scale;
  const int32_t* src;
  const int32_t* row_ptr;
  const void* q;
  const void* k;
  const void* v;
  const float* bias;      // or nullptr
  void* out;
  float* lse;             // or nullptr
  void* ws;
  hipStream_t stream;
};

struct AttnGradArgs {
  int64_t N, M, E;
  int D, heads, kv_heads;
  bool bf16;
  float scale;
  const int32_t* src;
  const int32_t* row_ptr;
  const void* q;
  const void* k;
  const void* v;
  const float* bias;      // or nullptr
  const float* lse;
  const void* gout;
  const int32_t* src_ptr; // with gk or gv
  const int32_t* dst_s;
  const int32_t* perm;
  void* gq;               // or nullptr
  void* gk;               // or nullptr
  void* gv;               // or nullptr
  float* gbias;           // or nullptr
  void* ws;
  hipStream_t stream;
};

// bias of the attention's logits by distance buckets (and its gradient: gbias, part)
struct BiasArgs {
  int64_t E;
  int H, B;
  int first_step;         // largest power of four below B (0 for B = 1)
  double cut2;            // square of the cut-off, NaN for none
  const float* vec;
  const float* bounds;    // [B - 1]
  const float* table;
  float* bias;
  const float* gbias;
  float* part;            // bias_workspace_floats floats
  hipStream_t stream;
};
int64_t bias_workspace_floats(int64_t E, int B, int H);
hipError_t launch_distance_bias(const BiasArgs& a);
hipError_t launch_distance_bias_grad(const BiasArgs& a, float* grad_table);

// norm of queries (side 0) and keys (side 1) by head and degree, with the rotation by position (and the gradients)
struct HeadSide {
  int64_t rows;
  int heads;
  bool whole;             // a group of threads takes all heads of a node
  const void* x;
  const float* weight;    // or nullptr
  const float* pos;       // with axes > 0
  void* out;
  const void* gout;
  void* gx;               // or nullptr
  float* gpos;            // or nullptr
  float* part;            // head_norm_workspace_floats floats, or nullptr
};
struct HeadNormArgs {
  int d, K, lmax;         // channels of a head
  bool bf16;
  float eps;
  int axes, R;            // axes of positions (0: no rotation), rotated pairs
  int turns;              // angles that a workgroup holds at a time, at most
  const float* freq;
  HeadSide side[2];
  int blocks_q, blocks_k;
  hipStream_t stream;
};
int64_t head_norm_workspace_floats(int64_t rows, int heads, int d, int lmax);
hipError_t launch_head_norm(const HeadNormArgs& a);
hipError_t launch_head_norm_grad(const HeadNormArgs& a, float* const (&gw)[2]);

// routing
constexpr int kMaxExperts = 256, kMaxTopK = 16;
struct RouteArgs {
  int64_t N;
  int X, k, groups, top_groups;
  bool bf16, sigmoid, renormalise;
  float scale;
  const void* logits;
  const float* bias;      // or nullptr
  int32_t* idx;           // (read by the gradient)
  float* weight;
  const float* gweight;
  void* glogits;
  hipStream_t stream;
};
hipError_t launch_route(const RouteArgs& a);
hipError_t launch_route_grad(const RouteArgs& a);

// the experts' per-degree linears
struct ExpertArgs {
  int64_t N;
  int C, lmax, X, k;
  bool bf16, out_bf16;
  const void* h;          // forward: features; backward: the output's gradient
  const void* W;          // [X, lmax+1, out channel, in channel] as the products take it
  bool as_is;             // very few nodes, backward: the weights as they are, the other way round
  const int32_t* idx;
  const float* weight;    // or nullptr
  const int32_t* order;   // or nullptr
  void* out;              // backward: h's gradient, or nullptr
  const void* dot_with;   // backward: h, for the gates' gradient
  float* gweight;         // or nullptr
  float* part;            // few nodes, with gweight: expert_gate_floats floats
  int64_t places;         // in the order (or rows) from a launch's first one on, where it takes a tile a workgroup
  hipStream_t stream;
};
int64_t expert_gate_floats(int64_t N, int C, int lmax, int k);
hipError_t launch_expert(const ExpertArgs& a);
bool expert_as_is(int64_t N);  // so few nodes that the backward pass takes the weights as they are
hipError_t launch_transpose_weights(int64_t matrices, int C, bool bf16, const void* W, void* WT, hipStream_t stream);
struct ExpertGradArgs {
  int64_t N;
  int C, lmax, X, k;
  bool bf16;
  const void* h;
  const void* gout;
  const float* weight;    // or nullptr
  const int32_t* slots;   // [N k] places n k + j by expert
  const int32_t* ptr;     // [X + 1]
  float* gW;
  float* part;            // expert_grad_floats floats
  hipStream_t stream;
};
int64_t expert_grad_floats(int64_t N, int C, int lmax, int X, int k, bool bf16);
hipError_t launch_expert_grad(const ExpertGradArgs& a);
int64_t expert_plan_ints(int64_t N, int k, int X);
hipError_t launch_expert_plan(int64_t N, int k, int X, const int32_t* idx, int32_t* order, int32_t* slots, int32_t* ptr,
                              int32_t* ws, hipStream_t stream);

int64_t attn_workspace_bytes(int64_t N, int64_t M, int64_t E, int D, int heads, int kv_heads);
hipError_t launch_attention(const AttnArgs& a);
int64_t attn_grad_workspace_bytes(int64_t N, int64_t M, int64_t E, int D, int heads, int kv_heads);
hipError_t launch_attention_grad(const AttnGradArgs& a);
hipError_t launch_norm(const NormArgs& a);
int64_t norm_workspace_floats(int64_t N, int C, int lmax);
hipError_t launch_norm_grad(const NormGradArgs& a);
// out[cols] = the sums of the columns of part [parts][cols], in 64 bits and a fixed order
struct LineSums {
  int cols, parts;  // cols 0: none
  const float* part;
  float* out;
};
hipError_t launch_line_sums(const LineSums& a, const LineSums& b, hipStream_t stream);
hipError_t launch_dropout(const DropArgs& a);
hipError_t launch_sh(const float* vec, int64_t E, int lmax, float* Y, hipStream_t stream);
hipError_t launch_conv_node(const ConvArgs& a);   // sorted edges, fixed weights, matrix cores
hipError_t launch_conv_edge(const ConvArgs& a);   // any order / weights, vector ALUs
hipError_t launch_conv_messages(const ConvArgs& a);  // per-edge messages into out [E, C, K]
hipError_t launch_probe_node(const ProbeArgs& a);
hipError_t launch_probe_edge(const ProbeArgs& a);
// mode 0: fp32 storage and products; 1: bf16 storage and products; 2: fp32 storage, bf16 products
hipError_t launch_linear(int64_t N, int C, int lmax, int mode, const void* h, const void* W, float* out,
                         hipStream_t stream);
// compute units of the current device (cached per device)
int num_cus();
hipError_t launch_fill_zero(float* p, int64_t n, hipStream_t stream);
// graph checks: kCheckWords int32 of counts and first offending indices into report (check.hip)
constexpr int kCheckWords = 8;
hipError_t launch_check_graph(int64_t N, int64_t E, const int32_t* row_ptr, const int32_t* src, const int32_t* dst,
                              const float* vec, int32_t* report, hipStream_t stream);
hipError_t launch_conv_backward(const BwdArgs& a);   // fixed weights, vector ALUs
hipError_t launch_conv_backward_radial(const BwdArgs& a);  // radial weights, lmax <= 3, C a multiple of 16
// the interaction layer's radial network: phi [E][4][16] (scaled by scale) from the edge lengths
hipError_t launch_radial_mlp(int64_t E, const float* vec, float r_cut, const float* W1, const float* W2, float* phi,
                             float scale, hipStream_t stream);
// edge-aligned (SO(2)) form, lmax 0..6, fixed fp32 weights, any C; C = 128 runs as two 64-channel halves from
// lmax 4 (forward, messages) or lmax 3 (gradients)
constexpr int kSo2MaxL = 6;
hipError_t launch_conv_so2(const ConvArgs& a);
// gradients in the edge-aligned form: fixed weights, lmax 0..6, any edge order (row_ptr or dst)
hipError_t launch_conv_backward_so2(const BwdArgs& a);
// edge-aligned form with radial weights on dst-sorted edges: lmax 0..3, C = 16, 32, 64 or 128
hipError_t launch_conv_so2_radial(const ConvArgs& a);
// grad_x / grad_w on the matrix cores from edges grouped by source: row_ptr =
// CSR over sources, vec / dst in that order (src unused)
hipError_t launch_conv_backward_by_source(const BwdArgs& a);
hipError_t launch_edge_rows(int64_t N, int64_t E, const int32_t* row_ptr, int32_t* rows, hipStream_t stream);
hipError_t launch_sort_edges(int64_t N, int64_t E, const int32_t* dst, const float* vec, const int32_t* src,
                             int32_t* row_ptr, int32_t* perm, float* vec_out, int32_t* src_out, hipStream_t stream);
// grouping by destination with each row in input order: staged [E] int32 scratch; vec_out, src_out required
// stable grouping by destination (LSD radix sort) for the workspace convolution: row_ptr [N+1], the sorted
// keys and edge indices end in keys_a / vals_a (keys_b / vals_b: the other buffers of the passes, hist:
// radix_hist_entries(E) ints); vec_out [E,3] / src_out [E] in that order, each may be null (vec_out may
// span keys_a..vals_b when they are laid out in that order and hold 12 E bytes; it must not overlap vals_a)
int64_t radix_hist_entries(int64_t E);
hipError_t launch_sort_edges_stable(int64_t N, int64_t E, const int32_t* dst, const float* vec, const int32_t* src,
                                    int32_t* row_ptr, int32_t* keys_a, int32_t* vals_a, int32_t* keys_b,
                                    int32_t* vals_b, int32_t* hist, float* vec_out, int32_t* src_out,
                                    hipStream_t stream);

}  // namespace eqtp
