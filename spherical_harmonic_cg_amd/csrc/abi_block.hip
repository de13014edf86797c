// abi_block.hip -- the extern "C" entry points of what stands before and behind
// the attention: the distance bias, the norm and rotation of queries and keys,
// routing and the experts' linears.
#include <math.h>
#include <stdint.h>

#include "abi_checks.hpp"
#include "eqtp_device.hpp"
#include "eqtp_kernels.hpp"

namespace {

constexpr int kMaxLmax = 6;
constexpr int kMaxBuckets = 512, kMaxHeads = 1024, kMaxRow = 2048, kMaxAxes = 3;

int bias_check(const eqtp_bias_desc* d, int64_t E) {
  if (!d || d->struct_size != (int32_t)sizeof(eqtp_bias_desc)) return EQTP_EINVAL;
  if (d->heads <= 0 || d->buckets <= 0 || E < 0 || E > kMaxIndex) return EQTP_EINVAL;
  if (!(d->r_cut >= 0.0f)) return EQTP_EINVAL;  // NaN, too
  if (d->heads > kMaxHeads || d->buckets > kMaxBuckets) return EQTP_EUNSUPPORTED;
  return EQTP_OK;
}

eqtp::BiasArgs bias_args(const eqtp_bias_desc* d, int64_t E, const float* vec, const float* bounds, void* stream) {
  eqtp::BiasArgs a = {};
  a.E = E;
  a.H = d->heads;
  a.B = d->buckets;
  for (int s = 1; s < d->buckets; s *= 4) a.first_step = s;
  a.cut2 = d->r_cut > 0.0f ? (double)d->r_cut * (double)d->r_cut : NAN;
  a.vec = vec;
  a.bounds = bounds;
  a.stream = (hipStream_t)stream;
  return a;
}

int qk_check(const eqtp_qk_norm_desc* d, int64_t N, int64_t M) {
  if (!d || d->struct_size != (int32_t)sizeof(eqtp_qk_norm_desc)) return EQTP_EINVAL;
  if (d->lmax < 0 || d->C <= 0 || d->heads <= 0 || d->kv_heads <= 0 || !dtype_ok(d->x_dtype)) return EQTP_EINVAL;
  if (d->C % d->heads != 0 || !(d->eps > 0.0f) || d->eps > 3.4028235e38f) return EQTP_EINVAL;
  if (N < 0 || M < 0 || N > kMaxIndex || M > kMaxIndex) return EQTP_EINVAL;
  const int width = d->C / d->heads;
  if (d->axes < 0 || d->pairs < 0 || (d->axes == 0) != (d->pairs == 0)) return EQTP_EINVAL;
  if (d->pairs > 0 && (width % 2 != 0 || d->pairs > width / 2)) return EQTP_EINVAL;
  if (d->lmax > kMaxLmax || (int64_t)width * eqtp::num_comp(d->lmax) > kMaxRow || d->heads > kMaxHeads ||
      d->kv_heads > kMaxHeads || d->axes > kMaxAxes)
    return EQTP_EUNSUPPORTED;
  return EQTP_OK;
}

eqtp::HeadNormArgs qk_args(const eqtp_qk_norm_desc* d, int64_t N, int64_t M, const void* q, const void* k,
                           const float* weight_q, const float* weight_k, const float* pos_q, const float* pos_k,
                           const float* freq, void* stream) {
  eqtp::HeadNormArgs a = {};
  a.d = d->C / d->heads;
  a.lmax = d->lmax;
  a.K = eqtp::num_comp(d->lmax);
  a.bf16 = d->x_dtype == EQTP_BF16;
  a.eps = d->eps;
  a.axes = d->axes;
  a.R = d->pairs;
  a.freq = freq;
  a.side[0].rows = N;
  a.side[0].heads = d->heads;
  a.side[0].x = q;
  a.side[0].weight = weight_q;
  a.side[0].pos = pos_q;
  a.side[1].rows = M;
  a.side[1].heads = d->kv_heads;
  a.side[1].x = k;
  a.side[1].weight = weight_k;
  a.side[1].pos = pos_k;
  a.stream = (hipStream_t)stream;
  return a;
}

int64_t qk_floats(const eqtp_qk_norm_desc* d, int64_t rows, int heads) {
  return (eqtp::head_norm_workspace_floats(rows, heads, d->C / d->heads, d->lmax) + 3) / 4 * 4;
}

int route_check(const eqtp_route_desc* d, int64_t N) {
  if (!d || d->struct_size != (int32_t)sizeof(eqtp_route_desc)) return EQTP_EINVAL;
  if (d->experts <= 0 || d->top_k <= 0 || d->groups <= 0 || d->top_groups <= 0 || !dtype_ok(d->x_dtype)) return EQTP_EINVAL;
  if (d->top_k > d->experts || d->experts % d->groups != 0 || d->top_groups > d->groups) return EQTP_EINVAL;
  if (d->score != EQTP_SCORE_SOFTMAX && d->score != EQTP_SCORE_SIGMOID) return EQTP_EINVAL;
  if (d->renormalise != 0 && d->renormalise != 1) return EQTP_EINVAL;
  if (!(d->scale >= -3.4028235e38f && d->scale <= 3.4028235e38f)) return EQTP_EINVAL;
  if (N < 0 || N > kMaxIndex) return EQTP_EINVAL;
  if (d->experts > eqtp::kMaxExperts || d->top_k > eqtp::kMaxTopK) return EQTP_EUNSUPPORTED;
  return EQTP_OK;
}

eqtp::RouteArgs route_args(const eqtp_route_desc* d, int64_t N, const void* logits, void* stream) {
  eqtp::RouteArgs a = {};
  a.N = N;
  a.X = d->experts;
  a.k = d->top_k;
  a.groups = d->groups;
  a.top_groups = d->top_groups;
  a.bf16 = d->x_dtype == EQTP_BF16;
  a.sigmoid = d->score == EQTP_SCORE_SIGMOID;
  a.renormalise = d->renormalise != 0;
  a.scale = d->scale;
  a.logits = logits;
  a.stream = (hipStream_t)stream;
  return a;
}

int plan_check(int64_t N, int top_k, int experts) {
  if (N < 0 || top_k <= 0 || experts <= 0 || N > kMaxIndex || N * top_k > kMaxIndex) return EQTP_EINVAL;
  if (experts > eqtp::kMaxExperts || top_k > eqtp::kMaxTopK) return EQTP_EUNSUPPORTED;
  return EQTP_OK;
}

int expert_check(const eqtp_expert_desc* d, int64_t N) {
  if (!d || d->struct_size != (int32_t)sizeof(eqtp_expert_desc)) return EQTP_EINVAL;
  if (d->lmax < 0 || d->C <= 0 || !dtype_ok(d->x_dtype) || !dtype_ok(d->out_dtype)) return EQTP_EINVAL;
  const int rc = plan_check(N, d->top_k, d->experts);
  if (rc != EQTP_OK) return rc;
  if (d->lmax > kMaxLmax || !valid_c(d->C)) return EQTP_EUNSUPPORTED;
  return EQTP_OK;
}

int64_t expert_weights(const eqtp_expert_desc* d) { return (int64_t)d->experts * (d->lmax + 1) * d->C * d->C; }
// the workspace of the backward pass: transposed weights, parts of the gates' gradient, the weight gradient's lines
struct ExpertWs {
  int64_t gates, lines, total;
};
ExpertWs expert_ws(const eqtp_expert_desc* d, int64_t N) {
  auto al = [](int64_t b) { return (b + 255) / 256 * 256; };
  const bool bf16 = d->x_dtype == EQTP_BF16;
  ExpertWs w;
  w.gates = eqtp::expert_as_is(N) ? 0 : al(expert_weights(d) * (bf16 ? 2 : 4));
  w.lines = w.gates + al(4 * eqtp::expert_gate_floats(N, d->C, d->lmax, d->top_k));
  w.total = w.lines + 4 * eqtp::expert_grad_floats(N, d->C, d->lmax, d->experts, d->top_k, bf16);
  if (w.total < 16) w.total = 16;
  return w;
}

}  // namespace

extern "C" {

int eqtp_distance_bias(const eqtp_bias_desc* d, int64_t E, const float* vec, const float* bounds, const float* table,
                       float* bias, void* stream) {
  const int rc = bias_check(d, E);
  if (rc != EQTP_OK) return rc;
  if (E == 0) return EQTP_OK;
  if (!vec || !table || !bias || (!bounds && d->buckets > 1)) return EQTP_EINVAL;
  if (!aligned4(vec) || !aligned4(bounds) || !aligned4(table) || !aligned4(bias)) return EQTP_EINVAL;
  eqtp::BiasArgs a = bias_args(d, E, vec, bounds, stream);
  a.table = table;
  a.bias = bias;
  return status_of(eqtp::launch_distance_bias(a));
}

int64_t eqtp_distance_bias_workspace_bytes(const eqtp_bias_desc* d, int64_t E) {
  const int rc = bias_check(d, E);
  if (rc != EQTP_OK) return -rc;
  return eqtp::bias_workspace_floats(E, d->buckets, d->heads) * 4;
}

int eqtp_distance_bias_backward(const eqtp_bias_desc* d, int64_t E, const float* vec, const float* bounds,
                                const float* grad_bias, float* grad_table, void* workspace, int64_t workspace_bytes,
                                void* stream) {
  const int rc = bias_check(d, E);
  if (rc != EQTP_OK) return rc;
  if (!grad_table || !aligned4(grad_table) || !aligned4(vec) || !aligned4(bounds) || !aligned4(grad_bias)) return EQTP_EINVAL;
  if (E > 0 && (!vec || !grad_bias || (!bounds && d->buckets > 1))) return EQTP_EINVAL;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < eqtp::bias_workspace_floats(E, d->buckets, d->heads) * 4)
    return EQTP_EINVAL;
  eqtp::BiasArgs a = bias_args(d, E, vec, bounds, stream);
  a.gbias = grad_bias;
  a.part = static_cast<float*>(workspace);
  return status_of(eqtp::launch_distance_bias_grad(a, grad_table));
}

int eqtp_qk_norm(const eqtp_qk_norm_desc* d, int64_t N, int64_t M, const void* q, const void* k, const float* weight_q,
                 const float* weight_k, const float* pos_q, const float* pos_k, const float* freq, void* out_q,
                 void* out_k, void* stream) {
  const int rc = qk_check(d, N, M);
  if (rc != EQTP_OK) return rc;
  const int t = d->x_dtype;
  if (!aligned_as(q, t) || !aligned_as(k, t) || !aligned_as(out_q, t) || !aligned_as(out_k, t) || !aligned4(weight_q) ||
      !aligned4(weight_k) || !aligned4(pos_q) || !aligned4(pos_k) || !aligned4(freq))
    return EQTP_EINVAL;
  if (N == 0 && M == 0) return EQTP_OK;
  if ((N > 0 && (!q || !out_q)) || (M > 0 && (!k || !out_k))) return EQTP_EINVAL;
  if (d->axes > 0 && (!freq || (N > 0 && !pos_q) || (M > 0 && !pos_k))) return EQTP_EINVAL;
  eqtp::HeadNormArgs a = qk_args(d, N, M, q, k, weight_q, weight_k, pos_q, pos_k, freq, stream);
  a.side[0].out = out_q;
  a.side[1].out = out_k;
  return status_of(eqtp::launch_head_norm(a));
}

int64_t eqtp_qk_norm_workspace_bytes(const eqtp_qk_norm_desc* d, int64_t N, int64_t M) {
  const int rc = qk_check(d, N, M);
  if (rc != EQTP_OK) return -rc;
  return 4 * (qk_floats(d, N, d->heads) + qk_floats(d, M, d->kv_heads));
}

int eqtp_qk_norm_backward(const eqtp_qk_norm_desc* d, int64_t N, int64_t M, const void* q, const void* k,
                          const float* weight_q, const float* weight_k, const float* pos_q, const float* pos_k,
                          const float* freq, const void* grad_out_q, const void* grad_out_k, void* grad_q, void* grad_k,
                          float* grad_weight_q, float* grad_weight_k, float* grad_pos_q, float* grad_pos_k,
                          void* workspace, int64_t workspace_bytes, void* stream) {
  const int rc = qk_check(d, N, M);
  if (rc != EQTP_OK) return rc;
  const int t = d->x_dtype;
  if (!aligned_as(q, t) || !aligned_as(k, t) || !aligned_as(grad_out_q, t) || !aligned_as(grad_out_k, t) ||
      !aligned_as(grad_q, t) || !aligned_as(grad_k, t) || !aligned4(weight_q) || !aligned4(weight_k) || !aligned4(pos_q) ||
      !aligned4(pos_k) || !aligned4(freq) || !aligned4(grad_weight_q) || !aligned4(grad_weight_k) || !aligned4(grad_pos_q) ||
      !aligned4(grad_pos_k))
    return EQTP_EINVAL;
  if ((grad_pos_q || grad_pos_k) && d->axes == 0) return EQTP_EINVAL;
  const bool need_q = grad_q || grad_weight_q || grad_pos_q, need_k = grad_k || grad_weight_k || grad_pos_k;
  if ((need_q && N > 0 && (!q || !grad_out_q)) || (need_k && M > 0 && (!k || !grad_out_k))) return EQTP_EINVAL;
  if (d->axes > 0 && ((need_q && N > 0 && (!pos_q || !freq)) || (need_k && M > 0 && (!pos_k || !freq)))) return EQTP_EINVAL;
  const int64_t fq = qk_floats(d, N, d->heads), fk = qk_floats(d, M, d->kv_heads);
  if ((grad_weight_q || grad_weight_k) && (!workspace || !aligned16(workspace) || workspace_bytes < 4 * (fq + fk)))
    return EQTP_EINVAL;
  // a side that nothing is asked of has no rows to walk over
  eqtp::HeadNormArgs a = qk_args(d, need_q ? N : 0, need_k ? M : 0, q, k, weight_q, weight_k, pos_q, pos_k, freq, stream);
  a.side[0].gout = grad_out_q;
  a.side[1].gout = grad_out_k;
  a.side[0].gx = grad_q;
  a.side[1].gx = grad_k;
  a.side[0].gpos = grad_pos_q;
  a.side[1].gpos = grad_pos_k;
  a.side[0].part = grad_weight_q ? static_cast<float*>(workspace) : nullptr;
  a.side[1].part = grad_weight_k ? static_cast<float*>(workspace) + fq : nullptr;
  float* const gw[2] = {grad_weight_q, grad_weight_k};
  return status_of(eqtp::launch_head_norm_grad(a, gw));
}

int eqtp_route(const eqtp_route_desc* d, int64_t N, const void* logits, const float* bias, int32_t* idx, float* weight,
               void* stream) {
  const int rc = route_check(d, N);
  if (rc != EQTP_OK) return rc;
  if (N == 0) return EQTP_OK;
  if (!logits || !idx || !weight || !aligned_as(logits, d->x_dtype) || !aligned4(bias) || !aligned4(idx) || !aligned4(weight))
    return EQTP_EINVAL;
  eqtp::RouteArgs a = route_args(d, N, logits, stream);
  a.bias = bias;
  a.idx = idx;
  a.weight = weight;
  return status_of(eqtp::launch_route(a));
}

int eqtp_route_backward(const eqtp_route_desc* d, int64_t N, const void* logits, const int32_t* idx,
                        const float* grad_weight, void* grad_logits, void* stream) {
  const int rc = route_check(d, N);
  if (rc != EQTP_OK) return rc;
  if (N == 0) return EQTP_OK;
  if (!logits || !idx || !grad_weight || !grad_logits || !aligned_as(logits, d->x_dtype) || !aligned4(idx) ||
      !aligned4(grad_weight) || !aligned_as(grad_logits, d->x_dtype))
    return EQTP_EINVAL;
  eqtp::RouteArgs a = route_args(d, N, logits, stream);
  a.idx = const_cast<int32_t*>(idx);
  a.gweight = grad_weight;
  a.glogits = grad_logits;
  return status_of(eqtp::launch_route_grad(a));
}

int64_t eqtp_expert_plan_workspace_bytes(int64_t N, int top_k, int experts) {
  const int rc = plan_check(N, top_k, experts);
  if (rc != EQTP_OK) return -rc;
  return 4 * eqtp::expert_plan_ints(N, top_k, experts);
}

int eqtp_expert_plan(int64_t N, int top_k, int experts, const int32_t* idx, int32_t* order, int32_t* slots, int32_t* ptr,
                     void* workspace, int64_t workspace_bytes, void* stream) {
  const int rc = plan_check(N, top_k, experts);
  if (rc != EQTP_OK) return rc;
  if (!ptr || !aligned4(ptr) || !aligned4(idx) || !aligned4(order) || !aligned4(slots)) return EQTP_EINVAL;
  if (N > 0 && (!idx || !slots)) return EQTP_EINVAL;
  if (!workspace || !aligned16(workspace) || workspace_bytes < 4 * eqtp::expert_plan_ints(N, top_k, experts)) return EQTP_EINVAL;
  return status_of(eqtp::launch_expert_plan(N, top_k, experts, idx, order, slots, ptr, static_cast<int32_t*>(workspace),
                                            (hipStream_t)stream));
}

int eqtp_expert_linear(const eqtp_expert_desc* d, int64_t N, const void* h, const void* W, const int32_t* idx,
                       const float* weight, const int32_t* order, void* out, void* stream) {
  const int rc = expert_check(d, N);
  if (rc != EQTP_OK) return rc;
  if (N == 0) return EQTP_OK;
  if (!h || !W || !idx || !out || !aligned16(h) || !aligned16(W) || !aligned16(out) || !aligned4(idx) || !aligned4(weight) ||
      !aligned4(order))
    return EQTP_EINVAL;
  eqtp::ExpertArgs a = {};
  a.N = N;
  a.C = d->C;
  a.lmax = d->lmax;
  a.X = d->experts;
  a.k = d->top_k;
  a.bf16 = d->x_dtype == EQTP_BF16;
  a.out_bf16 = d->out_dtype == EQTP_BF16;
  a.h = h;
  a.W = W;
  a.idx = idx;
  a.weight = weight;
  a.order = order;
  a.out = out;
  a.stream = (hipStream_t)stream;
  return status_of(eqtp::launch_expert(a));
}

int64_t eqtp_expert_linear_backward_workspace_bytes(const eqtp_expert_desc* d, int64_t N) {
  const int rc = expert_check(d, N);
  if (rc != EQTP_OK) return -rc;
  return expert_ws(d, N).total;
}

int eqtp_expert_linear_backward(const eqtp_expert_desc* d, int64_t N, const void* h, const void* W, const int32_t* idx,
                                const float* weight, const int32_t* order, const int32_t* slots, const int32_t* ptr,
                                const void* grad_out, void* grad_h, float* grad_W, float* grad_weight, void* workspace,
                                int64_t workspace_bytes, void* stream) {
  const int rc = expert_check(d, N);
  if (rc != EQTP_OK) return rc;
  if (!aligned16(h) || !aligned16(W) || !aligned16(grad_out) || !aligned16(grad_h) || !aligned16(grad_W) ||
      !aligned4(idx) || !aligned4(weight) || !aligned4(order) || !aligned4(slots) || !aligned4(ptr) || !aligned4(grad_weight))
    return EQTP_EINVAL;
  const bool bf16 = d->x_dtype == EQTP_BF16, rows = grad_h || grad_weight;
  if (N > 0 && !grad_h && !grad_W && !grad_weight) return EQTP_EINVAL;
  if (N > 0 && (!grad_out || (rows && (!W || !idx)) || ((grad_W || grad_weight) && !h))) return EQTP_EINVAL;
  if (grad_W && (!ptr || (N > 0 && !slots))) return EQTP_EINVAL;
  const ExpertWs ws = expert_ws(d, N);
  if (!workspace || !aligned16(workspace) || workspace_bytes < ws.total) return EQTP_EINVAL;
  unsigned char* base = static_cast<unsigned char*>(workspace);
  const hipStream_t st = (hipStream_t)stream;
  if (rows && N > 0) {
    const bool as_is = eqtp::expert_as_is(N);
    if (!as_is) {
      const int rt = status_of(eqtp::launch_transpose_weights((int64_t)d->experts * (d->lmax + 1), d->C, bf16, W, workspace, st));
      if (rt != EQTP_OK) return rt;
    }
    eqtp::ExpertArgs a = {};
    a.N = N;
    a.C = d->C;
    a.lmax = d->lmax;
    a.X = d->experts;
    a.k = d->top_k;
    a.bf16 = bf16;
    a.out_bf16 = bf16;
    a.h = grad_out;
    a.W = as_is ? W : workspace;
    a.as_is = as_is;
    a.idx = idx;
    a.weight = weight;
    a.order = order;
    a.out = grad_h;
    a.dot_with = h;
    a.gweight = grad_weight;
    a.part = reinterpret_cast<float*>(base + ws.gates);
    a.stream = st;
    const int rg = status_of(eqtp::launch_expert(a));
    if (rg != EQTP_OK) return rg;
  }
  if (!grad_W) return EQTP_OK;
  eqtp::ExpertGradArgs g = {};
  g.N = N;
  g.C = d->C;
  g.lmax = d->lmax;
  g.X = d->experts;
  g.k = d->top_k;
  g.bf16 = bf16;
  g.h = h;
  g.gout = grad_out;
  g.weight = weight;
  g.slots = slots;
  g.ptr = ptr;
  g.gW = grad_W;
  g.part = reinterpret_cast<float*>(base + ws.lines);
  g.stream = st;
  return status_of(eqtp::launch_expert_grad(g));
}

}  // extern "C"
