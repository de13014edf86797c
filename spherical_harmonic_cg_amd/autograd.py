"""PyTorch autograd wrappers of the fused convolution and of the parts of a
transformer block around it (norm, dropout, attention).

The forward calls eqtp_conv_fused.  The backward groups the edges by source
node on the GPU (eqtp_edge_rows, eqtp_sort_edges) so that grad_x is summed per
source without atomics, and
  * with fixed weights at lmax <= 3: grad_x and grad_w with
    eqtp_conv_backward_by_source (the adjoint of the node-factored forward, on
    the matrix cores) and grad_vec (for forces) with eqtp_conv_backward;
  * with radial weights (weight_mode = EQTP_W_RADIAL) or above lmax 3: all
    three with eqtp_conv_backward_by_source (one walk in each edge's frame;
    grad_vec back in the caller's edge order through the sort's permutation).
``grad_x_mode="edge"`` takes all three from eqtp_conv_backward on the edges as
given instead (grad_x by fp32 atomics).  All arithmetic runs in the HIP
library; this module only marshals arguments.

equivariant_layer_norm, equivariant_dropout, dropout_add_norm and
graph_attention keep what their backward calls need: the norm its input and
(lmax+2) numbers a node, dropout two integers (the mask is made again), the
attention q, k, v and one number a row and head.  Each takes its gradients
from entry points that give the same bits from call to call.  Their backward
passes cannot be differentiated again.  A forward pass that is run again
(activation checkpointing) reads rng again: it must still hold what it held
the first time, or the activations made then belong to another mask than the
output did, and no error says so.  Do not move one rng along between places;
give each place of a step a row of its own, made from seed and offset before
the step and left alone until its backward pass is over:
    places = torch.stack((rng[0].expand(n), rng[1] + torch.arange(n, device=rng.device)), 1)
To capture a training step into a
graph, drop every eager graph over the same leaves first (torch ends the
process when a captured backward pass meets one).
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import eqtp as _eq


def group_by_source(N: int, src, vec, dst=None, row_ptr=None, with_perm: bool = False):
    """(src_ptr [N+1], vec_s [E,3], dst_s [E]) and, with_perm, perm [E] (the
    caller's index of each grouped edge): the edges grouped by source node (the
    input of eqtp_conv_backward_by_source), each source's edges in input order,
    so grad_x, summed per source over them, is the same from call to call.
    Destinations come from dst, or from a dst-sorted CSR (row_ptr)."""
    E = src.shape[0]
    if dst is None:
        dst = _eq.eqtp_edge_rows(row_ptr, E)
    src_ptr, perm, vec_s, dst_s = _eq.eqtp_sort_edges_stable(src, N, vec=vec, src=dst)
    return (src_ptr, vec_s, dst_s, perm) if with_perm else (src_ptr, vec_s, dst_s)


class EquivariantConvFunction(torch.autograd.Function):
    """out = conv(vec, x, weights) over dst-sorted (row_ptr) or unsorted (dst) edges."""

    @staticmethod
    def forward(ctx, vec, x, weights, src, row_ptr, dst, lmax, path_set, grad_x_mode, weight_mode=_eq.EQTP_W_FIXED,
                r_cut=0.0):
        out = _eq.eqtp_conv_fused(vec, src, x, weights, lmax, row_ptr=row_ptr, dst=dst, path_set=path_set,
                                  weight_mode=weight_mode, r_cut=r_cut)
        ctx.save_for_backward(vec, x, weights, src, row_ptr, dst)
        ctx.lmax = lmax
        ctx.path_set = path_set
        ctx.grad_x_mode = grad_x_mode
        ctx.weight_mode = weight_mode
        ctx.r_cut = r_cut
        return out

    @staticmethod
    def backward(ctx, grad_out):
        vec, x, weights, src, row_ptr, dst = ctx.saved_tensors
        need_vec, need_x, need_w = ctx.needs_input_grad[0], ctx.needs_input_grad[1], ctx.needs_input_grad[2]
        g = grad_out.contiguous()
        gx = gw = gv = None
        walk = ctx.weight_mode == _eq.EQTP_W_RADIAL or ctx.lmax > 3  # one walk over the edges gives all three
        if walk and ctx.grad_x_mode == "by_source":
            if need_vec or need_x or need_w:
                src_ptr, vec_s, dst_s, perm = group_by_source(x.shape[0], src, vec, dst=dst, row_ptr=row_ptr,
                                                              with_perm=True)
                gx, gw, gv = _eq.eqtp_conv_backward_by_source(vec_s, dst_s, src_ptr, x, weights, g, ctx.lmax,
                                                              path_set=ctx.path_set, need_x=need_x, need_w=need_w,
                                                              need_vec=need_vec, perm=perm,
                                                              weight_mode=ctx.weight_mode, r_cut=ctx.r_cut)
        elif walk:
            if need_vec or need_x or need_w:
                gx, gw, gv = _eq.eqtp_conv_backward(vec, src, x, weights, g, ctx.lmax, row_ptr=row_ptr, dst=dst,
                                                    path_set=ctx.path_set, need_x=need_x, need_w=need_w,
                                                    need_vec=need_vec, weight_mode=ctx.weight_mode,
                                                    r_cut=ctx.r_cut)
        elif ctx.grad_x_mode == "edge":
            if need_vec or need_x or need_w:
                gx, gw, gv = _eq.eqtp_conv_backward(vec, src, x, weights, g, ctx.lmax, row_ptr=row_ptr, dst=dst,
                                                    path_set=ctx.path_set, need_x=need_x, need_w=need_w,
                                                    need_vec=need_vec)
        else:
            if need_x or need_w:
                src_ptr, vec_s, dst_s = group_by_source(x.shape[0], src, vec, dst=dst, row_ptr=row_ptr)
                gx, gw, _ = _eq.eqtp_conv_backward_by_source(vec_s, dst_s, src_ptr, x, weights, g, ctx.lmax,
                                                          path_set=ctx.path_set, need_x=need_x, need_w=need_w)
            if need_vec:
                _, _, gv = _eq.eqtp_conv_backward(vec, src, x, weights, g, ctx.lmax, row_ptr=row_ptr, dst=dst,
                                                  path_set=ctx.path_set, need_x=False, need_w=False, need_vec=True)
        return gv, gx, gw, None, None, None, None, None, None, None, None


def equivariant_conv(vec, x, weights, src, lmax: int, row_ptr=None, dst=None, path_set: int = _eq.EQTP_PATHS_PARITY,
                     grad_x_mode: str = "by_source", weight_mode: int = _eq.EQTP_W_FIXED, r_cut: float = 0.0):
    """Differentiable fused convolution (see eqtp_conv_fused for the layouts).
    grad_x_mode: "by_source" (default) or "edge" (see the module docstring).
    weight_mode=EQTP_W_RADIAL: weights [8, P*C] applied through the radial basis of cut-off r_cut."""
    if grad_x_mode not in ("by_source", "edge"):
        raise ValueError("grad_x_mode must be 'by_source' or 'edge'")
    return EquivariantConvFunction.apply(vec, x, weights, src, row_ptr, dst, lmax, path_set, grad_x_mode,
                                         weight_mode, r_cut)


def _dense(t):
    return t if t is None or t.is_contiguous() else t.contiguous()


class EquivariantLayerNormFunction(torch.autograd.Function):
    """out = layer norm by degree of x."""

    @staticmethod
    def forward(ctx, x, weight, bias, lmax, eps, out_dtype):
        stats = torch.empty((x.shape[0], lmax + 2), dtype=torch.float32, device=x.device)
        out = _eq.eqtp_layer_norm(x, lmax, weight, bias, eps=eps, out_dtype=out_dtype, stats=stats)
        ctx.save_for_backward(x, stats, weight)
        ctx.lmax = lmax
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        x, stats, weight = ctx.saved_tensors
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        if not (need_x or need_w or need_b):
            return (None,) * 6
        gx, _, gw, gb = _eq.eqtp_layer_norm_backward(x, stats, _dense(grad_out), ctx.lmax, weight,
                                                     need_residual=need_x, need_weight=need_w, need_bias=need_b)
        return gx, gw, gb, None, None, None


class EquivariantDropoutFunction(torch.autograd.Function):
    """out = residual + dropout(x) of whole channels."""

    @staticmethod
    def forward(ctx, x, residual, rng, p, lmax):
        # the values of rng now: the caller may move the offset on before the backward pass
        ctx.rng = rng.clone() if rng is not None and p > 0.0 else None
        ctx.p, ctx.lmax = p, lmax
        return _eq.eqtp_dropout(x, rng, p, lmax, residual=residual)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        gx = _eq.eqtp_dropout(_dense(grad_out), ctx.rng, ctx.p, ctx.lmax) if ctx.needs_input_grad[0] else None
        return gx, grad_out if ctx.needs_input_grad[1] else None, None, None, None


class DropoutAddNormFunction(torch.autograd.Function):
    """(out, total): total = residual + dropout(x), out = layer norm by degree of total."""

    @staticmethod
    def forward(ctx, x, residual, weight, bias, rng, p, lmax, eps, out_dtype):
        stats = torch.empty((x.shape[0], lmax + 2), dtype=torch.float32, device=x.device)
        out, total = _eq.eqtp_dropout_add_norm(x, residual, rng, p, lmax, weight, bias, eps=eps, out_dtype=out_dtype,
                                               stats=stats)
        ctx.rng = rng.clone() if rng is not None and p > 0.0 else None
        ctx.save_for_backward(total, stats, weight)
        ctx.p, ctx.lmax = p, lmax
        ctx.set_materialize_grads(False)
        return out, total

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out, grad_total):
        total, stats, weight = ctx.saved_tensors
        need_x, need_r, need_w, need_b = ctx.needs_input_grad[:4]
        none = (None,) * 5
        if grad_out is None:  # only total was used
            gx = gr = None
            if grad_total is not None:
                grad_total = _dense(grad_total)
                gr = grad_total if need_r else None
                gx = _eq.eqtp_dropout(grad_total, ctx.rng, ctx.p, ctx.lmax) if need_x else None
            return (gx, gr, None, None) + none
        if not (need_x or need_r or need_w or need_b):
            return (None,) * 4 + none
        gr, gx, gw, gb = _eq.eqtp_layer_norm_backward(total, stats, _dense(grad_out), ctx.lmax, weight,
                                                      grad_total=_dense(grad_total), rng=ctx.rng, p=ctx.p,
                                                      need_residual=need_r, need_x=need_x, need_weight=need_w,
                                                      need_bias=need_b)
        return (gx, gr, gw, gb) + none


class GraphAttentionFunction(torch.autograd.Function):
    """out = attention of q's rows over the edges of a dst-sorted graph."""

    @staticmethod
    def forward(ctx, q, k, v, bias, src, row_ptr, lmax, heads, scale, plan):
        scale = None if scale is None else float(scale)  # its value now, for both passes
        lse = torch.empty((q.shape[0], heads), dtype=torch.float32, device=q.device)
        out = _eq.eqtp_attention(q, k, v, src, row_ptr, lmax, heads, scale=scale, bias=bias, lse=lse)
        ctx.save_for_backward(q, k, v, bias, src, row_ptr, lse, *(plan if plan is not None else ()))
        ctx.lmax, ctx.heads, ctx.scale = lmax, heads, scale
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        q, k, v, bias, src, row_ptr, lse = ctx.saved_tensors[:7]
        plan = ctx.saved_tensors[7:]
        need_q, need_k, need_v, need_b = ctx.needs_input_grad[:4]
        if not (need_q or need_k or need_v or need_b):
            return (None,) * 10
        if need_k or need_v:
            src_ptr, dst_s, perm = plan if len(plan) == 3 else attention_plan(src, row_ptr, k.shape[0])
        else:
            src_ptr = dst_s = perm = None
        gq, gk, gv, gb = _eq.eqtp_attention_backward(q, k, v, src, row_ptr, lse, _dense(grad_out), src_ptr, dst_s, perm,
                                                     ctx.lmax, ctx.heads, scale=ctx.scale, bias=bias, need_q=need_q,
                                                     need_k=need_k, need_v=need_v, need_bias=need_b)
        return gq, gk, gv, gb, None, None, None, None, None, None


def attention_plan(src, row_ptr, M: int):
    """(src_ptr [M+1], dst_s [E], perm [E]): the edges grouped by source, what graph_attention's backward pass needs;
    made once, it serves every layer and step over the same graph."""
    rows = _eq.eqtp_edge_rows(row_ptr, src.shape[0])
    # the grouping could carry the rows along, but takes what it carries for nodes below M: debug mode would refuse them
    src_ptr, perm, _, _ = _eq.eqtp_sort_edges_stable(src, M)
    return src_ptr, rows.index_select(0, perm), perm


def equivariant_layer_norm(x, lmax: int, weight=None, bias=None, eps: float = 1e-5, out_dtype: int = None):
    """Differentiable layer norm by degree (see eqtp_layer_norm)."""
    return EquivariantLayerNormFunction.apply(x, weight, bias, lmax, eps, out_dtype)


def equivariant_dropout(x, rng, p: float, lmax: int, residual=None):
    """Differentiable dropout of whole channels, with an optional residual sum (see eqtp_dropout).  ``rng``: int64
    (seed, offset) on the GPU; its values at this call are kept for the backward pass.  Under activation checkpointing
    the call is made twice: rng must not change in between (see the head of this module)."""
    return EquivariantDropoutFunction.apply(x, residual, rng, float(p), lmax)


def dropout_add_norm(x, residual, rng, p: float, lmax: int, weight=None, bias=None, eps: float = 1e-5,
                     out_dtype: int = None):
    """Differentiable (out, total): total = residual + dropout(x), out = layer norm of total, one pass each way
    (see eqtp_dropout_add_norm).  ``rng`` as for equivariant_dropout."""
    return DropoutAddNormFunction.apply(x, residual, weight, bias, rng, float(p), lmax, eps, out_dtype)


def graph_attention(q, k, v, src, row_ptr, lmax: int, heads: int, scale: float = None, bias=None, plan=None):
    """Differentiable attention over a graph (see eqtp_attention).  ``plan``: attention_plan's result, or None to
    group the edges in each backward pass.  ``scale`` is a number and gets no gradient (scale q to learn one)."""
    return GraphAttentionFunction.apply(q, k, v, bias, src, row_ptr, lmax, heads, scale, plan)
