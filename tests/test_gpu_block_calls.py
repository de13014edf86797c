"""Ways to call the transformer-block operators on the GPU: optional
arguments, other streams, types and wrappers give what the plain calls give."""
import numpy as np
import pytest

import block_reference as ref
from test_gpu_attention import Case, _i32
from test_gpu_norm import RNG, _get, _inputs, _within
from test_gpu_parity import _eq, _say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_attention_backward_with_the_output(x):
    """The forward call's output before lse, as a training step that keeps both passes it: the same bits, and within
    the bounds of the statement."""
    eq = _eq()
    _say("attention backward with the output, %s" % x)
    import torch

    c = Case(9, 7, [3, 0, 5, 1, 4, 2, 6, 0, 40], 8, 1, 4, 2, x, seed=31)
    out, lse = c.forward(eq)
    head = (c.q[0], c.k[0], c.v[0], _i32(c.src), _i32(c.row_ptr))
    tail = (lse, c.g[0], *(_i32(t) for t in c.plan), c.lmax, c.heads)
    grads = eq.eqtp_attention_backward(*head, out, *tail, bias=c.bias[0])
    for a, b, d in zip(grads, c.backward(eq, lse), eq.eqtp_attention_backward(*head, *tail, bias=c.bias[0], out=out)):
        assert torch.equal(a, b) and torch.equal(a, d)
    args = (c.q[1], c.k[1], c.v[1], c.src, c.row_ptr, c.heads, c.scale)
    bounds = ref.attention_bounds(*args, c.g[1], c.bias[1], ref.U16 if x == "bf16" else ref.U32)
    for name, t, w, b in zip(("gq", "gk", "gv", "gbias"), grads, ref.attention_backward(*args, c.g[1], c.bias[1]), bounds[2:]):
        _within(_get(t), w, b, name)


def test_attention_scale():
    """An explicit scale, as a number and in a tensor that changes between the passes, which keep the forward
    call's value."""
    eq = _eq()
    _say("attention with a scale of its own")
    import torch

    from spherical_harmonic_cg_amd import autograd as ag

    c = Case(8, 9, [3, 0, 5, 1, 4, 2, 6, 9], 4, 1, 4, 2, seed=32)
    for scale in (0.9, -0.4):
        args = (c.q[1], c.k[1], c.v[1], c.src, c.row_ptr, c.heads, float(np.float32(scale)))
        bounds = ref.attention_bounds(*args, c.g[1], c.bias[1], ref.U32)
        out, lse = c.forward(eq, scale=scale)
        _within(_get(out), ref.attention(*args, c.bias[1])[0], bounds[0], "out")
        wants = ref.attention_backward(*args, c.g[1], c.bias[1])
        grads = c.backward(eq, lse, scale=scale)
        for t, w, b in zip(grads, wants, bounds[2:]):
            _within(_get(t), w, b, "gradient")
        held = torch.tensor(scale)
        leaves = [t[0].clone().requires_grad_() for t in (c.q, c.k, c.v, c.bias)]
        y = ag.graph_attention(*leaves[:3], _i32(c.src), _i32(c.row_ptr), 1, 4, scale=held, bias=leaves[3])
        held.fill_(5.0)
        y.backward(c.g[0])
        assert torch.equal(y, out)
        for t, g in zip(leaves, grads):
            assert torch.equal(t.grad, g)


@pytest.mark.parametrize("N,M,lengths", [(3, 700, [900, 0, 1400]), (9, 7, [3, 0, 5, 1, 4, 2, 6, 0, 3])])
def test_attention_workspace_of_the_caller(N, M, lengths):
    """A workspace of exactly the size that is asked for gives the same bits, and nothing behind it is written."""
    eq = _eq()
    _say("attention with the caller's workspace, N=%d" % N)
    import torch

    c = Case(N, M, lengths, 4, 1, 4, 2, seed=33)
    sizes = [f(c.N, c.M, c.E, 1, 16, 4, 2) for f in (eq.eqtp_attention_workspace_bytes, eq.eqtp_attention_backward_workspace_bytes)]
    assert sizes[1] > 0 and (sizes[0] > 0) == (N == 3)
    out, lse = c.forward(eq)
    grads = c.backward(eq, lse)
    spaces = [torch.full((s + 512,), 0xA5, dtype=torch.uint8, device="cuda") for s in sizes]
    got = c.forward(eq, workspace=spaces[0][:sizes[0]])
    assert torch.equal(got[0], out) and torch.equal(got[1], lse)
    for a, b in zip(c.backward(eq, lse, workspace=spaces[1][:sizes[1]]), grads):
        assert torch.equal(a, b)
    for s, n in zip(spaces, sizes):
        assert (s[n:] == 0xA5).all()
    if N == 3:
        with pytest.raises(eq.EqtpError):
            c.forward(eq, workspace=spaces[0][:sizes[0] - 1])
    with pytest.raises(eq.EqtpError):
        c.backward(eq, lse, workspace=spaces[1][:sizes[1] - 1])


def test_norm_workspace_of_the_caller():
    eq = _eq()
    _say("norm with the caller's workspace")
    import torch

    d = _inputs(300, 12, 2, 1)
    stats = torch.empty((300, 4), device="cuda")
    eq.eqtp_layer_norm(d["x"][0], 2, d["w"][0], d["b"][0], stats=stats)
    need = eq.eqtp_layer_norm_workspace_bytes(300, 12, 2)
    space = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    want = eq.eqtp_layer_norm_backward(d["x"][0], stats, d["g"][0], 2, d["w"][0])
    got = eq.eqtp_layer_norm_backward(d["x"][0], stats, d["g"][0], 2, d["w"][0], workspace=space[:need])
    for k in (0, 2, 3):
        assert torch.equal(got[k], want[k])
    assert (space[need:] == 0xA5).all()
    with pytest.raises(eq.EqtpError):
        eq.eqtp_layer_norm_backward(d["x"][0], stats, d["g"][0], 2, d["w"][0], workspace=space[:need - 1])


def test_calls_on_another_stream():
    """Inputs made, and every operator run, on a stream of its own: the bits of the default stream's calls."""
    eq = _eq()
    _say("block operators on another stream")
    import torch

    cases = [Case(40, 40, [9] * 40, 8, 3, 4, 4, seed=16), Case(2, 4000, [1500, 2500], 16, 0, 4, 4, seed=17)]
    d = _inputs(500, 24, 2, 5)
    rng = torch.tensor(RNG, device="cuda")

    def all_calls(scale):
        """The inputs times a power of two, made here, so that they exist on this stream only."""
        m = lambda t: t * scale  # noqa: E731
        res = []
        for c in cases:
            src, rp = _i32(c.src), _i32(c.row_ptr)
            plan = [_i32(t) for t in c.plan]
            lse = torch.empty((c.N, c.heads), device="cuda")
            q, k, v, g = m(c.q[0]), m(c.k[0]), m(c.v[0]), m(c.g[0])
            res.append(eq.eqtp_attention(q, k, v, src, rp, c.lmax, c.heads, bias=c.bias[0], lse=lse))
            res.extend(eq.eqtp_attention_backward(q, k, v, src, rp, lse, g, *plan, c.lmax, c.heads, bias=c.bias[0]))
        stats = torch.empty((500, 4), device="cuda")
        out, total = eq.eqtp_dropout_add_norm(m(d["x"][0]), m(d["res"][0]), rng, 0.3, 2, d["w"][0], d["b"][0], stats=stats)
        res += [out, total, eq.eqtp_dropout(m(d["x"][0]), rng, 0.3, 2)]
        res += eq.eqtp_layer_norm_backward(total, stats, m(d["g"][0]), 2, d["w"][0], rng=rng, p=0.3)
        return res

    want = all_calls(0.5)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = all_calls(0.5)
    side.synchronize()
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_autograd_in_bf16():
    """The wrappers on bf16 tensors: gradients come in bf16 (the affine ones in fp32), within the bounds of their
    statements."""
    _eq()
    _say("autograd in bf16")
    import torch

    from spherical_harmonic_cg_amd import autograd as ag

    d = _inputs(21, 10, 2, 1, "bf16", "bf16")
    x, w, b = (d[n][0].clone().requires_grad_() for n in ("x", "w", "b"))
    ag.equivariant_layer_norm(x, 2, w, b).backward(d["g"][0])
    want = ref.norm_backward(d["x"][1], 2, d["g"][1], d["w"][1])
    bound = ref.norm_backward_bounds(d["x"][1], 2, d["g"][1], d["w"][1], 1e-5, True)
    assert x.grad.dtype is torch.bfloat16 and w.grad.dtype is b.grad.dtype is torch.float32
    for t, e, o in zip((x, w, b), want, bound):
        _within(_get(t.grad), e, o, "norm gradient")

    rng = torch.tensor(RNG, device="cuda")
    x, r = (d[n][0].clone().requires_grad_() for n in ("x", "res"))
    w = d["w"][0].clone().requires_grad_()
    out, total = ag.dropout_add_norm(x, r, rng, 0.3, 2, w)
    torch.autograd.backward([out, total], [d["g"][0], d["gt"][0]])
    t64 = _get(total.detach())
    keep = ref.keep_mask(RNG[0], RNG[1], 21, 10, 0.3)[:, :, None]
    gr, gw, _ = ref.norm_backward(t64, 2, d["g"][1], d["w"][1])
    gr = gr + d["gt"][1]
    br, bw, _ = ref.norm_backward_bounds(t64, 2, d["g"][1], d["w"][1], 1e-5, True, extra=d["gt"][1])
    _within(_get(r.grad), gr, br, "residual")
    # grad_x is rounded on its own, from the fp32 sum: its bound is that of the fp32 sum and one more rounding
    b32 = ref.norm_backward_bounds(t64, 2, d["g"][1], d["w"][1], 1e-5, False, extra=d["gt"][1])[0]
    bx = (1.001 * b32 + 3 * ref.U32 * np.abs(gr)) / 0.7
    _within(_get(x.grad), np.where(keep, gr / 0.7, 0.0), bx + ref.U16 * (np.abs(gr) / 0.7 + bx), "x")
    _within(_get(w.grad), gw, bw, "weight")

    x = d["x"][0].clone().requires_grad_()
    ag.equivariant_dropout(x, rng, 0.25, 2).backward(d["g"][0])
    keep = ref.keep_mask(RNG[0], RNG[1], 21, 10, 0.25)[:, :, None]
    want = np.where(keep, d["g"][1] / 0.75, 0.0)
    # the factor is held in fp32, the product rounds to fp32 and then to bf16
    _within(_get(x.grad), want, np.abs(want) * (ref.U16 + 3 * ref.U32), "dropout")

    c = Case(9, 7, [3, 0, 5, 1, 4, 2, 6, 0, 3], 4, 1, 4, 2, "bf16", seed=5)
    leaves = [t[0].clone().requires_grad_() for t in (c.q, c.k, c.v, c.bias)]
    src, rp = _i32(c.src), _i32(c.row_ptr)
    ag.graph_attention(*leaves[:3], src, rp, 1, 4, bias=leaves[3], plan=ag.attention_plan(src, rp, 7)).backward(c.g[0])
    args = (c.q[1], c.k[1], c.v[1], c.src, c.row_ptr, 4, c.scale)
    bounds = ref.attention_bounds(*args, c.g[1], c.bias[1], ref.U16)[2:]
    for t, e, o in zip(leaves, ref.attention_backward(*args, c.g[1], c.bias[1]), bounds):
        assert t.grad.dtype is t.dtype
        _within(_get(t.grad), e, o, "attention gradient")


@pytest.mark.parametrize("reentrant", [False, True])
def test_dropout_under_checkpointing(reentrant):
    """A row of rng for each place, left alone while the step's own offset moves on: a recomputed forward pass makes
    the first one's masks, and the gradients have the bits of a run without checkpoints."""
    _eq()
    _say("dropout under activation checkpointing, reentrant=%s" % reentrant)
    import torch
    from torch.utils.checkpoint import checkpoint

    from spherical_harmonic_cg_amd import autograd as ag

    d = _inputs(40, 8, 1, 3)

    def grads(kept):
        rng = torch.tensor(RNG, device="cuda")
        places = torch.stack((rng[0].expand(3), rng[1] + torch.arange(3, device="cuda")), 1)
        x, w = d["x"][0].clone().requires_grad_(), d["w"][0].clone().requires_grad_()

        def layer(h, place):
            n, t = ag.dropout_add_norm(torch.tanh(h), h, place, 0.4, 1, w)
            return ag.equivariant_dropout(n, place, 0.2, 1, residual=t) * n

        h = x
        for i in range(3):
            h = layer(h, places[i]) if kept else checkpoint(layer, h, places[i], use_reentrant=reentrant)
            rng[1] += 1
        h.backward(d["g"][0])
        return h.detach(), x.grad, w.grad

    for a, b in zip(grads(True), grads(False)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("N,M", [(9, 7), (7, 9), (40, 1)])
def test_attention_plan_in_debug_mode(N, M):
    """More rows than sources, and fewer: the checks of debug mode take rows for rows and sources for sources."""
    eq = _eq()
    _say("attention plan in debug mode N=%d M=%d" % (N, M))
    import torch

    from spherical_harmonic_cg_amd import autograd as ag

    c = Case(N, M, [3] * N, 4, 1, 2, 2, seed=34)
    src, rp = _i32(c.src), _i32(c.row_ptr)
    was = eq.eqtp_set_debug(True)
    try:
        plan = ag.attention_plan(src, rp, M)
        for a, b in zip(plan, c.plan):
            assert (a.cpu().numpy() == b).all()
        leaves = [t[0].clone().requires_grad_() for t in (c.q, c.k, c.v)]
        ag.graph_attention(*leaves, src, rp, 1, 2, bias=c.bias[0]).backward(c.g[0])
    finally:
        eq.eqtp_set_debug(was)
    _, lse = c.forward(eq)
    for t, g in zip(leaves, c.backward(eq, lse)):
        assert torch.equal(t.grad, g)


def test_attention_without_rows_or_edges_through_autograd():
    """No edges, and no rows: zero gradients, from a plan made in the backward pass."""
    eq = _eq()
    _say("attention autograd without edges")
    import torch

    from spherical_harmonic_cg_amd import autograd as ag

    none = torch.empty(0, dtype=torch.int32, device="cuda")
    for N, M in ((4, 3), (0, 3), (4, 0), (0, 0)):
        q, k, v = (torch.randn((n, 6, 4), device="cuda", requires_grad=True) for n in (N, M, M))
        bias = torch.empty((0, 2), device="cuda", requires_grad=True)
        rp = torch.zeros(N + 1, dtype=torch.int32, device="cuda")
        out = ag.graph_attention(q, k, v, none, rp, 1, 2, bias=bias)
        out.backward(torch.ones_like(out))
        assert out.shape == q.shape and (out == 0).all()
        for t in (q, k, v, bias):
            assert t.grad.shape == t.shape and (t.grad == 0).all()
