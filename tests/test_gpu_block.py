"""The transformer-block operators through autograd, and the example that runs
them together: gradients against the 64-bit statements, rotations of the
whole block, training that lowers the loss."""
import importlib.util
import os

import numpy as np
import pytest

import block_reference as ref
from test_gpu_attention import Case, _i32
from test_gpu_norm import RNG, _get, _inputs, _within
from test_gpu_parity import _eq, _say

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _ag():
    _eq()
    from spherical_harmonic_cg_amd import autograd

    return autograd


def _example():
    spec = importlib.util.spec_from_file_location("transformer_block", os.path.join(ROOT, "examples", "transformer_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_layer_norm_autograd():
    ag = _ag()
    _say("layer norm autograd")
    import torch

    d = _inputs(21, 10, 2, 1)
    x, w, b = (d[n][0].clone().requires_grad_() for n in ("x", "w", "b"))
    y = ag.equivariant_layer_norm(x, 2, w, b)
    g = d["g"][0].transpose(0, 1).contiguous().transpose(0, 1)  # a gradient that is not contiguous
    y.backward(g)
    want = ref.norm_backward(d["x"][1], 2, d["g"][1], d["w"][1])
    bound = ref.norm_backward_bounds(d["x"][1], 2, d["g"][1], d["w"][1], 1e-5, False)
    for t, e, o in zip((x, w, b), want, bound):
        _within(_get(t.grad), e, o, "gradient")
    x2 = d["x"][0].clone().requires_grad_()
    ag.equivariant_layer_norm(x2, 2).sum().backward()
    assert x2.grad is not None
    with torch.no_grad():
        assert torch.equal(ag.equivariant_layer_norm(x, 2, w, b), y)


def test_dropout_autograd_keeps_its_offset():
    """The mask of the backward pass is the forward pass's, whatever the caller does to rng between."""
    ag = _ag()
    _say("dropout autograd")
    import torch

    rng = torch.tensor(RNG, device="cuda")
    x = torch.randn((30, 8, 4), device="cuda", requires_grad=True)
    r = torch.randn((30, 8, 4), device="cuda", requires_grad=True)
    y = ag.equivariant_dropout(x, rng, 0.4, 1, residual=r)
    rng[1] += 1
    g = torch.randn_like(x)
    y.backward(g)
    keep = torch.from_numpy(ref.keep_mask(RNG[0], RNG[1], 30, 8, 0.4)).cuda()[:, :, None]
    scale = torch.tensor(1.0 / 0.6, dtype=torch.float32, device="cuda")
    assert torch.equal(x.grad, torch.where(keep, g * scale, torch.zeros_like(g))) and torch.equal(r.grad, g)


@pytest.mark.parametrize("use", ["both", "out", "total"])
def test_dropout_add_norm_autograd(use):
    ag = _ag()
    _say("dropout_add_norm autograd, %s used" % use)
    import torch

    d = _inputs(17, 12, 1, 2)
    rng = torch.tensor(RNG, device="cuda")
    x, r, w, b = (d[n][0].clone().requires_grad_() for n in ("x", "res", "w", "b"))
    out, total = ag.dropout_add_norm(x, r, rng, 0.3, 1, w, b)
    rng[1] = 7
    parts = {"out": ((out, d["g"][0]),), "total": ((total, d["gt"][0]),), "both": ((out, d["g"][0]), (total, d["gt"][0]))}[use]
    torch.autograd.backward([t for t, _ in parts], [t for _, t in parts])
    keep = ref.keep_mask(RNG[0], RNG[1], 17, 12, 0.3)
    t64 = _get(total.detach())
    gr, gw, gb = np.zeros_like(t64), None, None
    br = 0.0
    if use != "total":
        gr, gw, gb = ref.norm_backward(t64, 1, d["g"][1], d["w"][1])
        br, bw, bb = ref.norm_backward_bounds(t64, 1, d["g"][1], d["w"][1], 1e-5, False, extra=d["gt"][1])
    if use != "out":
        gr = gr + d["gt"][1]
    _within(_get(r.grad), gr, br + 1e-37, "residual")
    _within(_get(x.grad), np.where(keep[:, :, None], gr / 0.7, 0.0), (1.001 * br + 3 * ref.U32 * np.abs(gr)) / 0.7 + 1e-37, "x")
    if use != "total":
        _within(_get(w.grad), gw, bw, "weight")
        _within(_get(b.grad), gb, bb, "bias")
    else:
        assert w.grad is None and b.grad is None


@pytest.mark.parametrize("plan", [False, True])
def test_graph_attention_autograd(plan):
    ag = _ag()
    _say("attention autograd")
    import torch

    c = Case(9, 7, [3, 0, 5, 1, 4, 2, 6, 0, 3], 4, 1, 4, 2, seed=5)
    leaves = [t[0].clone().requires_grad_() for t in (c.q, c.k, c.v, c.bias)]
    src, rp = _i32(c.src), _i32(c.row_ptr)
    out = ag.graph_attention(leaves[0], leaves[1], leaves[2], src, rp, 1, 4, bias=leaves[3],
                             plan=ag.attention_plan(src, rp, 7) if plan else None)
    out.backward(c.g[0])
    args = (c.q[1], c.k[1], c.v[1], c.src, c.row_ptr, 4, c.scale)
    bounds = ref.attention_bounds(*args, c.g[1], c.bias[1], ref.U32)[2:]
    for t, w, e in zip(leaves, ref.attention_backward(*args, c.g[1], c.bias[1]), bounds):
        _within(_get(t.grad), w, e, "gradient")
    k = c.k[0].clone().requires_grad_()  # only one of them
    ag.graph_attention(c.q[0], k, c.v[0], src, rp, 1, 4, bias=c.bias[0]).backward(c.g[0])
    assert torch.equal(k.grad, leaves[1].grad)


def test_block_commutes_with_rotations():
    """Edge vectors turned by a right angle about z and features by the matching matrices leave the readout unchanged
    and turn the residual stream.  The components are ordered 0, 1c, 1s, .. per degree; a quarter turn about z maps
    (x, y) to (-y, x), so cos(m phi) and sin(m phi) of order m change by the angle m pi / 2: signs and swaps only,
    and the two runs differ by the order of roundings alone (1e-4 of the largest value, as for the convolution)."""
    ex, ag = _example(), _ag()
    _say("block rotations")
    import torch

    dev = torch.device("cuda")
    lmax, C = 2, 16
    b = ex.batch(60, lmax, C, 3, dev)
    N = 4 * 60
    items = torch.arange(N, dtype=torch.int32, device=dev)
    plans = (ag.attention_plan(b["src"], b["row_ptr"], N), ag.attention_plan(items, b["cell_ptr"], N))
    model = ex.Block(C, lmax, 4, dev, 1)
    rng = torch.tensor(RNG, device=dev)
    K = 9
    R = np.zeros((K, K))
    for l in range(lmax + 1):
        R[l * l, l * l] = 1.0
        for m in range(1, l + 1):
            c, s = l * l + 2 * m - 1, l * l + 2 * m
            co, si = [(1, 0), (0, 1), (-1, 0), (0, -1)][m % 4]
            R[c, c], R[c, s], R[s, c], R[s, s] = co, -si, si, co   # cos(m(phi + 90)), sin(m(phi + 90))
    turned = dict(b)
    v = b["vec"]
    turned["vec"] = torch.stack((-v[:, 1], v[:, 0], v[:, 2]), 1).contiguous()
    turned["x"] = (b["x"].double() @ torch.from_numpy(R.T).to(dev)).float().contiguous()
    with torch.no_grad():
        e0, e1 = model(b, plans, rng, 0.2), model(turned, plans, rng, 0.2)
    assert (e0 - e1).abs().max() <= 1e-4 * e0.abs().max()
    other = dict(turned, x=b["x"])           # features that were not turned along
    with torch.no_grad():
        assert (e0 - model(other, plans, rng, 0.2)).abs().max() > 1e-2 * e0.abs().max()


def test_example_trains():
    ex = _example()
    _say("example trains")
    losses = ex.train(steps=25, atoms=80, channels=16, lmax=1, heads=4, p=0.1, seed=2, log=None)
    assert np.isfinite(losses).all() and np.mean(losses[-3:]) < 0.3 * losses[0]
