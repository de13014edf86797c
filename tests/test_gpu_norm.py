"""Layer norm by degree on the GPU, forward and backward, alone and fused with
dropout and the residual sum, against its 64-bit statement.

Tolerances are elementwise bounds derived from the roundings on the way (see
block_reference); a bf16 output adds half a step, 2^-8 of the value."""
import numpy as np
import pytest

import block_reference as ref
from test_gpu_parity import _eq, _say

pytestmark = pytest.mark.gpu

EPS = 1e-5
RNG = (0x123456789ABCDEF0, 0x0FEDCBA987654321)


def _dt(name):
    import torch

    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _code(eq, name):
    return eq.EQTP_BF16 if name == "bf16" else eq.EQTP_F32


def _put(a, dtype="f32", shift=0):
    """a on the GPU in the given type, `shift` elements into its storage (contiguous, less aligned); and the
    values it holds there, in 64 bits."""
    import torch

    a = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(_dt(dtype))
    buf = torch.empty(a.numel() + shift, dtype=a.dtype, device="cuda")
    t = buf[shift:].view(a.shape)
    t.copy_(a)
    return t, t.double().cpu().numpy()


def _get(t):
    import torch

    torch.cuda.synchronize()
    return t.double().cpu().numpy()


def _inputs(N, C, lmax, seed, x="f32", out="f32", shift=0, offset=0.5):
    r = np.random.default_rng(seed)
    K = (lmax + 1) ** 2
    base = r.standard_normal((N, C, K)) / (1.0 + ref.degrees(lmax)) + offset * (ref.degrees(lmax) == 0)
    d = {"x": _put(base, x, shift), "res": _put(r.standard_normal((N, C, K)), x, shift),
         "g": _put(r.standard_normal((N, C, K)), out, shift), "gt": _put(r.standard_normal((N, C, K)), x, shift),
         "w": _put(1.0 + 0.3 * r.standard_normal((lmax + 1, C))), "b": _put(0.3 * r.standard_normal(C))}
    return d


def _within(got, want, bound, what):
    got = np.asarray(got)
    assert np.isfinite(got).all(), what + ": non-finite output"
    over = np.abs(got - want) - bound
    assert (over <= 0).all(), "%s: off by %.3e where %.3e is allowed" % (
        what, np.abs(got - want).ravel()[over.argmax()], np.broadcast_to(bound, got.shape).ravel()[over.argmax()])


SIZES = [(0, 1, 3), (0, 2, 5), (0, 64, 37), (0, 65, 1), (0, 1000, 4), (0, 4097, 3), (0, 16384, 2), (0, 16383, 2),
         (1, 1, 2), (1, 8, 9), (1, 37, 5), (2, 8, 64), (2, 33, 7), (3, 1, 4), (3, 32, 50), (3, 64, 33), (3, 65, 5),
         (3, 128, 9), (3, 1000, 2), (4, 5, 6), (4, 33, 8), (5, 3, 7), (5, 64, 4), (6, 8, 5), (6, 128, 3), (6, 1, 1)]


@pytest.mark.parametrize("lmax,C,N", SIZES)
@pytest.mark.parametrize("x,out", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
def test_norm_forward(lmax, C, N, x, out):
    eq = _eq()
    _say("norm forward lmax=%d C=%d N=%d %s->%s" % (lmax, C, N, x, out))
    d = _inputs(N, C, lmax, 10 + lmax + C, x, out)
    import torch

    stats = torch.full((N, lmax + 2), float("nan"), device="cuda")
    got = eq.eqtp_layer_norm(d["x"][0], lmax, d["w"][0], d["b"][0], eps=EPS, out_dtype=_code(eq, out), stats=stats)
    assert got.dtype == _dt(out)
    want, _, r, mean = ref.norm(d["x"][1], lmax, d["w"][1], d["b"][1], EPS)
    _within(_get(got), want, ref.norm_bound(d["x"][1], lmax, d["w"][1], d["b"][1], EPS, out == "bf16"), "out")
    s = _get(stats)
    dmean = ref.CHAIN * ref.U32 * np.abs(d["x"][1][:, :, 0]).mean(axis=1)
    _within(s[:, 0], mean, dmean + 1e-37, "mean")
    rel = np.full(r.shape, 2 * ref.CHAIN * ref.U32)
    rel[:, 0] += (dmean * r[:, 0]) ** 2 + ref.CHAIN * ref.U32 * dmean * r[:, 0]
    _within(s[:, 1:], r, r * rel, "r")


@pytest.mark.parametrize("lmax,C,N", SIZES)
@pytest.mark.parametrize("x,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_norm_backward(lmax, C, N, x, out):
    eq = _eq()
    _say("norm backward lmax=%d C=%d N=%d %s->%s" % (lmax, C, N, x, out))
    import torch

    d = _inputs(N, C, lmax, 20 + lmax + C, x, out)
    stats = torch.empty((N, lmax + 2), device="cuda")
    eq.eqtp_layer_norm(d["x"][0], lmax, d["w"][0], d["b"][0], eps=EPS, out_dtype=_code(eq, out), stats=stats)
    gx, none, gw, gb = eq.eqtp_layer_norm_backward(d["x"][0], stats, d["g"][0], lmax, d["w"][0])
    assert none is None and gx.dtype == _dt(x)
    wx, ww, wb = ref.norm_backward(d["x"][1], lmax, d["g"][1], d["w"][1], EPS)
    bx, bw, bb = ref.norm_backward_bounds(d["x"][1], lmax, d["g"][1], d["w"][1], EPS, x == "bf16")
    _within(_get(gx), wx, bx, "gx")
    _within(_get(gw), ww, bw, "gweight")
    _within(_get(gb), wb, bb, "gbias")


@pytest.mark.parametrize("lmax,C,N", [(0, 64, 3001), (0, 7, 20011), (3, 32, 2003), (2, 9, 3001), (4, 50, 700), (0, 1024, 515)])
@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_norm_backward_many_nodes(lmax, C, N, x):
    """The gradients of weight and bias over more nodes than workgroups; the same bits twice."""
    eq = _eq()
    _say("norm backward lmax=%d C=%d N=%d %s" % (lmax, C, N, x))
    import torch

    d = _inputs(N, C, lmax, 30 + lmax + C, x, x)
    stats = torch.empty((N, lmax + 2), device="cuda")
    eq.eqtp_layer_norm(d["x"][0], lmax, d["w"][0], d["b"][0], eps=EPS, stats=stats)
    a = eq.eqtp_layer_norm_backward(d["x"][0], stats, d["g"][0], lmax, d["w"][0])
    b = eq.eqtp_layer_norm_backward(d["x"][0], stats, d["g"][0], lmax, d["w"][0])
    for s, t in zip(a, b):
        assert s is None or torch.equal(s, t)
    want = ref.norm_backward(d["x"][1], lmax, d["g"][1], d["w"][1], EPS)
    bound = ref.norm_backward_bounds(d["x"][1], lmax, d["g"][1], d["w"][1], EPS, x == "bf16")
    for got, w, e, what in zip((a[0], a[2], a[3]), want, bound, ("gx", "gweight", "gbias")):
        _within(_get(got), w, e, what)


@pytest.mark.parametrize("lmax,C", [(0, 65), (3, 32), (2, 7)])
def test_norm_gradient_against_differences(lmax, C):
    """The kernel's gradients along a direction equal central differences of the 64-bit forward pass.
    The elementwise bounds, summed along the direction, plus the differences' own 1e-6."""
    eq = _eq()
    _say("norm differences lmax=%d C=%d" % (lmax, C))
    import torch

    N, h = 6, 1e-4
    d = _inputs(N, C, lmax, 40 + C)
    stats = torch.empty((N, lmax + 2), device="cuda")
    eq.eqtp_layer_norm(d["x"][0], lmax, d["w"][0], d["b"][0], eps=EPS, stats=stats)
    gx, _, gw, gb = eq.eqtp_layer_norm_backward(d["x"][0], stats, d["g"][0], lmax, d["w"][0])
    args = [d["x"][1], d["w"][1], d["b"][1]]
    bounds = ref.norm_backward_bounds(d["x"][1], lmax, d["g"][1], d["w"][1], EPS, False)
    r = np.random.default_rng(1)
    f = lambda a: (ref.norm(a[0], lmax, a[1], a[2], EPS)[0] * d["g"][1]).sum()
    for k, grad in enumerate((gx, gw, gb)):
        v = r.standard_normal(args[k].shape)
        up, down = list(args), list(args)
        up[k], down[k] = args[k] + h * v, args[k] - h * v
        slope = (f(up) - f(down)) / (2 * h)
        mine = (_get(grad) * v).sum()
        allow = (bounds[k] * np.abs(v)).sum() + 1e-6 * (np.abs(_get(grad) * v).sum() + 1.0)
        assert abs(mine - slope) <= allow, (k, mine, slope, allow)


@pytest.mark.parametrize("lmax,C,N", [(0, 64, 33), (0, 7, 9), (3, 32, 21), (2, 5, 11), (4, 33, 6), (6, 3, 5), (0, 5000, 3)])
@pytest.mark.parametrize("x,out", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_fused_equals_its_parts(lmax, C, N, x, out, p):
    """total and out have the bits of dropout followed by the norm; the gradients those of the norm's, with the
    other gradient added and dropped channels zero."""
    eq = _eq()
    _say("fused lmax=%d C=%d N=%d %s->%s p=%g" % (lmax, C, N, x, out, p))
    import torch

    d = _inputs(N, C, lmax, 50 + C, x, out)
    rng = torch.tensor(RNG, device="cuda")
    sa, sb = torch.empty((N, lmax + 2), device="cuda"), torch.empty((N, lmax + 2), device="cuda")
    o, t = eq.eqtp_dropout_add_norm(d["x"][0], d["res"][0], rng, p, lmax, d["w"][0], d["b"][0], eps=EPS,
                                    out_dtype=_code(eq, out), stats=sa)
    t2 = eq.eqtp_dropout(d["x"][0], rng, p, lmax, residual=d["res"][0])
    o2 = eq.eqtp_layer_norm(t2, lmax, d["w"][0], d["b"][0], eps=EPS, out_dtype=_code(eq, out), stats=sb)
    assert torch.equal(t, t2) and torch.equal(o, o2) and torch.equal(sa, sb)
    keep = ref.keep_mask(RNG[0], RNG[1], N, C, p)
    want = ref.dropout(d["x"][1], keep, p, d["res"][1])
    _within(_get(t), want, (ref.U16 if x == "bf16" else ref.U32) * np.abs(want) * (1 + 1e-6) + 1e-37, "total")
    gr, gx, gw, gb = eq.eqtp_layer_norm_backward(t, sa, d["g"][0], lmax, d["w"][0], grad_total=d["gt"][0], rng=rng, p=p,
                                                 need_x=True)
    tt = _get(t)
    wr, ww, wb = ref.norm_backward(tt, lmax, d["g"][1], d["w"][1], EPS)
    br, bw, bb = ref.norm_backward_bounds(tt, lmax, d["g"][1], d["w"][1], EPS, x == "bf16", extra=d["gt"][1])
    wr = wr + d["gt"][1]
    _within(_get(gr), wr, br, "grad_residual")
    scale = 1.0 / (1.0 - p)
    _within(_get(gx), np.where(keep[:, :, None], wr * scale, 0.0), 1.001 * scale * br, "grad_x")
    assert (_get(gx)[~keep] == 0).all()
    _within(_get(gw), ww, bw, "gweight")
    _within(_get(gb), wb, bb, "gbias")


@pytest.mark.parametrize("lmax,C", [(0, 64), (0, 7), (3, 32), (2, 7), (4, 5)])
@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [1, 2, 3])
def test_norm_unaligned(lmax, C, x, shift):
    """Tensors that begin one to three elements into their storage give the same bits as aligned ones."""
    eq = _eq()
    _say("norm unaligned lmax=%d C=%d %s shift %d" % (lmax, C, x, shift))
    import torch

    N = 19
    rng = torch.tensor(RNG, device="cuda")
    got = []
    for s in (0, shift):
        d = _inputs(N, C, lmax, 60 + C, x, x, shift=s)
        K = (lmax + 1) ** 2
        out, total = (torch.empty(N * C * K + s, dtype=_dt(x), device="cuda")[s:].view(N, C, K) for _ in range(2))
        stats = torch.empty((N, lmax + 2), device="cuda")
        eq.eqtp_dropout_add_norm(d["x"][0], d["res"][0], rng, 0.2, lmax, d["w"][0], d["b"][0], out=out, total=total,
                                 stats=stats)
        got.append((out, total) + eq.eqtp_layer_norm_backward(total, stats, d["g"][0], lmax, d["w"][0],
                                                              grad_total=d["gt"][0], rng=rng, p=0.2))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_norm_without_weight_and_bias():
    eq = _eq()
    _say("norm without weight and bias")
    import torch

    d = _inputs(9, 12, 2, 70)
    for w, b in ((None, None), (d["w"], None), (None, d["b"])):
        stats = torch.empty((9, 4), device="cuda")
        got = eq.eqtp_layer_norm(d["x"][0], 2, w and w[0], b and b[0], eps=EPS, stats=stats)
        wv, bv = w and w[1], b and b[1]
        _within(_get(got), ref.norm(d["x"][1], 2, wv, bv, EPS)[0], ref.norm_bound(d["x"][1], 2, wv, bv, EPS, False), "out")
        gx, _, gw, gb = eq.eqtp_layer_norm_backward(d["x"][0], stats, d["g"][0], 2, w and w[0])
        want = ref.norm_backward(d["x"][1], 2, d["g"][1], wv, EPS)
        bound = ref.norm_backward_bounds(d["x"][1], 2, d["g"][1], wv, EPS, False)
        for g, e, t in zip((gx, gw, gb), want, bound):
            _within(_get(g), e, t, "gradient")
        for need in ((True, False, False), (False, True, False), (False, False, True)):
            part = eq.eqtp_layer_norm_backward(d["x"][0], stats, d["g"][0], 2, w and w[0], need_residual=need[0],
                                               need_weight=need[1], need_bias=need[2])
            for p, full, n in zip((part[0], part[2], part[3]), (gx, gw, gb), need):
                assert (p is None) != n and (not n or torch.equal(p, full))


def test_norm_degenerate_rows():
    """Constant and zero rows (variance 0), far-off means, tiny and huge values; a NaN or an infinity spoils its
    own row (its own degree) only."""
    eq = _eq()
    _say("norm degenerate rows")
    C, lmax = 24, 2
    x = np.random.default_rng(8).standard_normal((9, C, 9)).astype(np.float32)
    x[0] = 0.0
    x[1] = 3.25
    x[2, :, 0] += 4096.0
    x[3] *= 1e-20
    x[4] *= 1e15
    x[5, 3, 0] = np.nan
    x[6, 2, 5] = np.inf
    t, v = _put(x)
    w, b = _put(np.ones((3, C))), _put(np.zeros(C))
    got = _get(eq.eqtp_layer_norm(t, lmax, w[0], b[0], eps=EPS))
    clean = [0, 1, 2, 3, 4, 7, 8]
    want = ref.norm(v[clean], lmax, w[1], b[1], EPS)[0]
    _within(got[clean], want, ref.norm_bound(v[clean], lmax, w[1], b[1], EPS, False), "clean rows")
    assert (got[0] == 0).all() and (got[1, :, 0] == 0).all()
    assert np.isnan(got[5, :, 0]).all() and np.isfinite(got[5, :, 1:]).all()
    assert np.isnan(got[6, 2, 5]) and np.isfinite(got[6][:, [0, 1, 2, 3]]).all()


def test_norm_no_nodes():
    eq = _eq()
    _say("norm without nodes")
    import torch

    x = torch.empty((0, 6, 4), device="cuda")
    assert eq.eqtp_layer_norm(x, 1).shape == (0, 6, 4)
    o, t = eq.eqtp_dropout_add_norm(x, x.clone(), None, 0.0, 1)
    assert o.shape == t.shape == (0, 6, 4)
    gx, _, gw, gb = eq.eqtp_layer_norm_backward(x, torch.empty((0, 3), device="cuda"), x.clone(), 1)
    assert gx.shape == (0, 6, 4) and (gw == 0).all() and (gb == 0).all() and gw.shape == (2, 6)


def test_norm_two_dimensional():
    eq = _eq()
    import torch

    _say("norm of [N, C]")
    x = torch.randn(11, 40, device="cuda")
    assert torch.equal(eq.eqtp_layer_norm(x, 0), eq.eqtp_layer_norm(x.view(11, 40, 1), 0).view(11, 40))


def test_norm_large_offsets():
    """More than 2^32 elements, rows past that mark included; sampled rows against the 64-bit statement."""
    eq = _eq()
    _say("norm past 2^32 elements")
    import torch

    N, C = 270000, 16000
    x = torch.empty((N, C), dtype=torch.bfloat16, device="cuda")
    for at in range(0, N, 30000):
        x[at:at + 30000].normal_()
    rows = [0, 134217, 134218, 268435, 268436, N - 1]
    want, _, _, _ = ref.norm(x[rows].double().cpu().numpy()[:, :, None], 0, None, None, EPS)
    bound = ref.norm_bound(x[rows].double().cpu().numpy()[:, :, None], 0, None, None, EPS, True)
    stats = torch.empty((N, 2), device="cuda")
    got = eq.eqtp_layer_norm(x, 0, eps=EPS, stats=stats)
    _within(_get(got[rows])[:, :, None], want, bound, "sampled rows")
    gx, _, _, gb = eq.eqtp_layer_norm_backward(x, stats, got, 0)
    g = got[rows].double().cpu().numpy()[:, :, None]
    wx, _, _ = ref.norm_backward(x[rows].double().cpu().numpy()[:, :, None], 0, g, None, EPS)
    bx, _, _ = ref.norm_backward_bounds(x[rows].double().cpu().numpy()[:, :, None], 0, g, None, EPS, True)
    _within(_get(gx[rows])[:, :, None], wx, bx, "sampled rows of the gradient")


def test_norm_side_stream_and_graph():
    """On a stream of its own, and captured: every replay reproduces the eager result, with eager work between, and
    sees the offset that the device holds at that time."""
    eq = _eq()
    _say("norm graph")
    import torch

    N, C, lmax, p = 101, 32, 3, 0.25
    d = _inputs(N, C, lmax, 80)
    rng = torch.tensor(RNG, device="cuda")
    o, t = torch.empty((N, C, 16), device="cuda"), torch.empty((N, C, 16), device="cuda")
    stats = torch.empty((N, lmax + 2), device="cuda")
    ws = torch.empty(eq.eqtp_layer_norm_workspace_bytes(N, C, lmax), dtype=torch.uint8, device="cuda")

    def step():
        eq.eqtp_dropout_add_norm(d["x"][0], d["res"][0], rng, p, lmax, d["w"][0], d["b"][0], out=o, total=t, stats=stats)
        return eq.eqtp_layer_norm_backward(t, stats, d["g"][0], lmax, d["w"][0], grad_total=d["gt"][0], rng=rng, p=p,
                                           workspace=ws)

    eager = {}
    for off in (1, 2, 3):
        rng[1] = off
        eager[off] = [v.clone() for v in step()] + [o.clone(), t.clone()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        held = list(step())
        for a, b in zip(held + [o, t], eager[3]):
            assert torch.equal(a, b)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        grads = step()
    for off in (2, 1, 3, 2):
        rng[1] = off
        o.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(list(grads) + [o, t], eager[off]):
            assert torch.equal(a, b), off
        step()
        torch.cuda.synchronize()


@pytest.mark.parametrize("lmax,C,N", [(0, 130, 5), (0, 256, 9), (0, 301, 4), (0, 512, 5), (0, 600, 3), (0, 1500, 3), (0, 2048, 2),
                                      (0, 3001, 2), (0, 9000, 2), (1, 16, 40), (1, 33, 9), (1, 100, 6), (1, 3000, 2), (2, 3, 70),
                                      (2, 14, 9), (2, 28, 5), (2, 60, 4), (2, 300, 2), (3, 4, 30), (3, 8, 17), (4, 3, 20), (4, 16, 6),
                                      (4, 600, 2), (5, 1, 40), (5, 7, 9), (5, 20, 5), (6, 4, 9), (6, 10, 6), (6, 330, 2)])
@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_norm_more_widths(lmax, C, N, x, p):
    """Widths on both sides of every change of the group of threads, with and without dropout, both directions."""
    eq = _eq()
    _say("norm widths lmax=%d C=%d N=%d %s p=%g" % (lmax, C, N, x, p))
    import torch

    d = _inputs(N, C, lmax, 90 + C, x, x)
    rng = torch.tensor(RNG, device="cuda")
    stats = torch.empty((N, lmax + 2), device="cuda")
    o, t = eq.eqtp_dropout_add_norm(d["x"][0], d["res"][0], rng, p, lmax, d["w"][0], d["b"][0], eps=EPS, stats=stats)
    keep = ref.keep_mask(RNG[0], RNG[1], N, C, p)
    want = ref.dropout(d["x"][1], keep, p, d["res"][1])
    _within(_get(t), want, (ref.U16 if x == "bf16" else ref.U32) * np.abs(want) * (1 + 1e-6) + 1e-37, "total")
    tt = _get(t)
    _within(_get(o), ref.norm(tt, lmax, d["w"][1], d["b"][1], EPS)[0],
            ref.norm_bound(tt, lmax, d["w"][1], d["b"][1], EPS, x == "bf16"), "out")
    gr, gx, gw, gb = eq.eqtp_layer_norm_backward(t, stats, d["g"][0], lmax, d["w"][0], grad_total=d["gt"][0], rng=rng, p=p,
                                                 need_x=True)
    wr, ww, wb = ref.norm_backward(tt, lmax, d["g"][1], d["w"][1], EPS)
    br, bw, bb = ref.norm_backward_bounds(tt, lmax, d["g"][1], d["w"][1], EPS, x == "bf16", extra=d["gt"][1])
    wr, scale = wr + d["gt"][1], 1.0 / (1.0 - p)
    _within(_get(gr), wr, br, "grad_residual")
    _within(_get(gx), np.where(keep[:, :, None], wr * scale, 0.0), 1.001 * scale * br, "grad_x")
    _within(_get(gw), ww, bw, "gweight")
    _within(_get(gb), wb, bb, "gbias")
