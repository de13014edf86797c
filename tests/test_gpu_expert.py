"""The experts' per-degree linears on the GPU, and the plan of a routing, against
the 64-bit statements, within bounds derived in mix_reference."""
import numpy as np
import pytest

import mix_reference as ref
from test_gpu_norm import _code, _get, _put, _within
from test_gpu_parity import _eq, _say

pytestmark = pytest.mark.gpu


class Mix:
    def __init__(self, N, C, lmax, X, k, x="f32", gates=True, seed=0, holes=True):
        import torch

        r = np.random.default_rng(seed)
        K = (lmax + 1) ** 2
        self.N, self.C, self.lmax, self.X, self.k, self.x, self.gates = N, C, lmax, X, k, x, gates
        self.h, self.g = (_put(r.standard_normal((N, C, K)), x) for _ in range(2))
        self.W = _put(r.standard_normal((X, lmax + 1, C, C)) / np.sqrt(C), x)
        self.idx = r.integers(-1 if holes else 0, X + (1 if holes else 0), (N, k)).astype(np.int32)  # some outside
        if X > 2:
            self.idx[self.idx == 1] = 2  # an expert that nobody has
        self.w = _put(r.uniform(0.1, 1.0, (N, k))) if gates else (None, None)
        self.ti = torch.from_numpy(self.idx).cuda()

    def check(self, eq, plan, out="f32"):
        o = eq.eqtp_expert_linear(self.h[0], self.W[0], self.ti, self.lmax, weight=self.w[0], plan=plan, out_dtype=_code(eq, out))
        want, size = ref.expert(self.h[1], self.W[1], self.idx, self.lmax, self.w[1])
        half = ref.U16 if out == "bf16" else ref.U32
        _within(_get(o), want, ref.expert_bound(want, size, self.C, self.k, half), "out")
        grads = self.grads(eq, plan)
        wants, bounds = ref.expert_backward(self.h[1], self.W[1], self.idx, self.g[1], self.lmax, self.w[1], self.x == "bf16")
        for t, w, b, name in zip(grads, wants, bounds, ("grad_h", "grad_W", "grad_weight")):
            _within(_get(t), w, b, name)
        return o, grads

    def grads(self, eq, plan, **kw):
        return eq.eqtp_expert_linear_backward(self.h[0], self.W[0], self.ti, self.g[0], self.lmax, weight=self.w[0], plan=plan,
                                              **dict(dict(need_weight=True), **kw))


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("N,C,lmax,X,k,gates", [
    (1, 64, 3, 8, 2, True), (1, 8, 0, 1, 1, False), (16, 16, 1, 3, 1, False), (17, 32, 2, 4, 2, True), (50, 64, 3, 10, 1, False),
    (33, 128, 3, 5, 2, True), (40, 32, 3, 8, 4, True), (12, 8, 4, 6, 3, True), (9, 16, 6, 3, 2, True), (5, 128, 6, 2, 2, True),
    (7, 64, 5, 40, 3, True), (300, 16, 0, 256, 4, True), (100, 128, 0, 2, 1, True), (64, 32, 1, 33, 16, True),
    (70, 8, 3, 4, 2, False),
    # more than 512 nodes: tiles of 16 on the matrix cores, every width and stretch of degrees
    (520, 64, 3, 10, 1, False), (530, 64, 3, 8, 2, True), (515, 128, 3, 3, 2, True), (529, 32, 3, 8, 4, True),
    (521, 16, 3, 5, 2, True), (600, 8, 3, 6, 2, True), (517, 128, 0, 4, 2, True), (700, 64, 0, 9, 1, False),
    (540, 32, 1, 33, 5, True), (523, 64, 1, 7, 2, True), (531, 128, 1, 2, 1, False), (513, 32, 2, 4, 2, True),
    (518, 64, 2, 3, 1, True), (514, 16, 2, 256, 2, True), (519, 32, 4, 3, 2, True), (516, 64, 4, 4, 1, False),
    (513, 16, 5, 3, 2, True), (515, 8, 6, 4, 3, True), (514, 64, 6, 2, 2, True)])
def test_expert_linear(N, C, lmax, X, k, gates, x):
    eq = _eq()
    _say("experts N=%d C=%d lmax=%d X=%d k=%d %s" % (N, C, lmax, X, k, x))
    import torch

    m = Mix(N, C, lmax, X, k, x, gates, seed=N + C)
    plan = eq.eqtp_expert_plan(m.ti, X)
    o, grads = m.check(eq, plan, out="bf16" if x == "bf16" and lmax == 3 else "f32")
    # without a plan, and in another order: the same bits
    p = eq.eqtp_expert_linear(m.h[0], m.W[0], m.ti, lmax, weight=m.w[0], out=torch.empty_like(o),
                              out_dtype=_code(eq, "bf16" if o.dtype == torch.bfloat16 else "f32"))
    assert torch.equal(o, p)
    back = (torch.arange(N - 1, -1, -1, dtype=torch.int32, device="cuda"),) + plan[1:]
    for a, b in zip(grads, m.grads(eq, back)):
        assert torch.equal(a, b)


def _plan_want(idx, X):
    flat = np.where((idx >= 0) & (idx < X), idx, X).reshape(-1)
    slots = np.argsort(flat, kind="stable")
    return slots, np.searchsorted(flat[slots], np.arange(X + 1))


@pytest.mark.parametrize("N,k,X", [(0, 2, 4), (1, 1, 1), (1, 16, 256), (255, 1, 7), (256, 2, 8), (1000, 2, 31), (3000, 3, 32),
                                   (20011, 2, 64), (50000, 1, 256), (5, 4, 2)])
def test_expert_plan(N, k, X):
    eq = _eq()
    _say("expert plan N=%d k=%d X=%d" % (N, k, X))
    import torch

    idx = np.random.default_rng(N + k).integers(-2, X + 2, (N, k)).astype(np.int32)
    order, slots, ptr = (t.cpu().numpy() for t in eq.eqtp_expert_plan(torch.from_numpy(idx).cuda(), X))
    want, ends = _plan_want(idx, X)
    np.testing.assert_array_equal(slots, want)
    np.testing.assert_array_equal(ptr, ends)
    np.testing.assert_array_equal(np.sort(order), np.arange(N))
    if k > 1 and N:  # nodes by their lowest expert, and by the next one where the bins tell them apart
        e = np.sort(np.where((idx >= 0) & (idx < X), idx, X), axis=1)[order]
        assert (np.diff(e[:, 0]) >= 0).all()
        if (X + 1) ** 2 <= 1024:
            second = np.array([min([v for v in row if v > row[0]], default=X) for row in e])
            same = np.diff(e[:, 0]) == 0
            assert (np.diff(second)[same] >= 0).all()


@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_expert_same_index_twice(x):
    """The same expert twice in a node's list adds its weights; both places get their gradient."""
    eq = _eq()
    _say("experts, the same twice, %s" % x)
    m = Mix(20, 32, 2, 3, 3, x, True, seed=2)
    import torch

    m.idx[:] = np.array([2, 2, 0])
    m.idx[5] = [1, 1, 1]
    m.ti = torch.from_numpy(m.idx).cuda()
    m.check(eq, eq.eqtp_expert_plan(m.ti, 3))


def test_expert_nobody():
    """Nodes without an expert: zeros, whatever the features hold; a NaN stays in its own node."""
    eq = _eq()
    _say("experts, nobody")
    import torch

    m = Mix(40, 16, 3, 4, 2, "f32", True, seed=4, holes=False)
    m.ti[::2] = -1
    m.ti[1::4] = 9
    h = m.h[0].clone()
    h[0], h[3] = float("nan"), float("inf")
    m.ti[3] = 1
    plan = eq.eqtp_expert_plan(m.ti, 4)
    out = eq.eqtp_expert_linear(h, m.W[0], m.ti, 3, weight=m.w[0], plan=plan)
    assert (out[::2] == 0).all() and (out[1::4] == 0).all() and not torch.isfinite(out[3]).any()
    assert torch.isfinite(out[4:]).all() and torch.isfinite(out[:3]).all()
    m.ti[:] = -1
    gh, gW, gw = m.grads(eq, eq.eqtp_expert_plan(m.ti, 4))
    assert (gh == 0).all() and (gW == 0).all() and (gw == 0).all()


@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_expert_many_places(x):
    """Several chunks of an expert's places, summed in a fixed order."""
    eq = _eq()
    _say("experts, many places, %s" % x)
    import torch

    m = Mix(1500, 8, 1, 3, 2, x, True, seed=6)
    plan = eq.eqtp_expert_plan(m.ti, 3)
    _, grads = m.check(eq, plan)
    for a, b in zip(grads, m.grads(eq, plan)):
        assert torch.equal(a, b)
    few = m.grads(eq, None, need_h=False)
    assert few[0] is None and torch.equal(few[1], grads[1]) and torch.equal(few[2], grads[2])
    few = m.grads(eq, None, need_W=False, need_weight=False)
    assert few[1] is None and few[2] is None and torch.equal(few[0], grads[0])


@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_expert_is_the_linear(x):
    """One expert without weights is the per-degree linear."""
    eq = _eq()
    _say("experts as the linear, %s" % x)
    import torch

    r = np.random.default_rng(5)
    h, W = _put(r.standard_normal((45, 64, 16)), x), _put(r.standard_normal((1, 4, 64, 64)) / 8, x)
    idx = torch.zeros((45, 1), dtype=torch.int32, device="cuda")
    a = eq.eqtp_expert_linear(h[0], W[0], idx, 3, out_dtype=eq.EQTP_F32)
    b = eq.eqtp_linear(h[0], W[0][0].contiguous(), 3, _code(eq, x))
    want, size = ref.expert(h[1], W[1], np.zeros((45, 1), int), 3)
    _within(_get(a), _get(b), 2 * ref.expert_bound(want, size, 64, 1, ref.U32), "out")


def test_expert_empty():
    eq = _eq()
    _say("experts, no nodes")
    m = Mix(0, 16, 1, 3, 2, "f32", True)
    plan = eq.eqtp_expert_plan(m.ti, 3)
    assert eq.eqtp_expert_linear(m.h[0], m.W[0], m.ti, 1, weight=m.w[0], plan=plan).shape == (0, 16, 4)
    gh, gW, gw = m.grads(eq, plan)
    assert gh.shape == (0, 16, 4) and (gW == 0).all() and gw.shape == (0, 2)


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("N,C,lmax,k,gates", [(20, 16, 1, 1, False), (600, 64, 3, 1, False), (600, 32, 0, 1, False),
                                              (530, 8, 2, 1, False), (600, 64, 3, 2, True), (520, 32, 4, 1, False)])
def test_an_expert_that_is_not_finite(N, C, lmax, k, gates, x):
    """Its nodes get what it holds, the others' bits are those that they have without it."""
    import torch

    eq = _eq()
    _say("an expert that is not finite, N=%d C=%d lmax=%d k=%d %s" % (N, C, lmax, k, x))
    m = Mix(N, C, lmax, 4, k, x, gates, seed=N + lmax)
    W = m.W[0]
    bad = W.clone()
    bad[2, :, ::2] = float("nan")
    bad[2, :, 1::2] = float("inf")
    meets = (m.ti == 2).any(1)
    none = ((m.ti < 0) | (m.ti >= 4)).all(1)
    assert meets.any() and not meets.all()
    for plan in (None, eq.eqtp_expert_plan(m.ti, 4)):
        outs = []
        for weights in (W, bad):
            o = eq.eqtp_expert_linear(m.h[0], weights, m.ti, lmax, weight=m.w[0], plan=plan)
            gh, _, gw = eq.eqtp_expert_linear_backward(m.h[0], weights, m.ti, m.g[0], lmax, weight=m.w[0], plan=plan, need_W=False)
            outs.append((o, gh, gw))
        for clean, spoilt in zip(*outs):
            if clean is not None:
                assert torch.equal(clean[~meets], spoilt[~meets])
        assert not torch.isfinite(outs[1][0][meets]).any()
        assert not outs[1][0][none].any() and not outs[1][1][none].any()


@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_infinities_are_no_nan(x):
    """An infinite feature's gradients are infinite where no term of the sum is of the other sign."""
    import torch

    eq = _eq()
    _say("infinite features %s" % x)
    dt = torch.bfloat16 if x == "bf16" else torch.float32
    N, C, lmax = 5, 8, 1
    h = torch.ones(N, C, 4, dtype=dt, device="cuda")
    h[N - 1, 3, 0] = float("inf")
    g = torch.ones(N, C, 4, dtype=dt, device="cuda")
    W = torch.ones(1, 2, C, C, dtype=dt, device="cuda")
    idx = torch.zeros(N, 1, dtype=torch.int32, device="cuda")
    _, gW, _ = eq.eqtp_expert_linear_backward(h, W, idx, g, lmax)
    want = torch.full((1, 2, C, C), 5.0, device="cuda")
    want[:, 1] = 15.0
    want[0, 0, :, 3] = float("inf")
    assert torch.equal(gW, want)
    g[0, 0, 0] = float("inf")
    w = torch.ones(N, 1, device="cuda")
    _, _, gw = eq.eqtp_expert_linear_backward(torch.ones_like(h), W, idx, g, lmax, weight=w, need_W=False)
    assert torch.equal(gw[:, 0], torch.tensor([float("inf")] + [4.0 * C * C] * (N - 1), device="cuda"))


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("N,C,lmax,k", [(1, 8, 1, 2), (40, 64, 3, 2), (600, 64, 3, 1), (600, 64, 3, 2), (530, 128, 3, 1),
                                        (520, 8, 2, 1), (700, 16, 0, 1), (515, 32, 5, 2)])
def test_both_types_of_the_output(N, C, lmax, k, x):
    """One fp32 sum, rounded once: the bf16 output is the fp32 one's rounding, with and without a plan."""
    import torch

    eq = _eq()
    _say("both types of the output, N=%d C=%d lmax=%d k=%d %s" % (N, C, lmax, k, x))
    m = Mix(N, C, lmax, 5, k, x, k > 1, seed=N + C + lmax)
    for plan in (None, eq.eqtp_expert_plan(m.ti, 5)):
        wide, narrow = (eq.eqtp_expert_linear(m.h[0], m.W[0], m.ti, lmax, weight=m.w[0], plan=plan, out_dtype=t)
                        for t in (eq.EQTP_F32, eq.EQTP_BF16))
        assert torch.equal(wide.to(torch.bfloat16), narrow)


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("lmax", [0, 1, 3, 4])
def test_infinities_under_gates(lmax, x):
    """Infinite features and gradients under gates whose products with them fill more than one bf16: the weights'
    gradients are infinite where they enter a sum, as those without gates are, and nowhere else; NaN stays NaN."""
    import torch

    eq = _eq()
    _say("infinities under gates, lmax=%d %s" % (lmax, x))
    dt = torch.bfloat16 if x == "bf16" else torch.float32
    N, C, K = 9, 16, (lmax + 1) ** 2
    for gate in (0.3, 1.0 / 3.0, 0.7, 0.5):
        h, g = (torch.ones(N, C, K, dtype=dt, device="cuda") for _ in range(2))
        W = torch.ones(2, lmax + 1, C, C, dtype=dt, device="cuda")
        idx = torch.zeros(N, 1, dtype=torch.int32, device="cuda")
        idx[6:] = 1
        w = torch.full((N, 1), gate, device="cuda")
        back = lambda: eq.eqtp_expert_linear_backward(h, W, idx, g, lmax, weight=w, need_h=False, need_weight=False)[1]
        clean = back()
        assert torch.isfinite(clean).all()
        want = clean.clone()
        h[4, 3, K - 1] = float("inf")
        want[0, lmax, :, 3] = float("inf")
        assert torch.equal(back(), want)
        g[5, 7, K - 1] = -float("inf")
        want[0, lmax, 7, :] = -float("inf")
        got = back()
        assert torch.isnan(got[0, lmax, 7, 3])  # inf - inf
        got[0, lmax, 7, 3] = want[0, lmax, 7, 3] = 0.0
        assert torch.equal(got, want)
        h[4, 3, K - 1] = float("nan")
        got = back()
        assert torch.isnan(got[0, lmax, :, 3]).all()
        got[0, lmax, :, 3] = want[0, lmax, :, 3] = 0.0
        assert torch.equal(got, want)


def test_products_beyond_the_largest_bf16():
    """A gate's product with a gradient that fp32 holds and bf16 does not."""
    import torch

    eq = _eq()
    _say("products beyond the largest bf16")
    big = float(torch.finfo(torch.bfloat16).max)
    N, C = 6, 16
    h = torch.full((N, C, 1), 2.0 ** -40, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(N, C, 1, dtype=torch.bfloat16, device="cuda")
    g[2, 5], g[4, 6] = big, -big
    W = torch.ones(1, 1, C, C, dtype=torch.bfloat16, device="cuda")
    idx = torch.zeros(N, 1, dtype=torch.int32, device="cuda")
    w = torch.full((N, 1), 1.0035, device="cuda")
    gW = eq.eqtp_expert_linear_backward(h, W, idx, g, 0, weight=w, need_h=False, need_weight=False)[1]
    want = (w.double()[:, :, None] * g.double()).sum(0) @ h.double()[0].t()
    assert float((w * big).max()) < float("inf")
    # a term in two parts: 2^-16 of it; the other five are as nothing, or 1: six additions
    assert ((gW[0, 0].double() - want).abs() <= (2.0 ** -16 + 8 * 2.0 ** -24) * want.abs()).all()


@pytest.mark.parametrize("N,C,lmax", [(1, 64, 3), (3, 32, 0), (2, 16, 6), (1, 128, 1), (2, 64, 2), (1, 8, 4), (2, 32, 5)])
def test_gated_gradients_keep_fp32(N, C, lmax):
    """Few terms, so that what a term loses shows: a gate's product with a bf16 gradient keeps its 24 bits.  Each enters as
    three products, so a sum has three additions a term, which may cut (two half steps), and the gate's product is rounded."""
    eq = _eq()
    _say("gated gradients keep fp32, N=%d C=%d lmax=%d" % (N, C, lmax))
    m = Mix(N, C, lmax, 2, 2, "bf16", True, seed=C + lmax, holes=False)
    m.idx[:] = [0, 1]
    m.ti.copy_(m.ti.new_tensor(m.idx))
    gW = _get(m.grads(eq, eq.eqtp_expert_plan(m.ti, 2))[1])
    for e in range(2):
        for l in range(lmax + 1):
            s = slice(l * l, (l + 1) ** 2)
            t = m.w[1][:, e, None, None] * m.g[1][:, :, s]
            want = np.tensordot(t, m.h[1][:, :, s], axes=((0, 2), (0, 2)))
            size = np.tensordot(np.abs(t), np.abs(m.h[1][:, :, s]), axes=((0, 2), (0, 2)))
            _within(gW[e, l], want, ref.u * (6 * N * (2 * l + 1) + 3) * size, "grad_W")


def _far_reference(m):
    """The statement of mix_reference, expert by expert: (out, grad_h, grad_W, grad_weight), the sums of their terms'
    sizes, and each expert's places."""
    h, W, g = m.h[1], m.W[1], m.g[1]
    N, C, K = h.shape
    w = np.ones(m.idx.shape) if m.w[1] is None else m.w[1]
    vals = [np.zeros_like(h), np.zeros_like(h), np.zeros_like(W), np.zeros(m.idx.shape)]
    sizes, places = [np.zeros_like(v) for v in vals], np.zeros(m.X)
    for j in range(m.k):
        for e in range(m.X):
            n = np.nonzero(m.idx[:, j] == e)[0]
            places[e] += len(n)
            for l in range(m.lmax + 1):
                s = slice(l * l, (l + 1) ** 2)
                hl, gl, wl = h[n][:, :, s], g[n][:, :, s], w[n, j][:, None, None]
                for v, f in ((vals, lambda t: t), (sizes, np.abs)):
                    A, a, b, c = f(W[e, l]), f(hl), f(gl), f(wl)
                    y = np.matmul(A, a)
                    v[0][n, :, s] += c * y
                    v[1][n, :, s] += c * np.matmul(A.T, b)
                    v[2][e, l] += np.tensordot(c * b, a, axes=((0, 2), (0, 2)))
                    v[3][n, j] += (b * y).sum((1, 2))
    return vals, sizes, places


def test_far_reference_is_the_statement():
    m = Mix(7, 8, 2, 3, 2, seed=1)
    vals, _, _ = _far_reference(m)
    np.testing.assert_allclose(vals[0], ref.expert(m.h[1], m.W[1], m.idx, 2, m.w[1])[0], rtol=1e-12, atol=1e-13)
    for a, b in zip(vals[1:], ref.expert_backward(m.h[1], m.W[1], m.idx, m.g[1], 2, m.w[1])[0]):
        np.testing.assert_allclose(a, b, rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("k,gates", [(1, False), (2, True)])
@pytest.mark.parametrize("N,C,lmax", [(600, 128, 2), (530, 128, 3), (545, 128, 4), (521, 128, 5), (518, 128, 6), (600, 128, 1),
                                      (533, 64, 4), (520, 64, 5), (517, 32, 6)])
def test_expert_wide(N, C, lmax, k, gates, x):
    """The widest rows in the tiles' forms: every degree at 128 channels."""
    eq = _eq()
    _say("experts, wide, N=%d C=%d lmax=%d k=%d %s" % (N, C, lmax, k, x))
    m = Mix(N, C, lmax, 4, k, x, gates, seed=N + lmax)
    vals, sizes, places = _far_reference(m)
    K, u = (lmax + 1) ** 2, ref.u
    half = ref.U16 if x == "bf16" else u
    plan = eq.eqtp_expert_plan(m.ti, 4)
    for p in (plan, None):
        o = eq.eqtp_expert_linear(m.h[0], m.W[0], m.ti, lmax, weight=m.w[0], plan=p, out_dtype=eq.EQTP_F32)
        _within(_get(o), vals[0], ref.expert_bound(vals[0], sizes[0], C, k, u), "out")
    gh, gW, gw = m.grads(eq, plan)
    # (the bounds of mix_reference.expert_backward)
    _within(_get(gh), vals[1], ref.expert_bound(vals[1], sizes[1], C, k, half), "grad_h")
    terms = places[:, None, None, None] * (2 * lmax + 1)
    _within(_get(gW), vals[2], (2 * u * (terms + 4) + (ref.U16 ** 2 if x == "bf16" and gates else 0.0)) * sizes[2], "grad_W")
    _within(_get(gw), vals[3], 2 * u * (C + 16 * K + 16) * sizes[3], "grad_weight")


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("N,C,lmax,k,gates", [(30, 64, 3, 2, True), (600, 64, 3, 1, False), (600, 64, 3, 2, True), (600, 32, 0, 1, False),
                                              (530, 8, 2, 3, True), (520, 32, 4, 1, False), (520, 32, 5, 2, True),
                                              (515, 128, 2, 2, True)])
def test_a_node_that_is_not_finite(N, C, lmax, k, gates, x):
    """NaN and infinities in a node's features and gradients stay in its own rows and in its experts' weight gradients."""
    import torch

    eq = _eq()
    _say("a node that is not finite, N=%d C=%d lmax=%d k=%d %s" % (N, C, lmax, k, x))
    m = Mix(N, C, lmax, 5, k, x, gates, seed=N + lmax + k)
    bad = [3, N // 2, N - 1]
    for i, n in enumerate(bad):
        m.ti[n] = 2 if i < 2 else 3
    plan = eq.eqtp_expert_plan(m.ti, 5)
    h, g = m.h[0].clone(), m.g[0].clone()
    for n, v in zip(bad, ("nan", "inf", "nan")):
        h[n] = float(v)
        g[n] = float(v)
    keep = torch.ones(N, dtype=torch.bool, device="cuda")
    keep[bad] = False
    runs = []
    for a, b in ((m.h[0], m.g[0]), (h, g)):
        o = eq.eqtp_expert_linear(a, m.W[0], m.ti, lmax, weight=m.w[0], plan=plan)
        runs.append((o,) + eq.eqtp_expert_linear_backward(a, m.W[0], m.ti, b, lmax, weight=m.w[0], plan=plan))
    for i, (clean, spoilt) in enumerate(zip(*runs)):
        if clean is None:
            continue
        if i == 2:  # the weights' gradient, by expert
            assert torch.equal(clean[[0, 1, 4]], spoilt[[0, 1, 4]]) and not torch.isfinite(spoilt[[2, 3]]).any()
        else:
            assert torch.equal(clean[keep], spoilt[keep]) and not torch.isfinite(spoilt[bad]).any()
