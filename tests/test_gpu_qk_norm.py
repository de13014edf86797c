"""Norm and rotation of queries and keys on the GPU against the 64-bit
statement, within bounds derived in mix_reference."""
import numpy as np
import pytest

import mix_reference as ref
from test_gpu_norm import _get, _put, _within
from test_gpu_parity import _eq, _say

pytestmark = pytest.mark.gpu

HALF = {"f32": ref.U32, "bf16": ref.U16}


class Sides:
    def __init__(self, N, M, lmax, heads, kv, w, x="f32", axes=0, R=0, seed=0, shift=0, far=3.0):
        r = np.random.default_rng(seed)
        K = (lmax + 1) ** 2
        self.N, self.M, self.lmax, self.heads, self.kv, self.x = N, M, lmax, heads, kv, x
        spread = 2.0 / (1.0 + ref.degrees(lmax))
        self.q, self.k = (_put(r.standard_normal((n, h * w, K)) * spread, x, shift) for n, h in ((N, heads), (M, kv)))
        self.gq, self.gk = (_put(r.standard_normal((n, h * w, K)), x, shift) for n, h in ((N, heads), (M, kv)))
        self.wq, self.wk = (_put(1 + 0.3 * r.standard_normal((lmax + 1, w))) for _ in range(2))
        self.pq = self.pk = self.f = (None, None)
        if axes:
            self.pq, self.pk = (_put(far * r.standard_normal((n, axes))) for n in (N, M))
            self.f = _put(r.standard_normal((axes, R)))

    def how(self, weights=True):
        kw = dict(pos_q=self.pq[0], pos_k=self.pk[0], freq=self.f[0])
        return dict(kw, weight_q=self.wq[0], weight_k=self.wk[0]) if weights else kw

    def check(self, eq, weights=True):
        args = (self.q[0], self.k[0])
        outs = eq.eqtp_qk_norm(*args, self.lmax, self.heads, **self.how(weights))
        grads = eq.eqtp_qk_norm_backward(*args, self.gq[0], self.gk[0], self.lmax, self.heads,
                                         need_pos=self.f[0] is not None, **self.how(weights))
        hs = HALF[self.x]
        for i, (x, g, heads, w, pos) in enumerate(((self.q[1], self.gq[1], self.heads, self.wq[1], self.pq[1]),
                                                   (self.k[1], self.gk[1], self.kv, self.wk[1], self.pk[1]))):
            w = w if weights else None
            p = ref.head_norm(x, heads, self.lmax, w, pos, self.f[1])
            _within(_get(outs[i]), p["out"].reshape(x.shape), ref.head_norm_bounds(p, x.shape, hs), "out %d" % i)
            want, bound = ref.head_norm_backward(x, g, heads, self.lmax, w, pos, self.f[1], half_step=hs)
            for j, name in enumerate(("grad", "grad_weight", "grad_pos")):
                if want[j] is not None:
                    _within(_get(grads[2 * j + i]), want[j], bound[j], "%s %d" % (name, i))
        return outs, grads


CASES = [  # N, M, lmax, heads, kv, w, axes, R
    (1, 1, 0, 1, 1, 2, 1, 1), (3, 5, 0, 2, 1, 1, 0, 0), (64, 64, 2, 2, 2, 4, 3, 2), (7, 7, 3, 4, 2, 16, 3, 8),
    (33, 9, 3, 4, 4, 16, 1, 3), (10, 4, 1, 3, 1, 5, 0, 0), (5, 5, 4, 2, 2, 6, 2, 3), (4, 3, 6, 2, 1, 8, 3, 4),
    (3, 2, 6, 1, 1, 41, 0, 0), (3, 2, 5, 1, 1, 56, 3, 17), (2, 3, 4, 1, 1, 80, 1, 40), (200, 100, 0, 8, 2, 128, 1, 64),
    (50, 50, 0, 4, 4, 15, 0, 0), (9, 9, 0, 1, 1, 2048, 3, 1000), (6, 6, 0, 2, 2, 514, 1, 257), (300, 1, 1, 1, 1, 2, 2, 1),
    (1, 40, 2, 1, 3, 30, 1, 15), (17, 17, 3, 2, 2, 128, 3, 64), (2, 2, 2, 1, 1, 226, 1, 113), (40, 40, 0, 16, 4, 6, 1, 3),
    (12, 12, 1, 16, 8, 7, 0, 0), (1000, 1000, 1, 2, 2, 4, 3, 1)]


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_qk_norm(case, x):
    eq = _eq()
    N, M, lmax, heads, kv, w, axes, R = CASES[case]
    _say("qk norm %r %s" % (CASES[case], x))
    import torch

    s = Sides(N, M, lmax, heads, kv, w, x, axes, R, seed=case)
    outs, grads = s.check(eq)
    again = eq.eqtp_qk_norm_backward(s.q[0], s.k[0], s.gq[0], s.gk[0], lmax, heads, need_pos=axes > 0, **s.how())
    assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(grads, again))


@pytest.mark.parametrize("N,lmax,heads,w,axes,R", [(40001, 0, 2, 16, 1, 8), (3001, 3, 4, 8, 3, 4), (9001, 2, 4, 4, 0, 0)])
def test_qk_norm_many_rows(N, lmax, heads, w, axes, R):
    """More rows than the card holds groups at once: a group goes over several nodes and all their heads."""
    eq = _eq()
    _say("qk norm, %d rows" % N)
    Sides(N, N // 3, lmax, heads, heads, w, "f32", axes, R, seed=N).check(eq)


@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_qk_norm_less_aligned_and_without_weights(x):
    eq = _eq()
    _say("qk norm, less aligned, %s" % x)
    Sides(13, 11, 2, 3, 1, 6, x, 2, 3, seed=1, shift=1).check(eq, weights=False)
    Sides(13, 11, 0, 3, 1, 10, x, 2, 5, seed=2, shift=3).check(eq)


def test_qk_norm_far_positions():
    """Angles of hundreds of thousands of turns are as good as near ones."""
    eq = _eq()
    _say("qk norm, far positions")
    Sides(65, 65, 0, 2, 2, 16, "f32", 3, 8, seed=5, far=1e6).check(eq)


def test_qk_norm_in_place_and_single_sides():
    eq = _eq()
    _say("qk norm, in place")
    import torch

    s = Sides(37, 21, 2, 4, 2, 6, "f32", 1, 3, seed=6)
    a, b = eq.eqtp_qk_norm(s.q[0], s.k[0], 2, 4, **s.how())
    q, k = s.q[0].clone(), s.k[0].clone()
    c, d = eq.eqtp_qk_norm(q, k, 2, 4, out_q=q, out_k=k, **s.how())
    assert c is q and d is k and torch.equal(a, c) and torch.equal(b, d)
    grads = eq.eqtp_qk_norm_backward(s.q[0], s.k[0], s.gq[0], s.gk[0], 2, 4, need_pos=True, **s.how())
    only = eq.eqtp_qk_norm_backward(s.q[0], s.k[0], None, s.gk[0], 2, 4, need_pos=True, **s.how())
    assert only[0] is None and only[2] is None and only[4] is None
    for i in (1, 3, 5):
        assert torch.equal(only[i], grads[i])
    few = eq.eqtp_qk_norm_backward(s.q[0], s.k[0], s.gq[0], s.gk[0], 2, 4, need_q=False, need_weight_k=False,
                                   need_pos=True, **s.how())
    assert few[0] is None and few[3] is None
    for i in (1, 2, 4, 5):
        assert torch.equal(few[i], grads[i])
    # no rows on one side, or on both
    e = s.k[0][:0].contiguous()
    o, p = eq.eqtp_qk_norm(s.q[0], e, 2, 4, weight_q=s.wq[0])
    assert p.shape[0] == 0 and torch.equal(o, eq.eqtp_qk_norm(s.q[0], s.q[0], 2, 4, weight_q=s.wq[0])[0])
    z = eq.eqtp_qk_norm_backward(e, e, e, e, 2, 2, need_pos=False)
    assert (z[2] == 0).all() and (z[3] == 0).all() and z[0].shape[0] == 0


def test_qk_norm_spoilt_rows():
    """A NaN or an infinity spoils its own head and degree only; zero rows stay zero."""
    eq = _eq()
    _say("qk norm, NaN")
    import torch

    s = Sides(9, 9, 1, 2, 2, 4, "f32", 1, 2, seed=8)
    q = s.q[0].clone()
    good = eq.eqtp_qk_norm(q, s.k[0], 1, 2, **s.how())[0]
    q[3, 1, 2] = float("nan")  # head 0, degree 1
    q[5] = 0.0
    out = eq.eqtp_qk_norm(q, s.k[0], 1, 2, **s.how())[0]
    bad = torch.isnan(out)
    assert bad[3, :4, 1:].all() and int(bad.sum()) == 12 and (out[5] == 0).all()
    keep = torch.ones(9, dtype=torch.bool)
    keep[[3, 5]] = False
    assert torch.equal(out[keep.cuda()], good[keep.cuda()])


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("lmax,w,axes,R", [(0, 16, 0, 0), (0, 16, 1, 3), (0, 7, 0, 0), (1, 8, 0, 0), (1, 8, 3, 2), (2, 6, 2, 1),
                                           (2, 5, 0, 0), (3, 32, 1, 5), (0, 128, 1, 20)])
def test_qk_norm_channels_that_are_not_turned(lmax, w, axes, R, x):
    """A channel that is not turned is its own: what stands half a head further on (or back) does not reach it, infinite
    or not -- a weight, a feature, a gradient."""
    eq = _eq()
    _say("qk norm, channels that are not turned, lmax=%d w=%d R=%d %s" % (lmax, w, R, x))
    import torch

    s = Sides(6, 5, lmax, 2, 2, w, x, axes, R, seed=w + lmax)
    half = w // 2
    outs = eq.eqtp_qk_norm(s.q[0], s.k[0], lmax, 2, **s.how())
    back = lambda q, g, how: eq.eqtp_qk_norm_backward(q, s.k[0], g, s.gk[0], lmax, 2, need_pos=axes > 0, **how)
    clean = back(s.q[0], s.gq[0], s.how())
    for c in (R, half - 1, half + R, w - 1):  # (the first and the last of those not turned, of either half)
        # an infinite weight: its channel of all nodes and heads, and nothing else
        how = dict(s.how(), weight_q=s.wq[0].clone())
        how["weight_q"][lmax, c] = float("inf")
        got = eq.eqtp_qk_norm(s.q[0], s.k[0], lmax, 2, **how)
        spoilt = torch.zeros_like(got[0], dtype=torch.bool).reshape(6, 2, w, -1)
        spoilt[:, :, c, lmax * lmax:] = True
        spoilt = spoilt.reshape(got[0].shape)
        assert torch.equal(got[0][~spoilt], outs[0][~spoilt]) and torch.equal(got[1], outs[1])
        assert not torch.isfinite(got[0][spoilt]).any()
        # a channel's gradient of infinity: the gradients of its own node's head and degree, and of its own weight
        g = s.gq[0].clone()
        g[2, w + c, lmax * lmax] = float("inf")
        grads = back(s.q[0], g, s.how())
        spoilt = torch.zeros_like(g, dtype=torch.bool)
        spoilt[2, w:, lmax * lmax:] = True
        assert torch.equal(grads[0][~spoilt], clean[0][~spoilt]) and not torch.isfinite(grads[0][spoilt]).any()
        spoilt = torch.zeros_like(grads[2], dtype=torch.bool)
        spoilt[lmax, c] = True
        assert torch.equal(grads[2][~spoilt], clean[2][~spoilt]) and not torch.isfinite(grads[2][spoilt]).any()
        for i in (1, 3, 4, 5):
            assert (grads[i] is None and clean[i] is None) or torch.equal(grads[i], clean[i])
        # an infinite feature: NaN there, zeros in the rest of its degree (the norm is infinite)
        q = s.q[0].clone()
        q[2, w + c, lmax * lmax] = float("inf")
        got = eq.eqtp_qk_norm(q, s.k[0], lmax, 2, **s.how())[0]
        assert torch.isnan(got[2, w + c, lmax * lmax])
        rest = got[2, w:, lmax * lmax:].clone()
        rest[c, 0] = 0.0
        assert (rest == 0).all()
        keep = torch.ones_like(got, dtype=torch.bool)
        keep[2, w:, lmax * lmax:] = False
        assert torch.equal(got[keep], outs[0][keep])


def _group(w, K):
    """(threads, nodes' heads of a workgroup) of the gradient's groups: a quad of half a head's row a thread."""
    quads, per = ((w + 1) // 2 * K + 3) // 4, K // 4 if K % 4 == 0 else K
    for T in (2, 4, 8, 16, 32, 64):
        if T >= (8 if K > 1 else 2) and T >= per and (quads <= T // per * per or T == 64):
            return T, 256 // T


@pytest.mark.parametrize("N,M,lmax,heads,kv,w,axes,R", [
    (40001, 20000, 0, 2, 1, 16, 1, 8), (4001, 1000, 3, 4, 2, 8, 3, 4), (9001, 4500, 2, 4, 4, 4, 0, 0),
    # heads that are no divisor of a workgroup's groups, with gradients of positions: a group takes whole nodes, many of them
    (30001, 9000, 0, 3, 3, 16, 1, 8), (20003, 20003, 1, 3, 1, 4, 3, 1), (8001, 3000, 3, 6, 3, 8, 3, 4),
    (6007, 700, 0, 40, 40, 16, 2, 3), (2503, 2503, 2, 40, 10, 4, 3, 2)])
def test_qk_norm_many_rows_of_a_group(N, M, lmax, heads, kv, w, axes, R):
    """Many rounds of every group, whole nodes among them; the weights' gradients against bounds that count a thread's
    own additions, so that a lost row would show."""
    eq = _eq()
    _say("qk norm, many rows of a group, N=%d heads=%d" % (N, heads))
    import torch

    s = Sides(N, M, lmax, heads, kv, w, "f32", axes, R, seed=N)
    _, grads = s.check(eq)
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    rounds = 256 // _group(w, (lmax + 1) ** 2)[0]
    share = N * heads / (N * heads + M * kv)
    for i, (x, g, rows, h, pos, part) in enumerate(((s.q[1], s.gq[1], N, heads, s.pq[1], share),
                                                    (s.k[1], s.gk[1], M, kv, s.pk[1], 1.0 - share))):
        p = ref.head_norm(x, h, lmax, None, pos, s.f[1])
        g = g.reshape(p["x"].shape)
        t, xhat = g * p["c"] - p["other"](g) * p["s"], p["x"] * p["r"]
        size = (np.abs(g) + np.abs(p["other"](g))) * np.abs(xhat)
        # workgroups: one a compute unit at least, in the ratio of the sides' elements; a head is one addition a place
        groups = max(1, int(cus * part)) * rounds
        adds = -(-rows * h // groups) + h
        for l in range(lmax + 1):
            m = slice(l * l, (l + 1) ** 2)
            _within(_get(grads[2 + i])[l], (t * xhat)[..., m].sum(axis=(0, 1, 3)),
                    ref.u * (30 + adds) * size[..., m].sum(axis=(0, 1, 3)), "grad_weight %d" % i)
