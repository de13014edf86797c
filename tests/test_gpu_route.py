"""Routing on the GPU against the 64-bit statement: the choice exactly, weights
and gradients within bounds derived in mix_reference."""
import numpy as np
import pytest

import mix_reference as ref
from test_gpu_norm import _get, _put, _within
from test_gpu_parity import _eq, _say

pytestmark = pytest.mark.gpu


def _check(eq, t, k, x="f32", bias=None, groups=1, top=None, sigmoid=False, renorm=True, scale=1.0, seed=0, shift=0):
    t, values = _put(t, x, shift)
    b = None if bias is None else _put(bias)
    how = dict(score=eq.EQTP_SCORE_SIGMOID if sigmoid else eq.EQTP_SCORE_SOFTMAX, renormalise=renorm, scale=scale)
    idx, weight = eq.eqtp_route(t, k, bias=None if b is None else b[0], groups=groups, top_groups=top, **how)
    want, ww, _ = ref.route(values, k, sigmoid, None if b is None else b[1], groups, top, renorm, scale)
    np.testing.assert_array_equal(_get(idx), want)
    bound = ref.route_bound(values, k)
    good = ~np.isnan(ww).any(1)
    got = _get(weight)
    assert np.isnan(got[~good]).all()
    _within(got[good], ww[good], bound[good, None] * np.abs(ww[good]) + 1e-37, "weight")
    g = _put(np.random.default_rng(seed).standard_normal(ww.shape))
    gt = eq.eqtp_route_backward(t, idx, g[0], **how)
    gl, size = ref.route_backward(values, want, g[1], sigmoid, renorm, scale)
    half = ref.U16 if x == "bf16" else ref.U32
    got = _get(gt)
    _within(got[good], gl[good], 3 * bound[good, None] * size[good] + half * np.abs(gl[good]) + 1e-37, "grad_logits")
    return idx, weight


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("N,X,k,groups,top,biased", [
    (1, 1, 1, 1, 1, False), (1, 256, 16, 1, 1, True), (33, 2, 2, 1, 1, True), (100, 8, 2, 1, 1, False), (257, 9, 4, 3, 2, True),
    (64, 64, 6, 8, 4, True), (31, 17, 5, 1, 1, True), (20, 33, 8, 11, 3, False), (40, 128, 8, 8, 3, True),
    (9, 160, 16, 2, 1, False), (12, 250, 3, 125, 7, True), (5, 16, 16, 1, 1, True), (7, 24, 8, 24, 9, True)])
def test_route(N, X, k, groups, top, biased, sigmoid, renorm, x):
    eq = _eq()
    _say("route N=%d X=%d k=%d groups=%d" % (N, X, k, groups))
    r = np.random.default_rng(N * X + k)
    _check(eq, 1.5 * r.standard_normal((N, X)), k, x, 0.1 * r.standard_normal(X) if biased else None, groups, top, sigmoid,
           renorm, 2.5, seed=N)


@pytest.mark.parametrize("X", [3, 8, 11, 64, 200])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_ties(X, sigmoid):
    """Equal scores: the lower index goes first, whatever the lanes; all logits equal; a lead by a hair counts."""
    eq = _eq()
    _say("route ties X=%d" % X)
    r = np.random.default_rng(X)
    t = r.integers(0, 2, (50, X)).astype(np.float64)
    t[0] = 0.25
    for groups, top, bias in ((1, 1, None), (1, 1, np.zeros(X)), (X, X // 2, None)):
        _check(eq, t, min(3, X), bias=bias, groups=groups, top=top, sigmoid=sigmoid)
    # a bias, and logits one step apart: scores closer than fp32 tells apart
    t = np.full((4, X), 0.125, dtype=np.float32)
    t[1, X - 1] = np.nextafter(np.float32(0.125), np.float32(1))
    t[2, 0] = np.nextafter(np.float32(0.125), np.float32(0))
    t[3, X // 2:] = np.nextafter(np.float32(0.125), np.float32(1))
    idx, _ = _check(eq, t, 2, bias=np.full(X, 0.5), sigmoid=sigmoid)
    assert idx[1, 0] == X - 1 and idx[2, 0] == 1 and idx[3, 0] == X // 2


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_masks(sigmoid, renorm):
    """Masked experts, rows that a mask leaves empty, biases of -inf, NaN in a row, far logits."""
    eq = _eq()
    _say("route masks")
    r = np.random.default_rng(4)
    t = r.standard_normal((12, 12))
    t[1] = -np.inf
    t[2, 1:] = -np.inf
    t[3, ::2] = -np.inf
    t[4, 5] = np.nan
    t[5] = -80.0 + r.standard_normal(12)
    t[6] = 80.0 + r.standard_normal(12)
    t[7] = -np.finfo(np.float32).max
    t[8, :6] = -np.inf
    for bias, groups, top in ((None, 1, 1), (np.where(np.arange(12) == 3, -np.inf, 0.05), 1, 1), (np.zeros(12), 4, 2), (None, 2, 1)):
        idx, w = _check(eq, t, 4, bias=bias, groups=groups, top=top, sigmoid=sigmoid, renorm=renorm)
        assert (idx[1] == -1).all() and (w[1] == 0).all() and idx[2].tolist() in ([0, -1, -1, -1],)
        assert (idx[4] == -1).all()


def test_route_far_below():
    """Sigmoid scores that are 0 in fp32 still have weights beside each other."""
    eq = _eq()
    _say("route, far below")
    t = np.array([[-200.0, -200.5, -203.0, -400.0]])
    _check(eq, t, 3, sigmoid=True)


def test_route_less_aligned():
    eq = _eq()
    _say("route, less aligned")
    r = np.random.default_rng(9)
    for X in (8, 12, 64, 65):
        _check(eq, r.standard_normal((70, X)), 3, "bf16", shift=1)
        _check(eq, r.standard_normal((70, X)), 3, "f32", shift=3, sigmoid=True)


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("X", [3, 8, 9, 64, 200])
def test_route_zeros_of_both_signs(X, sigmoid, x):
    """0 and -0 are equal: the lower index goes first, within a lane's experts and across lanes.  In rows without other
    ties, alone and side by side (a tie in a row has its neighbours looked at again, too)."""
    eq = _eq()
    _say("route, zeros of both signs, X=%d %s" % (X, x))
    for at in {(0, 1), (0, X - 1), (X // 2, X - 1), (X // 3, X // 2 + 1)}:
        for top in (True, False):  # the zeros are the largest, or stand behind another
            t = -1.0 - np.arange(X) % 100 - 0.25 * (np.arange(X) // 100)
            t[at[0]], t[at[1]] = -0.0, 0.0
            if not top:
                t[[i for i in range(X) if i not in at][-1]] = 2.0
            for rows in (1, 70):
                for k in (1, min(2, X), min(3, X)):
                    idx, _ = _check(eq, np.tile(t, (rows, 1)), k, x, sigmoid=sigmoid)
                    assert not top or (idx[:, 0] == at[0]).all()
    t = np.full((1, X), -0.0)
    t[0, X - 1] = 0.0
    for groups, bias in ((1, None), (1, np.where(np.arange(X) % 2, 0.0, -0.0)), (X, None)):
        idx, _ = _check(eq, t, 1, x, bias=bias, groups=groups, sigmoid=sigmoid)
        assert int(idx[0, 0]) == 0
