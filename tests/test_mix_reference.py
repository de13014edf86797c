"""The 64-bit statements themselves: gradients against differences, invariances."""
import numpy as np
import pytest

import mix_reference as ref
from test_oracle_conv import _apply_D, _rotation, _wigner_blocks


def _differences(f, x, g, eps=1e-6):
    """d/dx of sum(g f(x)), central differences."""
    out = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += eps
        b[i] -= eps
        out[i] = ((f(a) - f(b)) * g).sum() / (2 * eps)
    return out


def test_distance_bias_gradient():
    r = np.random.default_rng(0)
    vec, bounds = r.standard_normal((40, 3)), np.array([0.5, 1.0, 1.7])
    table, g = r.standard_normal((4, 3)), r.standard_normal((40, 3))
    live = np.linalg.norm(vec, axis=1) < 2.0
    f = lambda t: np.where(live[:, None], ref.distance_bias(vec, bounds, t, 2.0), 0.0)
    got, _ = ref.distance_bias_backward(vec, bounds, g, 4, 2.0)
    np.testing.assert_allclose(got, _differences(f, table, g), rtol=1e-7, atol=1e-8)


@pytest.mark.parametrize("lmax,heads,w,axes", [(0, 2, 4, 1), (1, 1, 2, 3), (2, 2, 3, 0), (1, 2, 6, 2)])
def test_head_norm_gradient(lmax, heads, w, axes):
    r = np.random.default_rng(1)
    K = (lmax + 1) ** 2
    x, g = r.standard_normal((2, heads * w, K)), r.standard_normal((2, heads * w, K))
    weight = 1 + 0.2 * r.standard_normal((lmax + 1, w))
    freq = r.standard_normal((axes, max(1, w // 2 - 1))) if axes else None
    pos = r.standard_normal((2, axes)) if axes else None
    f = lambda **kw: ref.head_norm(**dict(dict(x=x, heads=heads, lmax=lmax, weight=weight, pos=pos, freq=freq), **kw))["out"].reshape(x.shape)
    (gx, gw, gp), _ = ref.head_norm_backward(x, g, heads, lmax, weight, pos, freq)
    np.testing.assert_allclose(gx, _differences(lambda t: f(x=t), x, g), rtol=1e-6, atol=1e-7)
    np.testing.assert_allclose(gw, _differences(lambda t: f(weight=t), weight, g), rtol=1e-6, atol=1e-7)
    if axes:
        np.testing.assert_allclose(gp, _differences(lambda t: f(pos=t), pos, g), rtol=1e-6, atol=1e-7)
        # inner products of turned rows depend on differences of positions
        q, k = r.standard_normal((2, 1, heads * w, K))
        at = lambda t, p: ref.head_norm(t, heads, lmax, weight, p, freq)["out"]
        p, o, s = r.standard_normal((3, 1, axes))
        np.testing.assert_allclose((at(q, p) * at(k, o)).sum(), (at(q, p + s) * at(k, o + s)).sum(), rtol=1e-9)


@pytest.mark.parametrize("lmax", [0, 1, 3])
def test_head_norm_in_turned_space(lmax):
    """With freq turned as the positions are, the result turns with space as the features do and gradients of positions
    turn with the positions; with freq held fixed, logits depend on the orientation."""
    r = np.random.default_rng(4)
    heads, w, K = 2, 6, (lmax + 1) ** 2
    Q = _rotation(lmax)
    D = _wigner_blocks(Q, lmax)
    x, g = r.standard_normal((2, 5, heads * w, K))
    weight, freq, pos = 1 + 0.2 * r.standard_normal((lmax + 1, w)), r.standard_normal((3, 2)), r.standard_normal((5, 3))
    at = lambda t, p, f: ref.head_norm(t, heads, lmax, weight, p, f)["out"].reshape(x.shape)  # noqa: E731
    out, turned = at(x, pos, freq), at(_apply_D(D, x), pos @ Q.T, Q @ freq)
    np.testing.assert_allclose(turned, _apply_D(D, out), atol=1e-12)
    (gx, gw, gpos), _ = ref.head_norm_backward(x, g, heads, lmax, weight, pos, freq)
    (tx, tw, tpos), _ = ref.head_norm_backward(_apply_D(D, x), _apply_D(D, g), heads, lmax, weight, pos @ Q.T, Q @ freq)
    np.testing.assert_allclose(tx, _apply_D(D, gx), atol=1e-12)
    np.testing.assert_allclose(tw, gw, atol=1e-12)
    np.testing.assert_allclose(tpos, gpos @ Q.T, atol=1e-12)
    logit = lambda y: (y[0] * y[1]).sum()  # noqa: E731
    np.testing.assert_allclose(logit(turned), logit(out), atol=1e-11)
    assert abs(logit(at(_apply_D(D, x), pos @ Q.T, freq)) - logit(out)) > 1e-3


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renormalise", [False, True])
def test_route_gradient(sigmoid, renormalise):
    r = np.random.default_rng(2)
    t, g = r.standard_normal((5, 6)), r.standard_normal((5, 3))
    bias = 0.1 * r.standard_normal(6)
    idx, w, _ = ref.route(t, 3, sigmoid, bias, 2, 2, renormalise, 1.5)
    f = lambda z: ref.route(z, 3, sigmoid, bias, 2, 2, renormalise, 1.5)[1]
    np.testing.assert_allclose(ref.route_backward(t, idx, g, sigmoid, renormalise, 1.5)[0], _differences(f, t, g), rtol=1e-6,
                               atol=1e-8)


def test_route_choice():
    t = np.array([[1.0, 3.0, 3.0, 2.0], [-np.inf, 0.0, -np.inf, -np.inf], [0.0, np.nan, 1.0, 2.0]])
    idx, w, _ = ref.route(t, 2)
    assert idx.tolist() == [[1, 2], [1, -1], [-1, -1]] and w[1].tolist() == [1.0, 0.0] and np.isnan(w[2]).all()
    # two groups: the better pair stays open
    idx, _, _ = ref.route(np.array([[5.0, -9.0, 3.0, 3.0]]), 2, True, np.zeros(4), 2, 1)
    assert idx.tolist() == [[2, 3]]


def test_expert_gradient():
    r = np.random.default_rng(3)
    h, g = r.standard_normal((2, 3, 2, 4))
    W, w = r.standard_normal((3, 2, 2, 2)), r.standard_normal((3, 2))
    idx = np.array([[0, 2], [1, 1], [2, -1]])
    (gh, gW, gw), _ = ref.expert_backward(h, W, idx, g, 1, w)
    np.testing.assert_allclose(gh, _differences(lambda t: ref.expert(t, W, idx, 1, w)[0], h, g), rtol=1e-6, atol=1e-7)
    np.testing.assert_allclose(gW, _differences(lambda t: ref.expert(h, t, idx, 1, w)[0], W, g), rtol=1e-6, atol=1e-7)
    np.testing.assert_allclose(gw, _differences(lambda t: ref.expert(h, W, idx, 1, t)[0], w, g), rtol=1e-6, atol=1e-7)
