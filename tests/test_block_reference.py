"""The 64-bit statements the transformer-block tests compare with: gradients
against central differences, the random words against published values,
rotation behaviour."""
import numpy as np
import pytest

import block_reference as ref


def _directional(f, x, d, h=1e-5):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("lmax,C", [(0, 7), (2, 5), (4, 3)])
def test_norm_gradient_against_differences(lmax, C):
    r = np.random.default_rng(3 + lmax)
    K = (lmax + 1) ** 2
    x, g, d = (r.standard_normal((4, C, K)) for _ in range(3))
    w, b, dw, db = r.standard_normal((lmax + 1, C)), r.standard_normal(C), r.standard_normal((lmax + 1, C)), r.standard_normal(C)
    gx, gw, gb = ref.norm_backward(x, lmax, g, w)
    assert np.isclose((gx * d).sum(), _directional(lambda t: (ref.norm(t, lmax, w, b)[0] * g).sum(), x, d), rtol=1e-7)
    assert np.isclose((gw * dw).sum(), _directional(lambda t: (ref.norm(x, lmax, t, b)[0] * g).sum(), w, dw), rtol=1e-7)
    assert np.isclose((gb * db).sum(), _directional(lambda t: (ref.norm(x, lmax, w, t)[0] * g).sum(), b, db), rtol=1e-7)


def test_norm_commutes_with_rotations():
    """An orthogonal map inside each degree commutes with the norm (the scalars stay)."""
    r = np.random.default_rng(5)
    lmax, C = 3, 6
    x = r.standard_normal((5, C, 16))
    w, b = r.standard_normal((4, C)), r.standard_normal(C)
    R = np.zeros((16, 16))
    for l in range(lmax + 1):
        s = slice(l * l, (l + 1) ** 2)
        R[s, s] = np.eye(1) if l == 0 else np.linalg.qr(r.standard_normal((2 * l + 1, 2 * l + 1)))[0]
    a = ref.norm(x @ R.T, lmax, w, b)[0]
    assert np.allclose(a, ref.norm(x, lmax, w, b)[0] @ R.T, atol=1e-13)


def test_philox_published_words():
    """The known answers that accompany the method's paper (ten rounds, 4x32)."""
    assert ref.philox((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    f = 0xFFFFFFFF
    assert ref.philox((f, f, f, f), (f, f)) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert ref.philox((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_keep_mask_rate():
    keep = ref.keep_mask(7, 9, 100, 100, 0.3)
    assert abs(keep.mean() - 0.7) < 5 * np.sqrt(0.21 / 1e4)
    assert ref.keep_mask(7, 9, 3, 5, 0.0).all()


def _small(seed, heads, kv_heads, D, masked=False):
    r = np.random.default_rng(seed)
    N, M = 4, 5
    row_ptr = np.array([0, 3, 3, 7, 9])
    src = r.integers(0, M, 9)
    q, g = (r.standard_normal((N, heads * D, 1)) for _ in range(2))
    k, v = (r.standard_normal((M, kv_heads * D, 1)) for _ in range(2))
    bias = r.standard_normal((9, heads))
    if masked:
        bias[4] = -np.inf
        bias[7:] = -np.inf
    return q, k, v, src, row_ptr, bias, g


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (4, 2), (3, 1)])
@pytest.mark.parametrize("masked", [False, True])
def test_attention_gradient_against_differences(heads, kv_heads, masked):
    q, k, v, src, rp, bias, g = _small(7, heads, kv_heads, 6, masked)
    grads = ref.attention_backward(q, k, v, src, rp, heads, 0.4, g, bias)
    args = [q, k, v, bias]
    r = np.random.default_rng(2)
    for i in range(4):
        d = r.standard_normal(args[i].shape)
        d[~np.isfinite(args[i])] = 0.0

        def f(t):
            a = list(args)
            a[i] = t
            return (ref.attention(a[0], a[1], a[2], src, rp, heads, 0.4, a[3])[0] * g).sum()

        assert np.isclose((grads[i] * d).sum(), _directional(f, args[i], d), rtol=1e-6, atol=1e-9), i


def test_attention_of_equal_logits_is_the_mean():
    q, k, v, src, rp, _, _ = _small(8, 2, 2, 5)
    out, w, lse, _ = ref.attention(np.zeros_like(q), k, v, src, rp, 2, 1.0)
    assert np.allclose(out[0], v[src[:3]].mean(axis=0)) and np.allclose(lse[0], np.log(3))
    assert (out[1] == 0).all() and np.isneginf(lse[1]).all()
