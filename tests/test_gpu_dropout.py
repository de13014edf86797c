"""Counter-based dropout on the GPU: the mask word for word against the plain
statement of the generator, values within half a step of their type."""
import numpy as np
import pytest

import block_reference as ref
from test_gpu_norm import _dt, _get, _put
from test_gpu_parity import _eq, _say

pytestmark = pytest.mark.gpu


def _rng(seed, offset):
    import torch

    wrap = lambda v: v - 2 ** 64 if v >= 2 ** 63 else v
    return torch.tensor([wrap(seed), wrap(offset)], dtype=torch.int64, device="cuda")


SIZES = [(0, 1, 1), (0, 1, 7), (0, 3, 5), (0, 4, 4), (0, 64, 100), (0, 1021, 9), (1, 1, 5), (1, 7, 33), (2, 1, 1), (2, 8, 64),
         (2, 5, 13), (3, 32, 70), (3, 3, 11), (4, 33, 9), (5, 6, 5), (6, 2, 9), (6, 9, 7)]


@pytest.mark.parametrize("lmax,C,N", SIZES)
@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout(lmax, C, N, x, residual):
    eq = _eq()
    K = (lmax + 1) ** 2
    for p, seed, offset in ((0.1, 1, 2), (0.5, 2 ** 64 - 5, 2 ** 63 + 9), (0.999999, 2 ** 33, 2 ** 40 + 1), (0.0, 0, 0)):
        _say("dropout lmax=%d C=%d N=%d %s residual=%s p=%g" % (lmax, C, N, x, residual, p))
        r = np.random.default_rng(C)
        t, v = _put(r.standard_normal((N, C, K)), x)
        s, w = _put(r.standard_normal((N, C, K)), x) if residual else (None, None)
        got = _get(eq.eqtp_dropout(t, _rng(seed, offset) if p else None, p, lmax, residual=s))
        keep = ref.keep_mask(seed, offset, N, C, p)
        want = ref.dropout(v, keep, p, w)
        half = ref.U16 if x == "bf16" else ref.U32
        # one rounding of the fp32 sum, and in bf16 one more of the result
        bound = ref.U32 * np.abs(want) * 1.001 + (half * np.abs(want) * 1.001 if x == "bf16" else 0.0)
        assert (np.abs(got - want) <= bound + 1e-37).all()
        dropped = np.broadcast_to(~keep[:, :, None], got.shape)
        assert (got[dropped] == (w[dropped] if residual else 0.0)).all()


@pytest.mark.parametrize("shift", [1, 2, 3])
@pytest.mark.parametrize("lmax,C", [(0, 64), (0, 7), (3, 8), (2, 5)])
@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_dropout_unaligned_and_in_place(shift, lmax, C, x):
    eq = _eq()
    _say("dropout unaligned %d lmax=%d C=%d %s" % (shift, lmax, C, x))
    import torch

    r = np.random.default_rng(5)
    N, K = 21, (lmax + 1) ** 2
    a, b = r.standard_normal((N, C, K)), r.standard_normal((N, C, K))
    want = eq.eqtp_dropout(_put(a, x)[0], _rng(4, 5), 0.3, lmax, residual=_put(b, x)[0])
    t, s = _put(a, x, shift)[0], _put(b, x, shift)[0]
    assert torch.equal(eq.eqtp_dropout(t, _rng(4, 5), 0.3, lmax, residual=s), want)
    assert torch.equal(eq.eqtp_dropout(t, _rng(4, 5), 0.3, lmax, residual=s, out=t.clone()), want)
    into = s.clone()
    assert eq.eqtp_dropout(t, _rng(4, 5), 0.3, lmax, residual=into, out=into) is into and torch.equal(into, want)
    plain = eq.eqtp_dropout(t, _rng(4, 5), 0.3, lmax)
    eq.eqtp_dropout(t, _rng(4, 5), 0.3, lmax, out=t)
    assert torch.equal(t, plain)


@pytest.mark.parametrize("p", [0.05, 0.1, 0.3, 0.5])
@pytest.mark.parametrize("lmax,C,N", [(0, 64, 300), (0, 7, 999), (1, 10, 200), (3, 32, 41), (6, 5, 37)])
def test_dropout_bf16_sums_fall_as_those_of_the_separate_operations(lmax, C, N, p):
    """In bf16 a kept sum has the bits of the fp32 product, the fp32 sum and one rounding: where 1 / (1 - p) is a
    short fraction many sums are exact ties, which the last bit of fp32 decides.  The fused call writes the same.
    Sums that cancel to less than 1/64 of the residual are within half a step of the formula instead."""
    eq = _eq()
    _say("bf16 dropout sums lmax=%d C=%d N=%d p=%g" % (lmax, C, N, p))
    import torch

    r = np.random.default_rng(17)
    x, s = (_put(r.standard_normal((N, C, (lmax + 1) ** 2)), "bf16")[0] for _ in range(2))
    keep = torch.from_numpy(ref.keep_mask(8, 9, N, C, p)).cuda()[:, :, None]
    kept = x.float() * (1.0 / (1.0 - p))
    want = torch.where(keep, kept + s.float(), s.float()).to(torch.bfloat16)
    got = eq.eqtp_dropout(x, _rng(8, 9), p, lmax, residual=s)
    apart = ~keep | ((kept + s.float()).abs() >= s.float().abs() / 64)
    assert apart.float().mean() > 0.9 and torch.equal(got[apart], want[apart])
    true = x.double() * float(np.float32(1.0 / (1.0 - p))) + s.double()  # the factor as the library holds it
    assert ((got.double() - true).abs() <= 1.001 * (ref.U16 + ref.U32) * true.abs())[~apart].all()
    assert torch.equal(eq.eqtp_dropout_add_norm(x, s, _rng(8, 9), p, lmax)[1], got)
    assert torch.equal(eq.eqtp_dropout(x, _rng(8, 9), p, lmax), torch.where(keep, kept, 0.0).to(torch.bfloat16))


def test_dropout_drops_what_is_not_finite():
    """A dropped channel contributes nothing, NaN and infinities included; kept ones pass them on."""
    eq = _eq()
    _say("dropout of non-finite values")
    N, C = 40, 16
    x = np.random.default_rng(2).standard_normal((N, C, 4)).astype(np.float32)
    x[::2] = np.nan
    x[1::4] = np.inf
    got = _get(eq.eqtp_dropout(_put(x)[0], _rng(11, 12), 0.5, 1))
    keep = ref.keep_mask(11, 12, N, C, 0.5)
    assert (got[~keep] == 0).all()
    assert np.isnan(got[::2][keep[::2]]).all() and np.isposinf(got[1::4][keep[1::4]]).all()


def test_dropout_is_its_own_backward_and_offsets_differ():
    eq = _eq()
    _say("dropout offsets")
    import torch

    one = torch.ones((64, 64), device="cuda")
    a, b, c = (eq.eqtp_dropout(one, _rng(3, o), 0.5) for o in (1, 1, 2))
    assert torch.equal(a, b) and not torch.equal(a, c)
    agree = (a == c).float().mean().item()
    assert abs(agree - 0.5) < 5 * 0.5 / 64  # five standard deviations of 4096 coin throws
    x = torch.randn((64, 64), device="cuda")
    assert torch.equal(eq.eqtp_dropout(x, _rng(3, 1), 0.5), x * a)


def test_dropout_no_nodes_and_large():
    """No rows; and more than 2^32 elements, whose last channels follow the counter."""
    eq = _eq()
    _say("dropout past 2^32 elements")
    import torch

    assert eq.eqtp_dropout(torch.empty((0, 4, 4), device="cuda"), _rng(1, 1), 0.5, 1).shape == (0, 4, 4)
    N, C = 90001, 1000  # K = 49: 4.4e9 elements
    x = torch.ones((N, C, 49), dtype=torch.bfloat16, device="cuda")
    got = eq.eqtp_dropout(x, _rng(21, 22), 0.5, 6)
    del x
    for n in (0, 43826, 43827, 87652, N - 1):
        words = []
        first = n * C
        for blk in range(first // 4, (first + C + 3) // 4):
            words += ref.philox((blk & 0xFFFFFFFF, blk >> 32, 22, 0), (21, 0))
        keep = np.array(words[first % 4:first % 4 + C]) >= 2 ** 31
        assert (_get(got[n]) == np.where(keep[:, None], 2.0, 0.0)).all(), n
