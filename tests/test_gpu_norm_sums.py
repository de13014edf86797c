"""The layer norm's sums over nodes (gradients of weight and bias), where one
node's terms are 2^28 times the others': fp32 additions one after the other
would lose the small ones."""
import numpy as np
import pytest

import block_reference as ref
from test_gpu_norm import _get, _put
from test_gpu_parity import _eq, _say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lmax,C,N", [(3, 32, 1000), (0, 64, 2000), (1, 8, 1500), (4, 33, 250), (6, 10, 250), (0, 4096, 200)])
@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_weight_and_bias_sums_keep_small_terms(lmax, C, N, x):
    """Every value of x is 1 or -1, so zhat is r times that, exactly, and every term of the sums is exact in fp32.  N is
    small enough that no thread adds two nodes: the sum over a workgroup's nodes and a degree's components, held in 64
    bits, is rounded once, and the sum over workgroups once more.  Both roundings are of sums of terms of one sign, half
    a step each; 2^-30 covers their product and the 64-bit additions."""
    eq = _eq()
    _say("norm sums lmax=%d C=%d N=%d %s" % (lmax, C, N, x))
    import torch

    K = (lmax + 1) ** 2
    sign = np.ones((N, C, K))
    # scalars of mean 0: half of them -1 (an odd last one is 0)
    sign[:, :, 0] = np.where(np.arange(C) % 2 == 0, 1.0, -1.0)[None, :]
    if C % 2:
        sign[:, C - 1, 0] = 0.0
    big = np.ones((N, 1, 1))
    big[0] = 2.0 ** 28
    xs, _ = _put(sign, x)
    g, _ = _put(sign * big, x)
    stats = torch.empty((N, lmax + 2), device="cuda")
    eq.eqtp_layer_norm(xs, lmax, stats=stats)
    st = _get(stats)
    assert (st[:, 0] == 0).all()
    gw, gb = eq.eqtp_layer_norm_backward(xs, stats, g, lmax)[2:]
    total = 2.0 ** 28 + (N - 1)
    allow = 2 * ref.U32 * (1 + 2.0 ** -6)
    assert (st[:, 1:] == st[0, 1:]).all()
    for l in range(lmax + 1):
        want = total * (2 * l + 1) * st[0, 1 + l] * (sign[0, :, 0] != 0 if l == 0 else np.ones(C))
        off = np.abs(_get(gw)[l] - want)
        assert (off <= allow * want).all(), (l, (off / np.maximum(want, 1.0)).max())
    want = total * sign[0, :, 0]
    off = np.abs(_get(gb) - want)
    assert (off <= allow * np.abs(want)).all(), (off / total).max()
