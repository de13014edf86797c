"""The attention's weights to the last bits: rows of two edges whose logits
are exact, so that only the exponential and the quotient round."""
import numpy as np
import pytest

import block_reference as ref
from test_gpu_attention import _i32
from test_gpu_norm import _get
from test_gpu_parity import _eq, _say

pytestmark = pytest.mark.gpu


def _rows(heads):
    """A row for each logit a in steps from -60 to 0, against the logit 0: (logits, row_ptr, src)."""
    a = -np.arange(0, 60 * 64 + 1) / 64.0
    a = a[: len(a) // heads * heads].reshape(-1, heads)
    n = len(a)
    row_ptr = (2 * np.arange(n + 1)).astype(np.int32)
    return a, row_ptr, np.tile(np.array([0, 1], np.int32), n)


@pytest.mark.parametrize("heads", [1, 4])
def test_weights_of_far_logits(heads):
    """w = exp(a) / (1 + exp(a)) for q = 0 and biases a and 0.  The exponential is off by one step of the hardware's
    (2 u), the remainder of its argument (below 1/2 after the whole powers of two) by 2^-25 twice over, which ln 2
    makes less than u; the sum, the quotient and the product round once each: 6 u, and no term that grows with |a|.
    grad_v of the far source is w again, from exp(s - lse) over the row's sum of these, so that an error of lse itself
    cancels.  The difference rounds by less than 8 u: half a step of it at |a| < 16, and beyond that less than lse, which
    is below exp(a).  With 3 u for each exponential, and one for the sum, the quotient and the product: 17 u."""
    eq = _eq()
    _say("attention weights of far logits, %d heads" % heads)
    import torch

    a, row_ptr, src = _rows(heads)
    n = len(a)
    bias = np.zeros((2 * n, heads), dtype=np.float32)
    bias[0::2] = a
    q = torch.zeros((n, heads), device="cuda")
    k = torch.zeros((2, heads), device="cuda")
    v = torch.zeros((2, heads), device="cuda")
    v[0] = 1.0                                        # the far edge's value
    lse = torch.empty((n, heads), device="cuda")
    b = torch.from_numpy(bias).cuda()
    out = eq.eqtp_attention(q, k, v, _i32(src), _i32(row_ptr), 0, heads, bias=b, lse=lse)
    want = np.exp(a) / (1.0 + np.exp(a))
    off = np.abs(_get(out) - want) / want / ref.U32
    _say("largest error of a weight, half steps: %.2f" % off.max())
    assert (off <= 6.0).all(), (off.max(), a.ravel()[off.argmax()])
    # each row with a far source of its own: grad_v of it is the row's weight
    src2 = np.empty(2 * n, dtype=np.int32)
    src2[0::2], src2[1::2] = np.arange(n), n
    order = np.argsort(src2, kind="stable")
    ptr = np.searchsorted(src2[order], np.arange(n + 2))
    dst = np.repeat(np.arange(n), 2)[order]
    k2 = torch.zeros((n + 1, heads), device="cuda")
    gv = eq.eqtp_attention_backward(q, k2, k2, _i32(src2), _i32(row_ptr), lse, torch.ones_like(q), _i32(ptr), _i32(dst),
                                    _i32(order), 0, heads, bias=b)[2]
    off = np.abs(_get(gv)[:n] - want) / want / ref.U32
    _say("largest error of a gradient's weight, half steps: %.2f" % off.max())
    assert (off <= 17.0).all(), (off.max(), a.ravel()[off.argmax()])


@pytest.mark.parametrize("shift", [0.0, 20.0, -50.0])
def test_gradient_weights_of_long_rows(shift):
    """Rows of 4096 edges, whose lse lies some 8 above the logits: the gradient's weights are formed from s and lse
    without rounding their difference (half a step of it is 8 u and more).  Every edge has a source of its own and the
    output's gradient is 1, so grad_v is the row's weights; over that of an edge at the row's largest logit the row's
    sum cancels.  Each of the two is off by 3 u for the exponential and one for the quotient's product: 8 u."""
    eq = _eq()
    _say("attention gradient weights of long rows, shift %g" % shift)
    import torch

    n, rows, heads = 4096, 2, 2
    r = np.random.default_rng(6)
    bias = (-5.0 * r.random((rows, n, heads))).astype(np.float32) + np.float32(shift)
    bias[:, 17] = shift
    E = n * rows
    row_ptr = (n * np.arange(rows + 1)).astype(np.int32)
    every = np.arange(E, dtype=np.int32)
    q, k = torch.zeros((rows, heads), device="cuda"), torch.zeros((E, heads), device="cuda")
    lse = torch.empty((rows, heads), device="cuda")
    b = torch.from_numpy(bias.reshape(E, heads)).cuda()
    eq.eqtp_attention(q, k, k, _i32(every), _i32(row_ptr), 0, heads, bias=b, lse=lse)
    gv = eq.eqtp_attention_backward(q, k, k, _i32(every), _i32(row_ptr), lse, torch.ones_like(q), _i32(np.arange(E + 1)),
                                    _i32(np.repeat(np.arange(rows), n)), _i32(every), 0, heads, bias=b)[2]
    w = _get(gv).reshape(rows, n, heads)
    want = np.exp(bias.astype(np.float64) - shift)
    off = np.abs(w / w[:, 17:18] - want) / want / ref.U32
    _say("largest error of a weight's ratio, half steps: %.2f" % off.max())
    assert (off <= 8.0).all(), off.max()
