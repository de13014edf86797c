"""Ways to call the transformer-block operators on the GPU: optional
arguments, other streams, types and wrappers give what the plain calls give."""
import numpy as np
import pytest

import block_reference as ref
from test_gpu_attention import Case, _i32
from test_gpu_norm import RNG, _get, _inputs, _within
from test_gpu_parity import _eq, _say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_attention_backward_with_the_output(x):
    """The forward call's output before lse, as a training step that keeps both passes it: the same bits, and within
    the bounds of the statement."""
    eq = _eq()
    _say("attention backward with the output, %s" % x)
    import torch

    c = Case(9, 7, [3, 0, 5, 1, 4, 2, 6, 0, 40], 8, 1, 4, 2, x, seed=31)
    out, lse = c.forward(eq)
    head = (c.q[0], c.k[0], c.v[0], _i32(c.src), _i32(c.row_ptr))
    tail = (lse, c.g[0], *(_i32(t) for t in c.plan), c.lmax, c.heads)
    grads = eq.eqtp_attention_backward(*head, out, *tail, bias=c.bias[0])
    for a, b, d in zip(grads, c.backward(eq, lse), eq.eqtp_attention_backward(*head, *tail, bias=c.bias[0], out=out)):
        assert torch.equal(a, b) and torch.equal(a, d)
    args = (c.q[1], c.k[1], c.v[1], c.src, c.row_ptr, c.heads, c.scale)
    bounds = ref.attention_bounds(*args, c.g[1], c.bias[1], ref.U16 if x == "bf16" else ref.U32)
    for name, t, w, b in zip(("gq", "gk", "gv", "gbias"), grads, ref.attention_backward(*args, c.g[1], c.bias[1]), bounds[2:]):
        _within(_get(t), w, b, name)


def test_attention_scale():
    """An explicit scale, as a number and in a tensor that changes between the passes, which keep the forward
    call's value."""
    eq = _eq()
    _say("attention with a scale of its own")
    import torch

    from spherical_harmonic_cg_amd import autograd as ag

    c = Case(8, 9, [3, 0, 5, 1, 4, 2, 6, 9], 4, 1, 4, 2, seed=32)
    for scale in (0.9, -0.4):
        args = (c.q[1], c.k[1], c.v[1], c.src, c.row_ptr, c.heads, float(np.float32(scale)))
        bounds = ref.attention_bounds(*args, c.g[1], c.bias[1], ref.U32)
        out, lse = c.forward(eq, scale=scale)
        _within(_get(out), ref.attention(*args, c.bias[1])[0], bounds[0], "out")
        wants = ref.attention_backward(*args, c.g[1], c.bias[1])
        grads = c.backward(eq, lse, scale=scale)
        for t, w, b in zip(grads, wants, bounds[2:]):
            _within(_get(t), w, b, "gradient")
        held = torch.tensor(scale)
        leaves = [t[0].clone().requires_grad_() for t in (c.q, c.k, c.v, c.bias)]
        y = ag.graph_attention(*leaves[:3], _i32(c.src), _i32(c.row_ptr), 1, 4, scale=held, bias=leaves[3])
        held.fill_(5.0)
        y.backward(c.g[0])
        assert torch.equal(y, out)
        for t, g in zip(leaves, grads):
            assert torch.equal(t.grad, g)
