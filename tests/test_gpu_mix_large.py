"""Tensors of more than 2^31 elements: what stands behind that offset is what a
call on the last rows alone gives, bit for bit.  Sums over all rows are of small
whole numbers in the last ones and zeros before, which fp32 holds exactly."""
import pytest

from test_gpu_parity import _eq, _say

pytestmark = pytest.mark.gpu

TAIL = 1000  # (more than the sizes at which a call takes another form)


def test_distance_bias_far():
    import torch

    eq = _eq()
    E, H, B = 2 ** 28 + TAIL, 8, 5
    _say("distance bias E=%d H=%d" % (E, H))
    torch.manual_seed(0)
    vec = torch.rand(E, 3, device="cuda")
    bounds = torch.tensor([0.2, 0.5, 0.9, 1.3], device="cuda")
    table = torch.randn(B, H, device="cuda")
    out = eq.eqtp_distance_bias(vec, bounds, table, r_cut=1.5)
    assert torch.equal(out[-TAIL:], eq.eqtp_distance_bias(vec[-TAIL:].contiguous(), bounds, table, r_cut=1.5))
    g = out.zero_()
    g[-TAIL:] = torch.randint(-4, 5, (TAIL, H), device="cuda").float()
    assert torch.equal(eq.eqtp_distance_bias_backward(vec, bounds, g, r_cut=1.5),
                       eq.eqtp_distance_bias_backward(vec[-TAIL:].contiguous(), bounds, g[-TAIL:].contiguous(), r_cut=1.5))


def test_qk_norm_far():
    import torch

    eq = _eq()
    lmax, heads, C, K = 1, 2, 32, 4
    N = 2 ** 31 // (C * K) + TAIL
    _say("norm of queries and keys N=%d C=%d K=%d" % (N, C, K))
    torch.manual_seed(1)
    q = torch.randn(N, C, K, device="cuda", dtype=torch.bfloat16)
    k = torch.randn(TAIL, C, K, device="cuda", dtype=torch.bfloat16)
    pos_q, pos_k = torch.randn(N, 2, device="cuda"), torch.randn(TAIL, 2, device="cuda")
    freq = torch.randn(2, 5, device="cuda")
    w = torch.rand(lmax + 1, C // heads, device="cuda")
    last = lambda t: t[-TAIL:].contiguous()  # noqa: E731
    out, _ = eq.eqtp_qk_norm(q, k, lmax, heads, w, w, pos_q, pos_k, freq)
    want, _ = eq.eqtp_qk_norm(last(q), k, lmax, heads, w, w, last(pos_q), pos_k, freq)
    assert torch.equal(last(out), want)
    how = dict(need_weight_q=False, need_weight_k=False, need_pos=True)
    got = eq.eqtp_qk_norm_backward(q, k, out, None, lmax, heads, w, w, pos_q, pos_k, freq, **how)
    want = eq.eqtp_qk_norm_backward(last(q), k, last(out), None, lmax, heads, w, w, last(pos_q), pos_k, freq, **how)
    assert torch.equal(last(got[0]), want[0]) and torch.equal(last(got[4]), want[4])


def test_route_far():
    import torch

    eq = _eq()
    X = 256
    N = 2 ** 31 // X + TAIL
    _say("routing N=%d X=%d" % (N, X))
    torch.manual_seed(2)
    logits = torch.randn(N, X, device="cuda", dtype=torch.bfloat16)
    tail = logits[-TAIL:].contiguous()
    idx, weight = eq.eqtp_route(logits, 4, groups=8, top_groups=3)
    for got, want in zip((idx, weight), eq.eqtp_route(tail, 4, groups=8, top_groups=3)):
        assert torch.equal(got[-TAIL:], want)
    got = eq.eqtp_route_backward(logits, idx, weight)
    assert torch.equal(got[-TAIL:], eq.eqtp_route_backward(tail, idx[-TAIL:].contiguous(), weight[-TAIL:].contiguous()))


@pytest.mark.parametrize("x,k", [("f32", 1), ("f32", 2), ("bf16", 2)])
def test_experts_far(x, k):
    import torch

    eq = _eq()
    C, lmax, K, X = 64, 3, 16, 3
    N = 2 ** 31 // (C * K) + TAIL
    dt = torch.bfloat16 if x == "bf16" else torch.float32
    _say("experts N=%d C=%d K=%d %s k=%d" % (N, C, K, x, k))
    torch.manual_seed(3)
    h = torch.zeros(N, C, K, device="cuda", dtype=dt)
    h[-TAIL:] = torch.randint(-3, 4, (TAIL, C, K), device="cuda").to(dt)
    W = torch.randint(-2, 3, (X, lmax + 1, C, C), device="cuda").to(dt)
    idx = torch.randint(-1, X, (N, k), device="cuda", dtype=torch.int32)
    weight = torch.randint(1, 4, (N, k), device="cuda").float() if k > 1 else None
    last = lambda t: None if t is None else t[-TAIL:].contiguous()  # noqa: E731
    plan = eq.eqtp_expert_plan(idx, X)
    out = eq.eqtp_expert_linear(h, W, idx, lmax, weight=weight, plan=plan)
    assert torch.equal(last(out), eq.eqtp_expert_linear(last(h), W, last(idx), lmax, weight=last(weight)))
    got = eq.eqtp_expert_linear_backward(h, W, idx, h, lmax, weight=weight, plan=plan)
    want = eq.eqtp_expert_linear_backward(last(h), W, last(idx), last(h), lmax, weight=last(weight))
    assert torch.equal(last(got[0]), want[0])
    assert torch.equal(got[1], want[1])
    if k > 1:
        assert torch.equal(last(got[2]), want[2])


@pytest.mark.parametrize("x,k,gates", [("f32", 1, False), ("f32", 1, True), ("bf16", 1, True)])
def test_experts_of_many_nodes(x, k, gates):
    """More than 2^30 nodes: more threads than a launch holds at one tile a workgroup."""
    import torch

    eq = _eq()
    C, X = 8, 3
    N = 2 ** 30 + TAIL
    dt = torch.bfloat16 if x == "bf16" else torch.float32
    _say("experts N=%d C=%d %s gates=%s" % (N, C, x, gates))
    torch.manual_seed(4)
    h = torch.zeros(N, C, device="cuda", dtype=dt)
    W = torch.randn(X, 1, C, C, device="cuda").to(dt)
    idx = torch.zeros(N, k, device="cuda", dtype=torch.int32)
    weight = torch.ones(N, k, device="cuda") if gates else None
    far = [slice(0, TAIL), slice(N // 2, N // 2 + TAIL), slice(N - TAIL, N)]
    for at in far:
        h[at] = torch.randn(TAIL, C, device="cuda").to(dt)
        idx[at] = torch.randint(-1, X, (TAIL, k), device="cuda", dtype=torch.int32)
        if gates:
            weight[at] = torch.rand(TAIL, k, device="cuda")
    cut = lambda t, at: None if t is None else t[at].contiguous()  # noqa: E731
    back = torch.arange(N - 1, -1, -1, device="cuda", dtype=torch.int32)  # an order: the last node first
    for plan in (None, (back, back, torch.zeros(X + 1, device="cuda", dtype=torch.int32))):
        out = eq.eqtp_expert_linear(h, W, idx, 0, weight=weight, plan=plan)
        for at in far:
            assert torch.equal(out[at], eq.eqtp_expert_linear(cut(h, at), W, cut(idx, at), 0, weight=cut(weight, at)))
        gh, _, gw = eq.eqtp_expert_linear_backward(h, W, idx, out, 0, weight=weight, plan=plan, need_W=False)
        for at in far:
            a, _, b = eq.eqtp_expert_linear_backward(cut(h, at), W, cut(idx, at), cut(out, at), 0, weight=cut(weight, at), need_W=False)
            assert torch.equal(gh[at], a)
            assert not gates or torch.equal(gw[at], b)
        del out, gh, gw
