"""The distance bias, the norm of queries and keys, routing and the experts'
linears as they are used together with the attention, and ways to call them:
autograd, captured graphs, other streams, the caller's workspace."""
import math

import numpy as np
import pytest

import mix_reference as ref
from test_gpu_norm import _get, _put
from test_gpu_parity import _eq, _say

pytestmark = pytest.mark.gpu


def _graph(N, E, seed):
    import torch

    r = np.random.default_rng(seed)
    dst = np.sort(r.integers(0, N - 2, E))  # two rows without edges
    src = r.integers(0, N, E)
    row_ptr = np.searchsorted(dst, np.arange(N + 1))
    i = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
    return dst, src, i(src), i(row_ptr)


class Block:
    """h -> attention(qk norm and rotation, distance bias) + h -> experts, with every parameter a leaf."""

    def __init__(self, N=600, E=6000, C=16, lmax=2, heads=2, X=5, top_k=2, seed=0):
        import torch

        r = np.random.default_rng(seed)
        K, w = (lmax + 1) ** 2, C // heads
        self.N, self.E, self.C, self.lmax, self.heads, self.X, self.top_k, self.K = N, E, C, lmax, heads, X, top_k, K
        self.dst, self.src, self.tsrc, self.row_ptr = _graph(N, E, seed)
        f = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32)).cuda()
        self.vec = f(E, 3) * 2.0
        self.bounds = torch.linspace(0.5, 4.0, 9).cuda()
        self.freq = f(3, w // 2 - 1)
        self.leaf = dict(h=f(N, C, K), table=0.5 * f(10, heads), wq=1 + 0.2 * f(lmax + 1, w), wk=1 + 0.2 * f(lmax + 1, w),
                         pos=f(N, 3), gate=f(C, X), W=f(X, lmax + 1, C, C) / math.sqrt(C))
        self.grad = f(N, C, K)

    def forward(self, leaf, idx_out=None):
        import spherical_harmonic_cg_amd as eq
        from spherical_harmonic_cg_amd import autograd as ag

        bias = ag.distance_bias(self.vec, self.bounds, leaf["table"], r_cut=4.5)
        q, k = ag.qk_norm(leaf["h"], leaf["h"], self.lmax, self.heads, leaf["wq"], leaf["wk"], leaf["pos"], None, self.freq)
        y = leaf["h"] + ag.graph_attention(q, k, leaf["h"], self.tsrc, self.row_ptr, self.lmax, self.heads, bias=bias)
        logits = y[:, :, 0] @ leaf["gate"]
        idx, weight = ag.route(logits, self.top_k, score=eq.EQTP_SCORE_SIGMOID)
        if idx_out is not None:
            idx_out.append(idx)
        return ag.expert_linear(y, leaf["W"], idx, self.lmax, weight=weight, plan=eq.eqtp_expert_plan(idx, self.X))

    def reference(self, idx):
        """The same in 64 bits on the CPU by elementary operations and torch's own differentiation (idx held)."""
        import torch

        L = {n: t.detach().double().cpu().requires_grad_() for n, t in self.leaf.items()}
        deg = torch.tensor(ref.degrees(self.lmax))
        N, C, K, H, w = self.N, self.C, self.K, self.heads, self.C // self.heads
        vec, freq = self.vec.double().cpu(), self.freq.double().cpu()
        bucket, live, _ = ref.buckets(vec.numpy(), self.bounds.cpu().numpy(), 4.5)
        bias = L["table"][torch.from_numpy(bucket)]

        def turned(weight):
            x = L["h"].reshape(N, H, w, K)
            r = torch.stack([(x[..., l * l:(l + 1) ** 2] ** 2).mean((2, 3)) + 1e-5 for l in range(self.lmax + 1)], 2) ** -0.5
            y = x * r[..., deg][:, :, None, :] * weight.t()[:, deg]
            th = L["pos"] @ freq
            R, half = freq.shape[1], w // 2
            c, s = torch.cos(th)[:, None, :, None], torch.sin(th)[:, None, :, None]
            a, b = y[:, :, :R], y[:, :, half:half + R]
            return torch.cat((a * c - b * s, y[:, :, R:half], a * s + b * c, y[:, :, half + R:]), 2).reshape(N, H, w * K)

        q, k, v = turned(L["wq"]), turned(L["wk"]), L["h"].reshape(N, H, w * K)
        at = torch.from_numpy(np.nonzero(live)[0])
        dst, src = torch.from_numpy(self.dst)[at], torch.from_numpy(self.src)[at]
        s = (q[dst] * k[src]).sum(2) / math.sqrt(w * K) + bias[at]
        e = torch.exp(s - s.detach().max())
        z = torch.zeros(N, H, dtype=torch.float64).index_add(0, dst, e)
        o = torch.zeros(N, H, w * K, dtype=torch.float64).index_add(0, dst, (e / z[dst])[:, :, None] * v[src])
        y = L["h"] + o.reshape(N, C, K)
        sc = torch.sigmoid(y[:, :, 0] @ L["gate"])
        taken = sc.gather(1, idx.cpu().long())
        weight = taken / taken.sum(1, keepdim=True)
        out = 0
        for j in range(self.top_k):
            M = L["W"][idx.cpu().long()[:, j]][:, deg]  # [N, K, C', C]
            out = out + weight[:, j, None, None] * torch.einsum("nkdc,nck->ndk", M, y)
        out.backward(self.grad.double().cpu())
        return out.detach(), {n: t.grad for n, t in L.items()}


def test_block_together():
    """Forward and gradients of all of them in a row against 64 bits: each tensor within 2000 u of its largest value
    (some twenty operators' roundings of about ten u each, amplified by the softmax's logits of up to ten)."""
    _eq()
    _say("block of bias, qk norm, attention, routing and experts")
    import torch

    b = Block()
    leaf = {n: t.clone().requires_grad_() for n, t in b.leaf.items()}
    chosen = []
    out = b.forward(leaf, chosen)
    out.backward(b.grad)
    want, grads = b.reference(chosen[0])
    for name, got, w in [("out", out, want)] + [(n, leaf[n].grad, grads[n]) for n in leaf]:
        far = float((got.detach().double().cpu() - w).abs().max())
        assert far <= 2000 * ref.u * float(w.abs().max()), (name, far, float(w.abs().max()))


def test_block_captured():
    """Captured once and replayed with other inputs, with eager work between the replays: each replay is the eager
    result, bit by bit."""
    eq = _eq()
    _say("block captured into a graph")
    import torch

    b = Block(N=700, seed=3)
    st = {n: t.clone() for n, t in b.leaf.items()}
    g = b.grad.clone()

    def step():
        bias = eq.eqtp_distance_bias(b.vec, b.bounds, st["table"], r_cut=4.5)
        how = dict(weight_q=st["wq"], weight_k=st["wk"], pos_q=st["pos"], pos_k=st["pos"], freq=b.freq)
        q, k = eq.eqtp_qk_norm(st["h"], st["h"], b.lmax, b.heads, **how)
        y = eq.eqtp_attention(q, k, st["h"], b.tsrc, b.row_ptr, b.lmax, b.heads, bias=bias)
        logits = y[:, :, 0] @ st["gate"]
        idx, weight = eq.eqtp_route(logits, 2)
        plan = eq.eqtp_expert_plan(idx, b.X)
        out = eq.eqtp_expert_linear(y, st["W"], idx, b.lmax, weight=weight, plan=plan)
        gy, gW, gw = eq.eqtp_expert_linear_backward(y, st["W"], idx, g, b.lmax, weight=weight, plan=plan)
        gl = eq.eqtp_route_backward(logits, idx, gw)
        gq = eq.eqtp_qk_norm_backward(st["h"], st["h"], gy, gy, b.lmax, b.heads, need_pos=True, **how)
        gt = eq.eqtp_distance_bias_backward(b.vec, b.bounds, bias.masked_fill(bias == -math.inf, 7.0), r_cut=4.5)
        return (out, idx, weight, gy, gW, gw, gl, gt) + gq + plan

    eager = [t.clone() for t in step()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for turn in range(3):
        for n in st:
            st[n].copy_(b.leaf[n] * (1.0 + 0.3 * turn))
        g.copy_(b.grad * (1.0 - 0.2 * turn))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        want = step()
        for i, (x, y) in enumerate(zip(got, want)):
            assert torch.equal(x, y), (turn, i)
        if turn == 0:
            assert all(torch.equal(x, y) for x, y in zip(got, eager))


def test_other_stream_and_workspaces():
    """On a stream of the caller's, with workspaces of exactly the size asked for: the same bits, nothing written behind
    them."""
    eq = _eq()
    _say("bias, qk norm and experts on another stream")
    import torch

    b = Block(N=530, seed=5)
    st = b.leaf
    idx, weight = eq.eqtp_route(b.leaf["h"][:, :, 0] @ st["gate"], 2)

    def calls(space):
        bias = eq.eqtp_distance_bias(b.vec, b.bounds, st["table"])
        gt = eq.eqtp_distance_bias_backward(b.vec, b.bounds, bias, workspace=space(
            eq.eqtp_distance_bias_workspace_bytes(b.E, b.heads, 10)))
        gq = eq.eqtp_qk_norm_backward(st["h"], st["h"], b.grad, b.grad, b.lmax, b.heads, workspace=space(
            eq.eqtp_qk_norm_workspace_bytes(b.N, b.N, b.lmax, b.C, b.heads)))
        plan = eq.eqtp_expert_plan(idx, b.X, workspace=space(eq.eqtp_expert_plan_workspace_bytes(b.N, 2, b.X)))
        ge = eq.eqtp_expert_linear_backward(st["h"], st["W"], idx, b.grad, b.lmax, weight=weight, plan=plan, workspace=space(
            eq.eqtp_expert_linear_backward_workspace_bytes(b.N, b.lmax, b.C, b.X, 2)))
        return (bias, gt) + gq[:4] + plan + ge

    want = calls(lambda n: None)
    torch.cuda.synchronize()
    spaces = []

    def space(n):
        spaces.append((torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda"), n))
        return spaces[-1][0][:n]

    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        got = calls(space)
    other.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    assert len(spaces) == 4 and all((t[n:] == 0xA5).all() for t, n in spaces)


@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_autograd_gives_the_calls_gradients(x):
    """The wrappers return what the entry points do, in the leaves' types; gradients that are not dense, outputs that
    nothing uses, a position that both sides share."""
    eq = _eq()
    _say("autograd of qk norm, routing and experts, %s" % x)
    import torch

    from spherical_harmonic_cg_amd import autograd as ag

    r = np.random.default_rng(7)
    q, k = (_put(r.standard_normal((9, 8, 4)), x)[0].requires_grad_() for _ in range(2))
    pos, freq = _put(r.standard_normal((9, 2)))[0].requires_grad_(), _put(r.standard_normal((2, 2)))[0]
    a, c = ag.qk_norm(q, k, 1, 2, pos_q=pos, freq=freq)
    g = torch.randn(4, 9, 8, device="cuda").to(q.dtype).permute(1, 2, 0)  # not dense
    torch.autograd.backward((a, c), (g, 2 * g))
    want = eq.eqtp_qk_norm_backward(q.detach(), k.detach(), g.contiguous(), (2 * g).contiguous(), 1, 2, pos_q=pos.detach(),
                                    freq=freq, need_pos=True)
    assert torch.equal(q.grad, want[0]) and torch.equal(k.grad, want[1]) and torch.equal(pos.grad, want[4] + want[5])
    q.grad = k.grad = None
    ag.qk_norm(q, k, 1, 2)[1].backward(g)
    assert q.grad is None and k.grad is not None
    t = _put(r.standard_normal((9, 6)), x)[0].requires_grad_()
    idx, w = ag.route(t, 2, scale=2.0)
    assert not idx.requires_grad
    W = _put(r.standard_normal((6, 2, 8, 8)), x)[0].requires_grad_()
    h = q.detach().requires_grad_()
    out = ag.expert_linear(h, W, idx, 1, weight=w, out_dtype=eq.EQTP_F32)
    go = torch.randn_like(out)
    out.backward(go)
    gh, gW, gw = eq.eqtp_expert_linear_backward(h.detach(), W.detach(), idx, go.to(h.dtype), 1, weight=w.detach())
    assert torch.equal(h.grad, gh) and torch.equal(W.grad, gW.to(W.dtype)) and W.grad.dtype == W.dtype
    assert torch.equal(t.grad, eq.eqtp_route_backward(t.detach(), idx, gw, scale=2.0))
