"""Attention over a graph on the GPU, forward and backward, against its 64-bit
statement.  Tolerances are elementwise bounds derived from the roundings on
the way (block_reference.attention_bounds)."""
import numpy as np
import pytest

import block_reference as ref
from test_gpu_norm import _dt, _get, _put, _within
from test_gpu_parity import _eq, _say

pytestmark = pytest.mark.gpu


def _graph(N, M, lengths, r):
    row_ptr = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    return row_ptr, r.integers(0, M, row_ptr[-1]).astype(np.int32)


def _by_source(row_ptr, src, M):
    dst = np.repeat(np.arange(len(row_ptr) - 1), np.diff(row_ptr)).astype(np.int32)
    perm = np.argsort(src, kind="stable").astype(np.int32)
    src_ptr = np.concatenate([[0], np.cumsum(np.bincount(src, minlength=M))]).astype(np.int32)
    return src_ptr, dst[perm], perm


def _i32(a):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class Case:
    def __init__(self, N, M, lengths, width, lmax, heads, kv_heads, x="f32", bias=True, masked=0.1, seed=0, shift=0,
                 size=1.0):
        r = np.random.default_rng(seed)
        K = (lmax + 1) ** 2
        self.N, self.M, self.lmax, self.heads, self.x = N, M, lmax, heads, x
        self.row_ptr, self.src = _graph(N, M, lengths, r)
        self.E = len(self.src)
        put = lambda n, c: _put(size * r.standard_normal((n, c, K)), x, shift)
        self.q, self.g = put(N, heads * width), _put(r.standard_normal((N, heads * width, K)), x, shift)
        self.k, self.v = put(M, kv_heads * width), _put(r.standard_normal((M, kv_heads * width, K)) + 0.5, x, shift)
        self.bias = None
        if bias:
            b = r.standard_normal((self.E, heads)).astype(np.float32)
            b[r.random((self.E, heads)) < masked] = -np.inf
            self.bias = _put(b)
        self.scale = 1.0 / np.sqrt(width * K)
        self.plan = _by_source(self.row_ptr, self.src, M)

    def forward(self, eq, **kw):
        import torch

        lse = torch.full((self.N, self.heads), float("nan"), device="cuda")
        out = eq.eqtp_attention(self.q[0], self.k[0], self.v[0], _i32(self.src), _i32(self.row_ptr), self.lmax,
                                self.heads, bias=self.bias and self.bias[0], lse=lse, **kw)
        return out, lse

    def backward(self, eq, lse, **kw):
        return eq.eqtp_attention_backward(self.q[0], self.k[0], self.v[0], _i32(self.src), _i32(self.row_ptr), lse,
                                          self.g[0], *(_i32(t) for t in self.plan), self.lmax, self.heads,
                                          bias=self.bias and self.bias[0], **kw)

    def check(self, eq, backward=True):
        args = (self.q[1], self.k[1], self.v[1], self.src, self.row_ptr, self.heads, self.scale)
        b = self.bias and self.bias[1]
        bounds = ref.attention_bounds(*args, self.g[1], b, ref.U16 if self.x == "bf16" else ref.U32)
        want, _, wlse, _ = ref.attention(*args, b)
        out, lse = self.forward(eq)
        _within(_get(out), want, bounds[0], "out")
        got = _get(lse)
        live = np.isfinite(wlse)
        assert (np.isneginf(got) == ~live).all()
        if live.any():
            _within(got[live], wlse[live], bounds[1][live], "lse")
        if backward:
            grads = self.backward(eq, lse, need_bias=True)
            wants = ref.attention_backward(*args, self.g[1], b)
            for name, t, w, e in zip(("gq", "gk", "gv", "gbias"), grads, wants, bounds[2:]):
                _within(_get(t), w, e, name)


LENGTHS = [0, 1, 2, 3, 7, 0, 15, 16, 17, 31, 33, 63, 64, 65, 5, 130]

SHAPES = [  # (width, lmax, heads, kv_heads)
    (1, 0, 1, 1), (3, 0, 2, 1), (4, 0, 2, 2), (16, 0, 8, 8), (16, 0, 4, 1), (64, 0, 2, 2), (100, 0, 3, 3), (8, 1, 2, 2),
    (1, 1, 4, 2), (4, 2, 2, 2), (5, 2, 3, 1), (1, 2, 8, 8), (8, 3, 4, 4), (16, 3, 4, 2), (32, 3, 2, 2), (1, 3, 3, 3),
    (3, 4, 2, 1), (8, 4, 1, 1), (7, 5, 2, 2), (4, 6, 2, 2), (1, 6, 1, 1), (128, 3, 1, 1), (41, 6, 1, 1), (2048, 0, 1, 1),
    (2, 0, 40, 10), (16, 1, 16, 16)]


@pytest.mark.parametrize("width,lmax,heads,kv_heads", SHAPES)
@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_attention(width, lmax, heads, kv_heads, x):
    eq = _eq()
    _say("attention width=%d lmax=%d heads=%d/%d %s" % (width, lmax, heads, kv_heads, x))
    big = width * (lmax + 1) ** 2 * heads > 1000
    lengths = LENGTHS[:8] + [33, 66] if big else LENGTHS
    Case(len(lengths), 23, lengths, width, lmax, heads, kv_heads, x, seed=width + heads).check(eq)


@pytest.mark.parametrize("N,M,lengths", [(1, 1, [1]), (1, 5, [0]), (3, 1, [2, 0, 4]), (1, 700, [700]), (2, 900, [3, 1500]),
                                         (5, 3, [300, 0, 1, 257, 256]), (40, 2, [9] * 40)])
@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("bias", [False, True])
def test_attention_row_lengths(N, M, lengths, x, bias):
    """One edge, none, rows and sources with many."""
    eq = _eq()
    _say("attention N=%d M=%d %s %s bias=%s" % (N, M, lengths[:5], x, bias))
    Case(N, M, lengths, 8, 1, 2, 1, x, bias=bias, seed=M).check(eq)


@pytest.mark.parametrize("N,E", [(1, 5000), (3, 20011), (7, 9001)])
@pytest.mark.parametrize("heads,kv_heads,width,lmax", [(4, 4, 16, 0), (4, 2, 5, 1)])
def test_attention_few_long_rows(N, E, heads, kv_heads, width, lmax):
    """Readout: each item in one row; rows cut anywhere, one of them empty."""
    eq = _eq()
    _say("attention readout N=%d E=%d" % (N, E))
    r = np.random.default_rng(E)
    cuts = np.sort(r.integers(0, E, N - 1))
    lengths = np.diff(np.concatenate([[0], cuts, [E]]))
    c = Case(N, E, lengths, width, lmax, heads, kv_heads, bias=True, seed=1)
    c.src = np.arange(E, dtype=np.int32)
    c.plan = _by_source(c.row_ptr, c.src, E)
    c.check(eq)


def test_attention_few_long_sources():
    eq = _eq()
    _say("attention with few sources")
    Case(3000, 2, [3] * 3000, 8, 1, 2, 2, seed=4).check(eq)


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [1, 2, 3])
@pytest.mark.parametrize("width,lmax,heads", [(16, 0, 4), (4, 3, 2), (3, 2, 2)])
def test_attention_unaligned(x, shift, width, lmax, heads):
    """Tensors that begin one to three elements into their storage give the bits of aligned ones."""
    eq = _eq()
    _say("attention unaligned width=%d lmax=%d %s %d" % (width, lmax, x, shift))
    import torch

    got = []
    for s in (0, shift):
        c = Case(9, 11, LENGTHS[:9], width, lmax, heads, heads, x, seed=3, shift=s)
        out, lse = c.forward(eq)
        got.append((out, lse) + c.backward(eq, lse))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_attention_masks():
    """Rows whose every edge is masked are zero with lse -inf and zero gradients; the type's lowest value is an
    ordinary bias (equal lowest biases weigh edges equally); masked edges take no part whatever k, v, q and g hold."""
    eq = _eq()
    _say("attention masks")
    import torch

    c = Case(6, 8, [4, 3, 0, 5, 4, 2], 8, 1, 2, 2, masked=0.0, seed=9)
    c.src = np.array([0, 1, 2, 3, 1, 2, 3, 4, 5, 6, 5, 4, 6, 5, 4, 7, 7, 0], dtype=np.int32)
    c.plan = _by_source(c.row_ptr, c.src, 8)
    b = c.bias[1].astype(np.float32).copy()
    b[4:7] = -np.inf                       # row 1: nothing left
    b[0, 0] = -np.inf                      # one head of one edge
    b[12:16] = np.finfo(np.float32).min    # row 4: all at the lowest value
    b[c.src == 7] = -np.inf                # source 7 masked everywhere...
    b[12:16][c.src[12:16] != 7] = np.finfo(np.float32).min
    c.bias = _put(b)
    c.check(eq)
    clean = c.forward(eq)
    grads = c.backward(eq, clean[1])
    out = _get(clean[0])
    assert (out[1] == 0).all() and (out[2] == 0).all()
    for t in (c.k, c.v):
        t[0][7] = float("nan")             # ... so what it holds does not matter
    c.v[0][7, 0] = float("inf")
    got = c.forward(eq)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
    again = c.backward(eq, got[1])
    for a, d in zip(again, grads):
        assert torch.equal(a, d)
    c.q[0][1] = float("nan")               # a row with every edge masked
    c.g[0][1] = float("inf")
    for a, d in zip(c.backward(eq, got[1])[1:], grads[1:]):
        assert torch.equal(a, d)
    assert torch.equal(c.forward(eq)[0], clean[0])


@pytest.mark.parametrize("bias", [float(np.finfo(np.float32).min), -1e30, 3e6])
@pytest.mark.parametrize("N,E", [(4, 24), (2, 3000)])
def test_attention_common_bias_cancels(bias, N, E):
    """A bias that all edges of a row share, the type's lowest value among them, changes neither the weights nor any
    gradient; logits that it rounds away leave equal weights."""
    eq = _eq()
    _say("attention common bias %g N=%d" % (bias, N))
    c = Case(N, 9, [E // N] * N, 8, 1, 2, 1, bias=True, masked=0.0, seed=18)
    c.q = _put(np.zeros(c.q[1].shape))     # equal logits, whatever the bias
    c.bias = _put(np.full((E, 2), bias))
    args = (c.q[1], c.k[1], c.v[1], c.src, c.row_ptr, 2, c.scale)
    want = ref.attention(*args)[0]
    bounds = ref.attention_bounds(*args, c.g[1], None, ref.U32)
    out, lse = c.forward(eq)
    _within(_get(out), want, bounds[0], "out")
    grads = c.backward(eq, lse)
    for name, t, w, e in zip(("gq", "gk", "gv", "gbias"), grads, ref.attention_backward(*args, c.g[1]), bounds[2:]):
        _within(_get(t), w, e, name)


def test_attention_not_finite():
    """A NaN in one source reaches the rows that read it and no others."""
    eq = _eq()
    _say("attention of non-finite values")
    c = Case(12, 9, [5] * 12, 4, 1, 2, 2, masked=0.0, seed=10)
    c.k[0][3, 0, 0] = float("nan")         # channel 0: head 0
    out = _get(c.forward(eq)[0])
    for n in range(12):
        hit = 3 in c.src[c.row_ptr[n]:c.row_ptr[n + 1]]
        assert np.isnan(out[n, :4]).all() == hit and np.isfinite(out[n, 4:]).all()
        assert hit or np.isfinite(out[n]).all()


@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_attention_large_logits(x):
    """Logits of several hundred: the running maximum keeps exp in range; one edge wins each row."""
    eq = _eq()
    _say("attention large logits %s" % x)
    Case(10, 30, LENGTHS[5:15], 16, 1, 2, 2, x, seed=11, size=20.0).check(eq)


def test_attention_gradient_against_differences():
    eq = _eq()
    _say("attention differences")
    c = Case(7, 9, [3, 0, 1, 8, 2, 5, 4], 6, 2, 4, 2, seed=12)
    _, lse = c.forward(eq)
    grads = c.backward(eq, lse)
    args = [c.q[1], c.k[1], c.v[1], c.bias[1]]
    bounds = ref.attention_bounds(*args[:3], c.src, c.row_ptr, 4, c.scale, c.g[1], args[3], ref.U32)[2:]
    r = np.random.default_rng(3)
    f = lambda a: (ref.attention(a[0], a[1], a[2], c.src, c.row_ptr, 4, c.scale, a[3])[0] * c.g[1]).sum()
    for i in range(4):
        d = r.standard_normal(args[i].shape)
        d[~np.isfinite(args[i])] = 0.0
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + 1e-4 * d, args[i] - 1e-4 * d
        slope, mine = (f(up) - f(down)) / 2e-4, (_get(grads[i]) * d).sum()
        allow = (bounds[i] * np.abs(d)).sum() + 1e-6 * (np.abs(_get(grads[i]) * d).sum() + 1.0)
        assert abs(mine - slope) <= allow, (i, mine, slope)


def test_attention_partial_requests_and_determinism():
    eq = _eq()
    _say("attention partial requests")
    import torch

    c = Case(30, 17, list(range(30)), 8, 2, 4, 2, seed=13)
    out, lse = c.forward(eq)
    again = c.forward(eq)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    full = c.backward(eq, lse)
    for need in ((True, False, False, False), (False, True, False, False), (False, False, True, True),
                 (False, False, False, True), (True, True, True, False)):
        part = c.backward(eq, lse, need_q=need[0], need_k=need[1], need_v=need[2], need_bias=need[3])
        for a, b, n in zip(part, full, need):
            assert (a is None) != n and (not n or torch.equal(a, b))


def test_attention_empty():
    eq = _eq()
    _say("attention without edges or rows")
    import torch

    q = torch.randn((4, 6, 4), device="cuda")
    rp = torch.zeros(5, dtype=torch.int32, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    lse = torch.empty((4, 2), device="cuda")
    out = eq.eqtp_attention(q, q[:0], q[:0], none, rp, 1, 2, lse=lse)
    assert (out == 0).all() and torch.isneginf(lse).all()
    k = torch.randn((3, 6, 4), device="cuda")
    gq, gk, gv, gb = eq.eqtp_attention_backward(q, k, k, none, rp, lse, q, rp[:4], none, none, 1, 2, need_bias=True)
    assert (gq == 0).all() and (gk == 0).all() and (gv == 0).all() and gb.shape == (0, 2)
    assert eq.eqtp_attention(q[:0], k, k, none, rp[:1], 1, 2).shape == (0, 6, 4)


def test_attention_bad_indexes_stay_inside():
    """Sources and row pointers out of range are clamped: results are unspecified, no access leaves the buffers."""
    eq = _eq()
    _say("attention clamps")
    import torch

    c = Case(5, 6, [3, 4, 2, 5, 1], 8, 0, 2, 2, seed=14)
    c.src = c.src.copy()
    c.src[::3] = [99, -7, 1 << 30, -(1 << 31), 6]
    c.row_ptr = np.array([0, 3, 2, 900, -4, 15], dtype=np.int32)
    _, lse = c.forward(eq)
    c.plan = (np.array([0, -1, 1 << 29, 4, 2, 15, 15], dtype=np.int32), c.plan[1] - 3, c.plan[2] * 7 - 9)
    c.backward(eq, lse)
    torch.cuda.synchronize()


def test_attention_debug_mode_names_bad_graphs():
    eq = _eq()
    _say("attention debug mode")
    c = Case(5, 6, [3, 4, 2, 5, 1], 8, 0, 2, 2, seed=15)
    was = eq.eqtp_set_debug(True)
    try:
        out, lse = c.forward(eq)
        c.backward(eq, lse)
        good = c.src.copy()
        c.src = good.copy()
        c.src[4] = 6                       # M = 6 > N = 5: checked against M
        with pytest.raises(eq.EqtpError) as err:
            c.forward(eq)
        assert err.value.status == eq.EQTP_EGRAPH
        c.src = good
        c.src[4] = 5
        c.forward(eq)
        for k, bad in ((0, 99), (1, 5), (2, -1)):
            plan = [t.copy() for t in c.plan]
            plan[k][2] = bad
            keep, c.plan = c.plan, tuple(plan)
            with pytest.raises(eq.EqtpError) as err:
                c.backward(eq, lse)
            assert err.value.status == eq.EQTP_EGRAPH
            c.plan = keep
    finally:
        eq.eqtp_set_debug(was)


def test_attention_large_offsets():
    """Rows, sources and edges whose byte and element offsets pass 2^32; sampled rows against the statement."""
    eq = _eq()
    _say("attention past 2^32 elements")
    import torch

    N, M, C, heads, E = 600, 2200000, 2048, 4, 3000
    k = torch.empty((M, C), dtype=torch.bfloat16, device="cuda")  # 4.5e9 elements
    for at in range(0, M, 100000):
        k[at:at + 100000].normal_()
    r = np.random.default_rng(5)
    src = r.integers(0, M, E).astype(np.int32)
    src[:10] = M - 1 - np.arange(10)
    row_ptr = (np.arange(N + 1) * 5).astype(np.int32)
    q = torch.randn((N, C), device="cuda").to(torch.bfloat16)
    got = eq.eqtp_attention(q, k, k, _i32(src), _i32(row_ptr), 0, heads)
    rows = 8
    kk = k[torch.from_numpy(src[:5 * rows].astype(np.int64)).cuda()].double().cpu().numpy()[:, :, None]
    args = (q[:rows].double().cpu().numpy()[:, :, None], kk, kk, np.arange(5 * rows), row_ptr[:rows + 1], heads, 512 ** -0.5)
    want = ref.attention(*args)[0]
    bound = ref.attention_bounds(*args, args[0], None, ref.U16)[0]
    _within(_get(got[:rows])[:, :, None], want, bound, "sampled rows")


def test_attention_edge_tables_past_2_31():
    """E heads past 2^31: bias, weights and logits' gradients are indexed in 64 bits."""
    eq = _eq()
    _say("attention with E heads past 2^31")
    import torch

    N, E, heads = 50000, 40000000, 64
    rp = (torch.arange(N + 1, device="cuda") * (E // N)).to(torch.int32)
    src = torch.randint(0, N, (E,), dtype=torch.int32, device="cuda")
    q, k, v = (torch.randn((N, heads), device="cuda") for _ in range(3))
    bias = torch.empty((E, heads), device="cuda")
    for at in range(0, E, 4000000):
        bias[at:at + 4000000].normal_()
    got = eq.eqtp_attention(q, k, v, src, rp, 0, heads, bias=bias)
    n0 = N - 2
    e0 = int(rp[n0])
    args = (q[n0:].double().cpu().numpy()[:, :, None], k.double().cpu().numpy()[:, :, None],
            v.double().cpu().numpy()[:, :, None], src[e0:].cpu().numpy(), (rp[n0:] - e0).cpu().numpy(), heads, 1.0)
    b = bias[e0:].double().cpu().numpy()
    want = ref.attention(*args, b)[0]
    bound = ref.attention_bounds(*args, args[0], b, ref.U32)[0]
    _within(_get(got[n0:])[:, :, None], want, bound, "last rows")


def test_attention_graph_capture():
    """Captured once: every replay has the eager bits, with eager work on the same buffers between."""
    eq = _eq()
    _say("attention graph capture")
    import torch

    cases = [Case(40, 40, [9] * 40, 8, 3, 4, 4, seed=16), Case(2, 4000, [1500, 2500], 16, 0, 4, 4, seed=17)]
    for c in cases:
        src, rp = _i32(c.src), _i32(c.row_ptr)
        plan = [_i32(t) for t in c.plan]
        lse = torch.empty((c.N, c.heads), device="cuda")
        out = torch.empty_like(c.q[0])

        def step():
            eq.eqtp_attention(c.q[0], c.k[0], c.v[0], src, rp, c.lmax, c.heads, bias=c.bias[0], lse=lse, out=out)
            return eq.eqtp_attention_backward(c.q[0], c.k[0], c.v[0], src, rp, lse, c.g[0], *plan, c.lmax, c.heads,
                                              bias=c.bias[0])

        want = [t.clone() for t in step()] + [out.clone(), lse.clone()]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            grads = step()
        for _ in range(4):
            out.fill_(float("nan"))
            for t in grads:
                t.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(list(grads) + [out, lse], want):
                assert torch.equal(a, b)
            step()
            torch.cuda.synchronize()


@pytest.mark.parametrize("x,heads,kv_heads,width,lmax,N,M,each", [
    ("f32", 4, 4, 16, 3, 350, 1500, 21),    # each XCD has one head's slice of k and v, four edges side by side
    ("f32", 4, 2, 16, 3, 350, 3000, 19),    # two heads to each key and value head
    ("bf16", 8, 8, 16, 3, 300, 1400, 17),   # eight slices
    ("f32", 4, 4, 16, 3, 900, 1500, 4),     # rows of few edges side by side
    ("f32", 2, 2, 33, 3, 300, 1300, 18)])   # rows that are not whole units
@pytest.mark.parametrize("bias", [False, True])
def test_attention_dealt_heads(x, heads, kv_heads, width, lmax, N, M, each, bias):
    """Keys, values, queries and gradients of more than an L2: heads are dealt to the XCDs and the tables of weights
    lie head by head."""
    eq = _eq()
    _say("attention dealt heads %s %d/%d width=%d each=%d bias=%s" % (x, heads, kv_heads, width, each, bias))
    r = np.random.default_rng(each)
    lengths = r.integers(0, 2 * each + 1, N)
    Case(N, M, lengths, width, lmax, heads, kv_heads, x, bias=bias, seed=each).check(eq)


@pytest.mark.parametrize("heads,kv_heads,width,lmax,x", [(4, 4, 1, 0, "f32"), (1, 1, 1, 2, "f32"), (2, 1, 5, 0, "bf16"), (3, 3, 4, 0, "f32")])
def test_attention_many_short_rows(heads, kv_heads, width, lmax, x):
    """Enough rows of some twenty edges that each wave takes several side by side, sources among them with one edge."""
    eq = _eq()
    _say("attention many rows heads=%d/%d width=%d %s" % (heads, kv_heads, width, x))
    r = np.random.default_rng(7)
    N = 9000
    lengths = np.zeros(N, dtype=np.int64)
    lengths[r.integers(0, N, 700)] = r.integers(1, 60, 700)
    lengths[:64] = 20
    lengths[N - 1] = 33
    c = Case(N, 12000, lengths, width, lmax, heads, kv_heads, x, seed=8)
    c.check(eq)
