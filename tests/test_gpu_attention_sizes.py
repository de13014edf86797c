"""The attention's ways of dealing its work out, each at sizes that reach it:
source passes dealt to the XCDs, tables of weights past 2^31 elements, more
waves than one launch holds, rows and sources of very unequal length."""
import numpy as np
import pytest

import block_reference as ref
from test_gpu_attention import Case, _by_source, _i32
from test_gpu_norm import _get, _within
from test_gpu_parity import _eq, _say

pytestmark = pytest.mark.gpu


def _pieces(rows, E):
    """Pieces that a row is cut into, as the library's rule has it."""
    if rows >= 2048:
        return 1
    s = min((2048 + rows - 1) // rows, E // rows // 32, 1024)
    return 1 if s < 2 else s


def _dealt(rows, E, kv, row_bytes, gathered):
    """Whether a pass deals its heads to the XCDs: the library's rule, for powers of two of heads."""
    nb = min(kv, 8)
    while nb > 1 and kv // nb * row_bytes < 512:
        nb //= 2
    return _pieces(rows, E) == 1 and nb > 1 and gathered > 8 << 20 and gathered // nb <= 32 << 20


@pytest.mark.parametrize("x,heads,kv_heads,width,N,M,each,rows_too", [
    ("f32", 4, 4, 16, 1100, 1500, 4, True),     # sources of few edges, side by side in a wave
    ("f32", 4, 4, 16, 1100, 1200, 16, True),    # a source's edges side by side
    ("f32", 4, 4, 16, 1100, 300, 8, False),     # the rows' pass is not dealt: the tables lie edge by edge
    ("f32", 4, 2, 16, 1100, 2200, 6, True),     # two heads to each key and value head
    ("bf16", 8, 8, 16, 1100, 1200, 5, True),
    ("f32", 2, 2, 33, 1100, 1300, 7, True)])    # rows that are not whole units
def test_attention_dealt_sources(x, heads, kv_heads, width, N, M, each, rows_too):
    """Queries and output gradients of more than the 8 MiB from which on the source pass is dealt by heads."""
    eq = _eq()
    _say("attention dealt sources %s %d/%d width=%d N=%d M=%d" % (x, heads, kv_heads, width, N, M))
    r = np.random.default_rng(each)
    lengths = r.integers(0, 2 * each + 1, N)
    c = Case(N, M, lengths, width, 3, heads, kv_heads, x, seed=each)
    row = width * 16 * (2 if x == "bf16" else 4)
    assert _dealt(M, c.E, kv_heads, row, 2 * N * heads * row)
    assert _dealt(N, c.E, kv_heads, row, 2 * M * kv_heads * row) == rows_too
    c.check(eq)


@pytest.mark.parametrize("width,N,dealt", [(1, 2100, False), (16, 2100, True), (1, 60, False)])
def test_attention_gradients_past_2_31(width, N, dealt):
    """E heads past 2^31: the weights, the logits' gradients and the bias's are addressed in 64 bits by rows and by
    sources, edge by edge, head by head (dealt) and where few rows are cut into pieces.  Nearly all edges lie in the
    first rows; the last 50 rows, whose numbers lie past 2^31, read eight sources that no other row reads."""
    eq = _eq()
    _say("attention gradients past 2^31, width %d, %d rows" % (width, N))
    import torch

    from spherical_harmonic_cg_amd import autograd as ag

    heads, M, last, each = 64, 2500, 50, 10
    bulk = (2 ** 31 // heads + 6000) // (N - last) * (N - last) + (N - last)
    E = bulk + last * each
    assert bulk * heads > 2 ** 31
    assert _dealt(N, E, heads, 4 * width, 2 * M * heads * width * 4) == dealt
    g = torch.Generator(device="cuda")
    g.manual_seed(N + width)
    counts = torch.full((N,), bulk // (N - last), device="cuda")
    counts[-last:] = each
    rp = torch.zeros(N + 1, dtype=torch.int32, device="cuda")
    rp[1:] = torch.cumsum(counts, 0).to(torch.int32)
    assert int(rp[-1]) == E
    src = torch.randint(0, M - 8, (E,), dtype=torch.int32, device="cuda", generator=g)
    src[bulk:] = torch.randint(M - 8, M, (E - bulk,), dtype=torch.int32, device="cuda", generator=g)
    normal = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    q, grad = normal(N, heads * width), normal(N, heads * width)
    k, v = normal(M, heads * width), normal(M, heads * width)
    bias = torch.empty((E, heads), device="cuda")
    for at in range(0, E, 1 << 22):
        bias[at:at + (1 << 22)].normal_(generator=g)
    plan = ag.attention_plan(src, rp, M)
    lse = torch.empty((N, heads), device="cuda")
    out = eq.eqtp_attention(q, k, v, src, rp, 0, heads, bias=bias, lse=lse)
    gq, gk, gv, gb = eq.eqtp_attention_backward(q, k, v, src, rp, lse, grad, *plan, 0, heads, bias=bias)
    wide = lambda t: t.double().cpu().numpy()  # noqa: E731
    args = (wide(q[-last:])[:, :, None], wide(k[-8:])[:, :, None], wide(v[-8:])[:, :, None],
            src[bulk:].cpu().numpy() - (M - 8), (np.arange(last + 1) * each).astype(np.int32), heads, width ** -0.5)
    b, go = wide(bias[bulk:]), wide(grad[-last:])[:, :, None]
    bounds = ref.attention_bounds(*args, go, b, ref.U32)
    _within(_get(out[-last:])[:, :, None], ref.attention(*args, b)[0], bounds[0], "out")
    wants = ref.attention_backward(*args, go, b)
    for name, t, w, e in zip(("gq", "gk", "gv"), (gq[-last:], gk[-8:], gv[-8:]), wants, bounds[2:]):
        _within(_get(t)[:, :, None], w, e, name)
    _within(_get(gb[bulk:]), wants[3], bounds[5], "gbias")


@pytest.mark.parametrize("side", ["rows", "sources"])
def test_attention_more_waves_than_a_launch(side):
    """8.4 million rows (or sources) of 128 heads, two head blocks each, are more than the 2^24 waves of one launch:
    those on both sides of the border, the first and the last hold edges, and all others come out zero."""
    eq = _eq()
    _say("attention over several launches, %s" % side)
    import torch

    many, few, heads = 8400000, 100, 128
    at = np.array([0, 1, 5, 2 ** 23 - 2, 2 ** 23 - 1, 2 ** 23, 2 ** 23 + 1, many - 2, many - 1])  # in order
    assert many * 2 > 2 ** 24 and 2 ** 23 * 2 == 2 ** 24  # the border lies before row 2^23
    r = np.random.default_rng(3)
    N, M = (many, few) if side == "rows" else (few, many)
    if side == "rows":
        lengths = r.integers(1, 6, len(at))
        rows, small_ptr = at, np.concatenate([[0], np.cumsum(lengths)])
        src = r.integers(0, few, small_ptr[-1])
        row_ptr = np.searchsorted(np.repeat(at, lengths), np.arange(N + 1)).astype(np.int32)
        sources, small_src = np.arange(few), src
    else:
        rows, lengths = np.arange(few), r.integers(0, 4, few)
        row_ptr = small_ptr = np.concatenate([[0], np.cumsum(lengths)])
        small_src = r.integers(0, len(at), small_ptr[-1])
        src, sources = at[small_src], at
    E = int(small_ptr[-1])
    dst = np.repeat(rows, lengths)
    perm = np.argsort(src, kind="stable")
    src_ptr = np.searchsorted(src[perm], np.arange(M + 1))
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    normal = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    q, grad, k, v = normal(N, heads), normal(N, heads), normal(M, heads), normal(M, heads)
    bias = normal(E, heads)
    lse = torch.empty((N, heads), device="cuda")
    out = eq.eqtp_attention(q, k, v, _i32(src), _i32(row_ptr), 0, heads, bias=bias, lse=lse)
    gq, gk, gv, gb = eq.eqtp_attention_backward(q, k, v, _i32(src), _i32(row_ptr), lse, grad, _i32(src_ptr),
                                                _i32(dst[perm]), _i32(perm), 0, heads, bias=bias)
    pick = lambda t, i: t[torch.from_numpy(i).cuda()].double().cpu().numpy()[:, :, None]  # noqa: E731
    args = (pick(q, rows), pick(k, sources), pick(v, sources), small_src, small_ptr.astype(np.int32), heads, 1.0)
    b, go = bias.double().cpu().numpy(), pick(grad, rows)
    bounds = ref.attention_bounds(*args, go, b, ref.U32)
    _within(pick(out, rows), ref.attention(*args, b)[0], bounds[0], "out")
    wants = ref.attention_backward(*args, go, b)
    _within(pick(gq, rows), wants[0], bounds[2], "gq")
    for name, t, w, e in zip(("gk", "gv"), (gk, gv), wants[1:3], bounds[3:5]):
        _within(pick(t, sources), w, e, name)
    _within(_get(gb), wants[3], bounds[5], "gbias")
    rest = np.ones(many, dtype=bool)
    rest[at] = False
    rest = torch.from_numpy(rest).cuda()[:, None]
    for t in ((out, gq) if side == "rows" else (gk, gv)):
        assert not bool(((t != 0) & rest).any())
    if side == "rows":
        assert bool((torch.isneginf(lse) | ~rest).all())


@pytest.mark.parametrize("heads,kv_heads,width,x", [(4, 4, 1, "f32"), (4, 2, 16, "f32"), (2, 2, 5, "bf16")])
def test_attention_hubs(heads, kv_heads, width, x):
    """One row and one source with most of the edges among thousands with a few: a row's sum is one wave's there."""
    eq = _eq()
    _say("attention hubs heads=%d/%d width=%d %s" % (heads, kv_heads, width, x))
    r = np.random.default_rng(11)
    N, M = 2500, 2600
    lengths = r.integers(0, 4, N)
    lengths[1234] = 5000
    c = Case(N, M, lengths, width, 0, heads, kv_heads, x, seed=12)
    c.src = c.src.copy()
    c.src[r.permutation(c.E)[:3000]] = 77
    c.plan = _by_source(c.row_ptr, c.src, M)
    c.check(eq)
