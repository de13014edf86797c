"""The distance bias on the GPU against its 64-bit statement: the forward pass
picks table rows, so it is compared bit by bit; the gradient's bounds count its
additions (see mix_reference)."""
import numpy as np
import pytest

import mix_reference as ref
from test_gpu_norm import _get, _put, _within
from test_gpu_parity import _eq, _say

pytestmark = pytest.mark.gpu


def _edges(E, B, seed, r_cut):
    r = np.random.default_rng(seed)
    bounds = np.sort(r.uniform(0.2, 5.0, B - 1)).astype(np.float32)
    vec = (r.standard_normal((E, 3)) * 2.0).astype(np.float32)
    # lengths at the bounds themselves, a step to either side, zero, and at the cut-off
    special = list(bounds[:20]) + ([np.float32(r_cut)] if r_cut else []) + [np.float32(0.0)]
    for i, b in enumerate(special):
        for j, v in enumerate((b, np.nextafter(b, np.float32(9.0)), np.nextafter(b, np.float32(-1.0)))):
            if 3 * i + j < E:
                vec[3 * i + j] = 0.0
                vec[3 * i + j, (i + j) % 3] = v
    return vec, bounds


@pytest.mark.parametrize("E", [0, 1, 63, 64, 65, 257, 5003])
@pytest.mark.parametrize("H,B,r_cut", [(1, 1, 0.0), (4, 16, 4.0), (3, 2, 2.5), (8, 33, 0.0), (5, 64, 3.0), (16, 257, 4.0),
                                       (64, 7, 0.0), (65, 512, 4.0), (130, 130, 2.0)])
def test_distance_bias(E, H, B, r_cut):
    eq = _eq()
    _say("distance bias E=%d H=%d B=%d" % (E, H, B))
    import torch

    vec, bounds = _edges(E, B, 7 * E + H, r_cut)
    r = np.random.default_rng(E + 1)
    tv, tb = _put(vec)[0], _put(bounds)[0]
    table, g = _put(r.standard_normal((B, H))), _put(r.standard_normal((E, H)))
    out = eq.eqtp_distance_bias(tv, tb, table[0], r_cut=r_cut)
    np.testing.assert_array_equal(_get(out), ref.distance_bias(vec, bounds, table[1], r_cut))
    got = eq.eqtp_distance_bias_backward(tv, tb, g[0], r_cut=r_cut)
    want, bound = ref.distance_bias_backward(vec, bounds, g[1], B, r_cut)
    _within(_get(got), want, bound, "grad_table")
    assert torch.equal(got, eq.eqtp_distance_bias_backward(tv, tb, g[0], r_cut=r_cut))


def test_distance_bias_odd_values():
    """NaN and infinite components, bounds of zero and below, less aligned buffers, values in masked places."""
    eq = _eq()
    _say("distance bias, odd values")
    vec = np.array([[np.nan, 0, 0], [np.inf, 0, 0], [-np.inf, 1, 2], [0, 0, 0], [1, 0, 0], [3e38, 3e38, 0], [1e-30, 0, 0]],
                   dtype=np.float32)
    bounds = np.array([-1.0, 0.0, 1e-25, 1.0, 2.0], dtype=np.float32)
    tv, tb = _put(vec, shift=1)[0], _put(bounds, shift=3)[0]
    table = _put(np.arange(24).reshape(6, 4), shift=1)
    for r_cut in (0.0, 1e9, 1.0):
        out = _get(eq.eqtp_distance_bias(tv, tb, table[0], r_cut=r_cut))
        np.testing.assert_array_equal(out, ref.distance_bias(vec, bounds, table[1], r_cut))
    assert np.isnan(out[0]).all() and (out[4] == -np.inf).all() and out[6, 0] == 8.0
    g = np.ones((7, 4))
    g[[0, 1, 2, 4, 5]] = np.nan  # what masked places hold does not matter
    got = _get(eq.eqtp_distance_bias_backward(tv, tb, _put(g, shift=1)[0], r_cut=1.0))
    # the zero vector and the short one are above the bounds -1 and 0 and below 1e-25: bucket 2
    assert (got[2] == 2.0).all() and got.sum() == 8.0


def test_distance_bias_long_sums():
    """Half a million edges in one bucket: the additions of a lane are few, so the sum is close."""
    eq = _eq()
    _say("distance bias, long sums")
    r = np.random.default_rng(3)
    E, H = 500009, 4
    vec = np.tile(np.float32([1.0, 0.0, 0.0]), (E, 1))
    bounds = np.float32([0.5, 2.0])
    g = _put(1.0 + r.standard_normal((E, H)))
    got = _get(eq.eqtp_distance_bias_backward(_put(vec)[0], _put(bounds)[0], g[0]))
    # 1024 workgroups of 4 waves of 16 edges side by side: 8 additions a lane, and one rounding of a line and the result
    _within(got[1], g[1].sum(0), ref.u * 12 * np.abs(g[1]).sum(0), "grad_table")
    assert (got[[0, 2]] == 0).all()


@pytest.mark.parametrize("B,H,one", [(512, 1, False), (512, 3, False), (512, 8, False), (512, 65, False), (512, 8, True),
                                     (512, 65, True), (257, 1, True), (257, 3, False), (257, 65, False), (64, 8, False),
                                     (64, 65, False), (64, 3, True), (2, 1, False), (2, 8, True)])
def test_distance_bias_many_rounds(B, H, one):
    """Every wave goes over many stretches of edges, all with gradients: the sums are those of all edges, in many buckets
    or all in one, within bounds that count a lane's own additions."""
    eq = _eq()
    _say("distance bias, many rounds, B=%d H=%d one=%s" % (B, H, one))
    import torch

    # a lane's table has B + 1 places of 4 bytes in LDS, beside the bounds: 80 KB of them a workgroup, 160 KB a compute unit
    waves = min(4, max(1, (80 << 10) // ((B + 1) * 256 + 8 * B)))
    held = min(32 // waves, max(1, (160 << 10) // (waves * (B + 1) * 256 + 8 * B)))
    blocks = min(2048, torch.cuda.get_device_properties(0).multi_processor_count * held)
    rounds = 5
    E = 64 * waves * blocks * (rounds - 1) + 12345  # some waves have a last round, one of them in part
    r = np.random.default_rng(H + B)
    bounds = np.sort(r.uniform(0.2, 5.0, B - 1)).astype(np.float32)
    away = np.full(E, 0.01, np.float32) if one else r.uniform(0.0, 5.5, E).astype(np.float32)
    vec = np.zeros((E, 3), dtype=np.float32)
    vec[np.arange(E), r.integers(0, 3, E)] = away
    g = _put(1.0 + r.standard_normal((E, H)))
    got = _get(eq.eqtp_distance_bias_backward(_put(vec)[0], _put(bounds)[0], g[0], r_cut=5.25))
    bucket = np.where(away < 5.25, np.searchsorted(bounds, away, side="right"), B)
    rows = np.argsort(bucket, kind="stable")
    upto = np.searchsorted(bucket[rows], np.arange(B + 1))
    want, size = np.zeros((B, H)), np.zeros((B, H))
    for b in range(B):
        mine = g[1][rows[upto[b]:upto[b + 1]]]
        want[b], size[b] = mine.sum(0), np.abs(mine).sum(0)
    # a lane: one edge in 64 / heads places of each stretch; then a line's rounding, and the result's
    adds = rounds * -(-64 // (64 // min(H, 64)))
    _within(got, want, ref.u * (adds + 3) * size, "grad_table")
