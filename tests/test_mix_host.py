"""Refusals of the distance bias, the norm of queries and keys, routing and the
experts' linears: every call here is rejected or answered before any HIP call,
so no GPU is needed."""
import ctypes

import pytest

from test_abi_host import FAKE, NULL, _lib

ODD2, ODD1, OFF4, OFF8 = (ctypes.c_void_p(0x10000 + n) for n in (2, 1, 4, 8))
BIG = 1 << 40


def _desc(cls, **kw):
    return ctypes.byref(cls(struct_size=kw.pop("struct_size", ctypes.sizeof(cls)), **kw))


def _bias(e, **kw):
    return _desc(e._BiasDesc, **dict(dict(heads=4, buckets=8, r_cut=4.0), **kw))


def _qk(e, **kw):
    return _desc(e._QkNormDesc, **dict(dict(lmax=2, C=16, heads=4, kv_heads=2, x_dtype=0, axes=3, pairs=2, eps=1e-5), **kw))


def _route(e, **kw):
    return _desc(e._RouteDesc, **dict(dict(experts=8, top_k=2, groups=2, top_groups=1, score=0, renormalise=1, x_dtype=0,
                                           scale=1.0), **kw))


def _expert(e, **kw):
    return _desc(e._ExpertDesc, **dict(dict(lmax=2, C=16, experts=8, top_k=2, x_dtype=0, out_dtype=0), **kw))


def _each(f, n, holes, want=1):
    """f with one of n pointers after the other replaced."""
    for k, p in holes:
        args = [FAKE] * n
        args[k] = p
        assert f(*args) == want, (k, p)


@pytest.mark.parametrize("kw,want", [(dict(heads=0), 1), (dict(heads=1025), 2), (dict(buckets=0), 1), (dict(buckets=513), 2),
                                     (dict(r_cut=-1.0), 1), (dict(r_cut=float("nan")), 1), (dict(struct_size=12), 1)])
def test_bias_descriptor(kw, want):
    e = _lib()
    lib = e.load_library()
    d = _bias(e, **kw)
    assert lib.eqtp_distance_bias(d, 4, *[FAKE] * 4, NULL) == want
    assert lib.eqtp_distance_bias_workspace_bytes(d, 4) == -want
    assert lib.eqtp_distance_bias_backward(d, 4, *[FAKE] * 5, BIG, NULL) == want


def test_bias_pointers():
    e = _lib()
    lib = e.load_library()
    d = _bias(e)
    f = lambda *a: lib.eqtp_distance_bias(d, 4, *a, NULL)
    _each(f, 4, [(k, p) for k in range(4) for p in (NULL, ODD2)])
    assert lib.eqtp_distance_bias(d, 0, *[NULL] * 4, NULL) == 0 and lib.eqtp_distance_bias(d, -1, *[FAKE] * 4, NULL) == 1
    assert lib.eqtp_distance_bias(d, 1 << 31, *[FAKE] * 4, NULL) == 1
    need = lib.eqtp_distance_bias_workspace_bytes(d, 1000)
    g = lambda *a: lib.eqtp_distance_bias_backward(d, 1000, *a, need, NULL)
    _each(g, 5, [(k, p) for k in range(5) for p in (NULL, ODD2)] + [(4, OFF8)])
    assert lib.eqtp_distance_bias_backward(d, 1000, *[FAKE] * 5, need - 1, NULL) == 1


@pytest.mark.parametrize("kw,want", [
    (dict(lmax=-1), 1), (dict(lmax=7), 2), (dict(C=0), 1), (dict(C=18), 1), (dict(heads=0), 1), (dict(kv_heads=0), 1),
    (dict(x_dtype=2), 1), (dict(eps=0.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(axes=-1), 1),
    (dict(axes=4), 2), (dict(axes=0), 1), (dict(pairs=0), 1), (dict(pairs=3), 1), (dict(C=12, pairs=1), 1),
    (dict(C=4 * 229, axes=0, pairs=0), 2), (dict(lmax=0, C=4 * 2049, axes=0, pairs=0), 2), (dict(kv_heads=1025), 2),
    (dict(C=1025 * 4, heads=1025), 2), (dict(struct_size=32), 1)])
def test_qk_descriptor(kw, want):
    e = _lib()
    lib = e.load_library()
    d = _qk(e, **kw)
    assert lib.eqtp_qk_norm(d, 4, 4, *[FAKE] * 9, NULL) == want
    assert lib.eqtp_qk_norm_workspace_bytes(d, 4, 4) == -want
    assert lib.eqtp_qk_norm_backward(d, 4, 4, *[FAKE] * 16, BIG, NULL) == want


def test_qk_pointers():
    e = _lib()
    lib = e.load_library()
    d, b, n = _qk(e), _qk(e, x_dtype=1), _qk(e, axes=0, pairs=0)
    # q k weight_q weight_k pos_q pos_k freq out_q out_k
    f = lambda *a: lib.eqtp_qk_norm(d, 5, 4, *a, NULL)
    _each(f, 9, [(k, NULL) for k in (0, 1, 4, 5, 6, 7, 8)] + [(k, ODD2) for k in range(9)])
    assert lib.eqtp_qk_norm(b, 5, 4, ODD1, *[FAKE] * 8, NULL) == 1
    for N, M in ((-1, 4), (4, -1), (1 << 31, 4), (4, 1 << 31)):
        assert lib.eqtp_qk_norm(d, N, M, *[FAKE] * 9, NULL) == 1
    assert lib.eqtp_qk_norm(d, 0, 0, *[NULL] * 9, NULL) == 0
    need = lib.eqtp_qk_norm_workspace_bytes(d, 5, 4)
    # q k wq wk pq pk freq goq gok gq gk gwq gwk gpq gpk workspace
    g = lambda *a: lib.eqtp_qk_norm_backward(d, 5, 4, *a, need, NULL)
    _each(g, 16, [(k, NULL) for k in (0, 1, 4, 5, 6, 7, 8, 15)] + [(k, ODD2) for k in range(16)] + [(15, OFF8)])
    assert lib.eqtp_qk_norm_backward(d, 5, 4, *[FAKE] * 16, need - 1, NULL) == 1
    assert lib.eqtp_qk_norm_backward(n, 5, 4, *[FAKE] * 16, BIG, NULL) == 1  # gradients of positions without any


@pytest.mark.parametrize("kw,want", [
    (dict(experts=0), 1), (dict(experts=258), 2), (dict(top_k=0), 1), (dict(top_k=9), 1), (dict(experts=64, top_k=17), 2),
    (dict(groups=0), 1), (dict(groups=3), 1), (dict(top_groups=0), 1), (dict(top_groups=3), 1), (dict(score=2), 1),
    (dict(renormalise=2), 1), (dict(x_dtype=2), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(struct_size=40), 1)])
def test_route_descriptor(kw, want):
    e = _lib()
    lib = e.load_library()
    d = _route(e, **kw)
    assert lib.eqtp_route(d, 4, *[FAKE] * 4, NULL) == want
    assert lib.eqtp_route_backward(d, 4, *[FAKE] * 4, NULL) == want


def test_route_pointers():
    e = _lib()
    lib = e.load_library()
    d, b = _route(e), _route(e, x_dtype=1)
    f = lambda *a: lib.eqtp_route(d, 4, *a, NULL)  # logits bias idx weight
    _each(f, 4, [(k, NULL) for k in (0, 2, 3)] + [(k, ODD2) for k in range(4)])
    g = lambda *a: lib.eqtp_route_backward(d, 4, *a, NULL)  # logits idx grad_weight grad_logits
    _each(g, 4, [(k, p) for k in range(4) for p in (NULL, ODD2)])
    assert lib.eqtp_route(b, 4, ODD1, FAKE, FAKE, FAKE, NULL) == 1
    for N, want in ((-1, 1), (1 << 31, 1), (0, 0)):
        assert lib.eqtp_route(d, N, *[FAKE] * 4, NULL) == want and lib.eqtp_route_backward(d, N, *[FAKE] * 4, NULL) == want


def test_expert_plan_refusals():
    e = _lib()
    lib = e.load_library()
    need = lib.eqtp_expert_plan_workspace_bytes(100, 2, 8)
    f = lambda N, k, X, *a, size=BIG: lib.eqtp_expert_plan(N, k, X, *a, size, NULL)
    for N, k, X, want in ((-1, 2, 8, 1), (1 << 31, 1, 8, 1), (1 << 30, 2, 8, 1), (4, 0, 8, 1), (4, 2, 0, 1), (4, 2, 257, 2),
                          (4, 17, 8, 2)):
        assert f(N, k, X, *[FAKE] * 5) == want and lib.eqtp_expert_plan_workspace_bytes(N, k, X) == -want
    g = lambda *a: f(100, 2, 8, *a, size=need)  # idx order slots ptr workspace
    _each(g, 5, [(k, NULL) for k in (0, 2, 3, 4)] + [(k, ODD2) for k in range(5)] + [(4, OFF8)])
    assert f(100, 2, 8, *[FAKE] * 5, size=need - 1) == 1


@pytest.mark.parametrize("kw,want", [(dict(lmax=-1), 1), (dict(lmax=7), 2), (dict(C=0), 1), (dict(C=24), 2), (dict(C=256), 2),
                                     (dict(experts=0), 1), (dict(experts=257), 2), (dict(top_k=0), 1), (dict(top_k=17), 2),
                                     (dict(x_dtype=2), 1), (dict(out_dtype=2), 1), (dict(struct_size=24), 1)])
def test_expert_descriptor(kw, want):
    e = _lib()
    lib = e.load_library()
    d = _expert(e, **kw)
    assert lib.eqtp_expert_linear(d, 4, *[FAKE] * 6, NULL) == want
    assert lib.eqtp_expert_linear_backward_workspace_bytes(d, 4) == -want
    assert lib.eqtp_expert_linear_backward(d, 4, *[FAKE] * 12, BIG, NULL) == want


def test_expert_pointers():
    e = _lib()
    lib = e.load_library()
    d = _expert(e)
    f = lambda *a: lib.eqtp_expert_linear(d, 4, *a, NULL)  # h W idx weight order out
    _each(f, 6, [(k, NULL) for k in (0, 1, 2, 5)] + [(k, ODD2) for k in range(6)] + [(k, OFF8) for k in (0, 1, 5)])
    for N, want in ((-1, 1), (1 << 31, 1), (1 << 30, 1), (0, 0)):
        assert lib.eqtp_expert_linear(d, N, *[FAKE] * 6, NULL) == want
    need = lib.eqtp_expert_linear_backward_workspace_bytes(d, 100)
    # h W idx weight order slots ptr grad_out grad_h grad_W grad_weight workspace
    g = lambda *a: lib.eqtp_expert_linear_backward(d, 100, *a, need, NULL)
    _each(g, 12, [(k, NULL) for k in (0, 1, 2, 5, 6, 7, 11)] + [(k, ODD2) for k in range(12)]
          + [(k, OFF8) for k in (0, 1, 7, 8, 9, 11)])
    assert lib.eqtp_expert_linear_backward(d, 100, *[FAKE] * 12, need - 1, NULL) == 1
    none = [FAKE] * 8 + [NULL] * 3 + [FAKE]
    assert lib.eqtp_expert_linear_backward(d, 100, *none, need, NULL) == 1  # nothing asked for


def test_binding_refusals():
    """The binding names what is wrong with a tensor before the library is called."""
    import torch

    e = _lib()
    x, i = torch.zeros(4, 8, 4), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="on the GPU"):
        e.eqtp_distance_bias(torch.zeros(4, 3), torch.zeros(2), torch.zeros(3, 2))
    with pytest.raises(ValueError, match="on the GPU"):
        e.eqtp_qk_norm(x, x, 1, 2)
    with pytest.raises(ValueError, match="on the GPU"):
        e.eqtp_route(torch.zeros(4, 8), 2)
    with pytest.raises(ValueError, match="on the GPU"):
        e.eqtp_expert_plan(i, 8)
    with pytest.raises(ValueError, match="on the GPU"):
        e.eqtp_expert_linear(x, torch.zeros(2, 2, 8, 8), i, 1)


def test_r_cut_that_float32_has_not():
    """A cut-off too short for float32 is refused: as 0 it would mask no edge where it has to mask all."""
    e = _lib()
    for r in (1e-50, -1e-50):
        with pytest.raises(ValueError, match="float32"):
            e._bias_desc(4, 8, r)
    for r in (0.0, 1e-45, 5.0, 1e300):
        e._bias_desc(4, 8, r)
