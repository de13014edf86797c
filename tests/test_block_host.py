"""Refusals of the transformer-block entry points: every call here is rejected
or answered before any HIP call, so no GPU is needed."""
import ctypes

import pytest

from test_abi_host import FAKE, NULL, _lib

ODD2, ODD1, OFF4 = ctypes.c_void_p(0x10002), ctypes.c_void_p(0x10001), ctypes.c_void_p(0x10004)


def _norm_desc(e, **kw):
    d = dict(lmax=3, C=64, x_dtype=0, out_dtype=0, eps=1e-5, p=0.0)
    d.update(kw)
    return e._NormDesc(ctypes.sizeof(e._NormDesc), d["lmax"], d["C"], d["x_dtype"], d["out_dtype"], d["eps"], d["p"])


@pytest.mark.parametrize("kw,want", [
    (dict(lmax=-1), 1), (dict(lmax=7), 2), (dict(C=0), 1), (dict(C=-3), 1), (dict(C=1025), 2), (dict(lmax=0, C=16385), 2),
    (dict(lmax=6, C=335), 2), (dict(x_dtype=2), 1), (dict(out_dtype=-1), 1), (dict(eps=0.0), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(p=-0.1), 1), (dict(p=1.0), 1),
    (dict(p=float("nan")), 1)])
def test_norm_descriptor(kw, want):
    e = _lib()
    lib = e.load_library()
    d = ctypes.byref(_norm_desc(e, **kw))
    assert lib.eqtp_layer_norm(d, 4, FAKE, FAKE, FAKE, FAKE, FAKE, NULL) == want
    assert lib.eqtp_dropout_add_norm(d, 4, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, NULL) == want
    assert lib.eqtp_layer_norm_workspace_bytes(d, 4) == -want
    assert lib.eqtp_layer_norm_backward(d, 4, *[FAKE] * 11, 1 << 40, NULL) == want


def test_norm_descriptor_size():
    e = _lib()
    lib = e.load_library()
    d = _norm_desc(e)
    d.struct_size -= 4
    assert lib.eqtp_layer_norm(ctypes.byref(d), 4, FAKE, FAKE, FAKE, FAKE, FAKE, NULL) == 1
    assert lib.eqtp_layer_norm(None, 4, FAKE, FAKE, FAKE, FAKE, FAKE, NULL) == 1


def test_norm_pointers_and_sizes():
    e = _lib()
    lib = e.load_library()
    d, b, p = (ctypes.byref(_norm_desc(e, **kw)) for kw in ({}, dict(x_dtype=1, out_dtype=1), dict(p=0.5)))
    f = lambda desc, n, *a: lib.eqtp_layer_norm(desc, n, *a, NULL)
    assert f(d, -1, *[FAKE] * 5) == 1 and f(d, 1 << 31, *[FAKE] * 5) == 1
    assert f(d, 0, *[NULL] * 5) == 0  # nothing to do
    assert f(d, 4, NULL, FAKE, FAKE, FAKE, FAKE) == 1 and f(d, 4, FAKE, FAKE, FAKE, NULL, FAKE) == 1
    assert f(p, 4, *[FAKE] * 5) == 1  # dropout is not this call's
    for k in range(5):
        args = [FAKE] * 5
        args[k] = ODD2
        assert f(d, 4, *args) == 1
    args = [ODD1, FAKE, FAKE, FAKE, FAKE]
    assert f(b, 4, *args) == 1
    g = lambda desc, *a: lib.eqtp_dropout_add_norm(desc, 4, *a, NULL)
    for k in (0, 1, 5, 6):
        args = [FAKE] * 8
        args[k] = NULL
        assert g(d, *args) == 1
    assert g(p, FAKE, FAKE, NULL, *[FAKE] * 5) == 1       # p > 0 needs rng
    assert g(p, FAKE, FAKE, OFF4, *[FAKE] * 5) == 1       # rng on 8 bytes
    for k in (0, 1, 3, 4, 5, 6, 7):
        args = [FAKE] * 8
        args[k] = ODD2
        assert g(d, *args) == 1


def test_norm_backward_refusals():
    e = _lib()
    lib = e.load_library()
    d, p = ctypes.byref(_norm_desc(e)), ctypes.byref(_norm_desc(e, p=0.5))
    need = lib.eqtp_layer_norm_workspace_bytes(d, 100)
    assert need > 0
    # total stats weight grad_out grad_total rng grad_residual grad_x grad_weight grad_bias workspace
    f = lambda desc, n, a, size=need: lib.eqtp_layer_norm_backward(desc, n, *a, size, NULL)
    ok = [FAKE] * 11
    put = lambda k, v: ok[:k] + [v] + ok[k + 1:]
    assert f(d, 100, ok, need - 1) == 1 and f(d, -1, ok) == 1
    for k in (0, 1, 3, 10):
        assert f(d, 100, put(k, NULL)) == 1
    for k in (0, 1, 2, 3, 4, 6, 7, 8, 9):
        assert f(d, 100, put(k, ODD2)) == 1
    assert f(d, 100, put(10, ctypes.c_void_p(0x10008))) == 1
    assert f(p, 100, put(5, NULL)) == 1 and f(p, 100, put(5, OFF4)) == 1
    assert f(d, 100, ok[:6] + [NULL] * 4 + [FAKE]) == 1   # nothing asked for


def test_dropout_refusals():
    e = _lib()
    lib = e.load_library()
    f = lambda N, C, L, dt, p, x=FAKE, r=FAKE, g=FAKE, o=FAKE: lib.eqtp_dropout(N, C, L, dt, p, x, r, g, o, NULL)
    assert f(-1, 8, 1, 0, 0.5) == 1 and f(1 << 31, 8, 1, 0, 0.5) == 1 and f(4, 0, 1, 0, 0.5) == 1
    assert f(4, 8, -1, 0, 0.5) == 1 and f(4, 8, 7, 0, 0.5) == 2 and f(4, 8, 1, 2, 0.5) == 1
    assert f((1 << 31) - 1, (1 << 31) - 1, 6, 0, 0.5) == 1
    for p in (-0.01, 1.0, 2.0, float("nan")):
        assert f(4, 8, 1, 0, p) == 1
    assert f(0, 8, 1, 0, 0.5, NULL, NULL, NULL, NULL) == 0
    assert f(4, 8, 1, 0, 0.5, x=NULL) == 1 and f(4, 8, 1, 0, 0.5, o=NULL) == 1 and f(4, 8, 1, 0, 0.5, g=NULL) == 1
    assert f(4, 8, 1, 0, 0.5, g=OFF4) == 1
    for kw in (dict(x=ODD2), dict(r=ODD2), dict(o=ODD2)):
        assert f(4, 8, 1, 0, 0.5, **kw) == 1
    for kw in (dict(x=ODD1), dict(r=ODD1), dict(o=ODD1)):
        assert f(4, 8, 1, 1, 0.5, **kw) == 1


def test_binding_refusals():
    """The binding names what is wrong with a tensor before the library is called."""
    import torch

    e = _lib()
    x = torch.zeros(4, 8, 4)
    with pytest.raises(ValueError, match="on the GPU"):
        e.eqtp_layer_norm(x, 1)
    with pytest.raises(ValueError, match="on the GPU"):
        e.eqtp_dropout(x, None, 0.0, 1)
    with pytest.raises(ValueError, match="on the GPU"):
        e.eqtp_dropout_add_norm(x, x, None, 0.0, 1)
    with pytest.raises(ValueError, match="on the GPU"):
        e.eqtp_layer_norm_backward(x, x, x, 1)
    with pytest.raises(TypeError, match="torch.Tensor"):
        e._check([1.0], "x", torch.float32)


def _attn_desc(e, **kw):
    d = dict(lmax=3, C=64, heads=4, kv_heads=2, x_dtype=0, scale=0.1)
    d.update(kw)
    return e._AttentionDesc(ctypes.sizeof(e._AttentionDesc), d["lmax"], d["C"], d["heads"], d["kv_heads"], d["x_dtype"],
                            d["scale"])


@pytest.mark.parametrize("kw,want", [
    (dict(lmax=-1), 1), (dict(lmax=7), 2), (dict(C=0), 1), (dict(heads=0), 1), (dict(heads=5), 1), (dict(kv_heads=3), 1),
    (dict(kv_heads=0), 1), (dict(kv_heads=8), 1), (dict(C=1024, heads=4), 2), (dict(lmax=0, C=2049, heads=1, kv_heads=1), 2),
    (dict(lmax=0, C=2048, heads=2048, kv_heads=1), 2), (dict(x_dtype=2), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1)])
def test_attention_descriptor(kw, want):
    e = _lib()
    lib = e.load_library()
    d = ctypes.byref(_attn_desc(e, **kw))
    assert lib.eqtp_attention_workspace_bytes(d, 4, 4, 8) == -want
    assert lib.eqtp_attention_backward_workspace_bytes(d, 4, 4, 8) == -want
    assert lib.eqtp_attention(d, 4, 4, 8, *[FAKE] * 9, 1 << 40, NULL) == want
    assert lib.eqtp_attention_backward(d, 4, 4, 8, *[FAKE] * 16, 1 << 40, NULL) == want


def test_attention_pointers_and_sizes():
    e = _lib()
    lib = e.load_library()
    d = ctypes.byref(_attn_desc(e))
    bad = _attn_desc(e)
    bad.struct_size += 4
    assert lib.eqtp_attention(ctypes.byref(bad), 4, 4, 8, *[FAKE] * 9, 1 << 40, NULL) == 1
    assert lib.eqtp_attention(None, 4, 4, 8, *[FAKE] * 9, 1 << 40, NULL) == 1
    # src row_ptr q k v bias out lse workspace
    ok = [FAKE] * 9
    put = lambda k, v: ok[:k] + [v] + ok[k + 1:]
    f = lambda N, M, E, a, size=1 << 40: lib.eqtp_attention(d, N, M, E, *a, size, NULL)
    for N, M, E in ((-1, 4, 8), (4, -1, 8), (4, 4, -8), (1 << 31, 4, 8), (4, 1 << 31, 8), (4, 4, 1 << 31), (0, 4, 8), (4, 0, 8)):
        assert f(N, M, E, ok) == 1
    assert f(0, 4, 0, [NULL] * 9) == 0
    for k in (0, 1, 2, 3, 4, 6):
        assert f(4, 4, 8, put(k, NULL)) == 1
    for k in range(8):
        assert f(4, 4, 8, put(k, ODD2)) == 1
    # few long rows need a workspace
    need = lib.eqtp_attention_workspace_bytes(d, 1, 100000, 100000)
    if need > 0:
        assert f(1, 100000, 100000, put(8, NULL)) == 1 and f(1, 100000, 100000, ok, need - 1) == 1
        assert f(1, 100000, 100000, put(8, ctypes.c_void_p(0x10008))) == 1


def test_attention_backward_refusals():
    e = _lib()
    lib = e.load_library()
    d = ctypes.byref(_attn_desc(e))
    # src row_ptr q k v bias lse grad_out src_ptr dst_s perm grad_q grad_k grad_v grad_bias workspace
    ok = [FAKE] * 16
    put = lambda k, v: ok[:k] + [v] + ok[k + 1:]
    need = lib.eqtp_attention_backward_workspace_bytes(d, 4, 4, 8)
    assert need > 0
    f = lambda N, M, E, a, size=need: lib.eqtp_attention_backward(d, N, M, E, *a, size, NULL)
    assert f(4, 4, 8, ok, need - 1) == 1 and f(-1, 4, 8, ok) == 1 and f(4, 4, 1 << 31, ok) == 1
    for k in (0, 1, 2, 3, 4, 6, 7, 8, 9, 10, 15):
        assert f(4, 4, 8, put(k, NULL)) == 1
    for k in range(15):
        assert f(4, 4, 8, put(k, ODD2)) == 1
    assert f(4, 4, 8, put(15, ctypes.c_void_p(0x10008))) == 1


def test_attention_binding_refusals():
    import torch

    e = _lib()
    x = torch.zeros(4, 8, 4)
    i = torch.zeros(5, dtype=torch.int32)
    with pytest.raises(ValueError, match="on the GPU"):
        e.eqtp_attention(x, x, x, i, i, 1, 2)
    with pytest.raises(ValueError, match="on the GPU"):
        e.eqtp_attention_backward(x, x, x, i, i, x, x, i, i, i, 1, 2)
