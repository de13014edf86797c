"""Python binding of the C ABI in include/eqtp.h (argument marshalling only).

Every function has the name of the C entry point it calls.  Tensors are
PyTorch tensors on the current HIP device; work is enqueued on
``torch.cuda.current_stream()`` and nothing is synchronised.  All arithmetic
runs in the HIP library: if ``libeqtp.so`` has not been built, the first call
raises -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libeqtp.so")

EQTP_OK, EQTP_EINVAL, EQTP_EUNSUPPORTED, EQTP_EHIP, EQTP_ETOOLARGE, EQTP_EGRAPH = 0, 1, 2, 3, 4, 5
EQTP_CHECK_WORDS = 8
EQTP_PATHS_PARITY, EQTP_PATHS_SO3 = 0, 1
EQTP_W_FIXED, EQTP_W_RADIAL = 0, 1
EQTP_EDGES_DST_SORTED, EQTP_EDGES_UNSORTED = 0, 1
EQTP_ALGO_AUTO, EQTP_ALGO_NODE_MFMA, EQTP_ALGO_EDGE_VALU, EQTP_ALGO_EDGE_SO2 = 0, 1, 2, 3
EQTP_F32, EQTP_BF16, EQTP_F32_BF16 = 0, 1, 2
EQTP_SCORE_SOFTMAX, EQTP_SCORE_SIGMOID = 0, 1

EXPORTED = ("eqtp_num_paths", "eqtp_path_table", "eqtp_sh", "eqtp_conv_fused", "eqtp_conv_workspace_bytes",
            "eqtp_conv_fused_ws", "eqtp_conv_fused_noalloc", "eqtp_conv_messages",
            "eqtp_conv_backward", "eqtp_conv_backward_by_source", "eqtp_edge_rows", "eqtp_sort_edges",
            "eqtp_sort_workspace_bytes", "eqtp_sort_edges_stable",
            "eqtp_linear", "eqtp_interaction_workspace_bytes", "eqtp_interaction",
            "eqtp_layer_norm", "eqtp_dropout_add_norm", "eqtp_layer_norm_workspace_bytes",
            "eqtp_layer_norm_backward", "eqtp_dropout",
            "eqtp_attention_workspace_bytes", "eqtp_attention", "eqtp_attention_backward_workspace_bytes",
            "eqtp_attention_backward",
            "eqtp_distance_bias", "eqtp_distance_bias_workspace_bytes", "eqtp_distance_bias_backward",
            "eqtp_qk_norm", "eqtp_qk_norm_workspace_bytes", "eqtp_qk_norm_backward",
            "eqtp_route", "eqtp_route_backward", "eqtp_expert_plan_workspace_bytes", "eqtp_expert_plan",
            "eqtp_expert_linear", "eqtp_expert_linear_backward_workspace_bytes", "eqtp_expert_linear_backward",
            "eqtp_status_string", "eqtp_check_graph", "eqtp_set_debug", "eqtp_test_segment_probe")


class EqtpError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s" % (where, eqtp_status_string(status)))


class _ConvDesc(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_int32), ("lmax", ctypes.c_int32), ("C", ctypes.c_int32),
                ("path_set", ctypes.c_int32), ("weight_mode", ctypes.c_int32), ("edge_order", ctypes.c_int32),
                ("algo", ctypes.c_int32), ("r_cut", ctypes.c_float), ("n_basis", ctypes.c_int32),
                ("x_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


class _InteractionDesc(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_int32), ("lmax", ctypes.c_int32), ("C", ctypes.c_int32),
                ("path_set", ctypes.c_int32), ("r_cut", ctypes.c_float), ("n_basis", ctypes.c_int32),
                ("hidden", ctypes.c_int32), ("norm", ctypes.c_float)]


class _NormDesc(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_int32), ("lmax", ctypes.c_int32), ("C", ctypes.c_int32),
                ("x_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("eps", ctypes.c_float),
                ("p", ctypes.c_double)]


class _AttentionDesc(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_int32), ("lmax", ctypes.c_int32), ("C", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("x_dtype", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class _BiasDesc(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_int32), ("heads", ctypes.c_int32), ("buckets", ctypes.c_int32),
                ("r_cut", ctypes.c_float)]


class _QkNormDesc(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_int32), ("lmax", ctypes.c_int32), ("C", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("x_dtype", ctypes.c_int32),
                ("axes", ctypes.c_int32), ("pairs", ctypes.c_int32), ("eps", ctypes.c_float)]


class _RouteDesc(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_int32), ("experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32), ("score", ctypes.c_int32),
                ("renormalise", ctypes.c_int32), ("x_dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class _ExpertDesc(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_int32), ("lmax", ctypes.c_int32), ("C", ctypes.c_int32),
                ("experts", ctypes.c_int32), ("top_k", ctypes.c_int32), ("x_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32)]


_lib = None
_lock = threading.Lock()


def load_library(path: str = LIB_PATH):
    """Load libeqtp.so (raises if it has not been built)."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError("HIP library %s not built; run `python -m spherical_harmonic_cg_amd.build`" % path)
            lib = ctypes.CDLL(path)
            vp, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
            lib.eqtp_num_paths.argtypes = [i32, i32]
            lib.eqtp_num_paths.restype = i32
            lib.eqtp_path_table.argtypes = [i32, i32, vp]
            lib.eqtp_path_table.restype = i32
            lib.eqtp_sh.argtypes = [vp, i64, i32, vp, vp]
            lib.eqtp_sh.restype = i32
            lib.eqtp_conv_fused.argtypes = [ctypes.POINTER(_ConvDesc), i64, i64, vp, vp, vp, vp, vp, vp, vp, vp]
            lib.eqtp_conv_fused.restype = i32
            lib.eqtp_conv_workspace_bytes.argtypes = [ctypes.POINTER(_ConvDesc), i64, i64]
            lib.eqtp_conv_workspace_bytes.restype = i64
            lib.eqtp_conv_fused_ws.argtypes = [ctypes.POINTER(_ConvDesc), i64, i64] + [vp] * 8 + [i64, vp]
            lib.eqtp_conv_fused_ws.restype = i32
            lib.eqtp_conv_fused_noalloc.argtypes = [ctypes.POINTER(_ConvDesc), i64, i64] + [vp] * 8
            lib.eqtp_conv_fused_noalloc.restype = i32
            lib.eqtp_conv_messages.argtypes = [ctypes.POINTER(_ConvDesc), i64, i64] + [vp] * 6
            lib.eqtp_conv_messages.restype = i32
            lib.eqtp_conv_backward.argtypes = [ctypes.POINTER(_ConvDesc), i64, i64] + [vp] * 11
            lib.eqtp_conv_backward.restype = i32
            lib.eqtp_conv_backward_by_source.argtypes = [ctypes.POINTER(_ConvDesc), i64, i64] + [vp] * 11
            lib.eqtp_conv_backward_by_source.restype = i32
            lib.eqtp_edge_rows.argtypes = [i64, i64, vp, vp, vp]
            lib.eqtp_edge_rows.restype = i32
            lib.eqtp_sort_edges.argtypes = [i64, i64] + [vp] * 8
            lib.eqtp_sort_edges.restype = i32
            lib.eqtp_sort_workspace_bytes.argtypes = [i64, i64]
            lib.eqtp_sort_workspace_bytes.restype = i64
            lib.eqtp_sort_edges_stable.argtypes = [i64, i64] + [vp] * 8 + [i64, vp]
            lib.eqtp_sort_edges_stable.restype = i32
            lib.eqtp_linear.argtypes = [i64, i32, i32, i32, vp, vp, vp, vp]
            lib.eqtp_linear.restype = i32
            lib.eqtp_interaction_workspace_bytes.argtypes = [ctypes.POINTER(_InteractionDesc), i64, i64]
            lib.eqtp_interaction_workspace_bytes.restype = i64
            lib.eqtp_interaction.argtypes = [ctypes.POINTER(_InteractionDesc), i64, i64] + [vp] * 11 + [i64, vp]
            lib.eqtp_interaction.restype = i32
            lib.eqtp_layer_norm.argtypes = [ctypes.POINTER(_NormDesc), i64] + [vp] * 6
            lib.eqtp_layer_norm.restype = i32
            lib.eqtp_dropout_add_norm.argtypes = [ctypes.POINTER(_NormDesc), i64] + [vp] * 9
            lib.eqtp_dropout_add_norm.restype = i32
            lib.eqtp_layer_norm_workspace_bytes.argtypes = [ctypes.POINTER(_NormDesc), i64]
            lib.eqtp_layer_norm_workspace_bytes.restype = i64
            lib.eqtp_layer_norm_backward.argtypes = [ctypes.POINTER(_NormDesc), i64] + [vp] * 11 + [i64, vp]
            lib.eqtp_layer_norm_backward.restype = i32
            lib.eqtp_dropout.argtypes = [i64, i32, i32, i32, ctypes.c_double] + [vp] * 5
            lib.eqtp_dropout.restype = i32
            ap = ctypes.POINTER(_AttentionDesc)
            lib.eqtp_attention_workspace_bytes.argtypes = [ap, i64, i64, i64]
            lib.eqtp_attention_workspace_bytes.restype = i64
            lib.eqtp_attention.argtypes = [ap, i64, i64, i64] + [vp] * 9 + [i64, vp]
            lib.eqtp_attention.restype = i32
            lib.eqtp_attention_backward_workspace_bytes.argtypes = [ap, i64, i64, i64]
            lib.eqtp_attention_backward_workspace_bytes.restype = i64
            lib.eqtp_attention_backward.argtypes = [ap, i64, i64, i64] + [vp] * 16 + [i64, vp]
            lib.eqtp_attention_backward.restype = i32
            bp, qp, rp, xp = (ctypes.POINTER(t) for t in (_BiasDesc, _QkNormDesc, _RouteDesc, _ExpertDesc))
            for name, args, res in (
                    ("eqtp_distance_bias", [bp, i64] + [vp] * 5, i32),
                    ("eqtp_distance_bias_workspace_bytes", [bp, i64], i64),
                    ("eqtp_distance_bias_backward", [bp, i64] + [vp] * 5 + [i64, vp], i32),
                    ("eqtp_qk_norm", [qp, i64, i64] + [vp] * 10, i32),
                    ("eqtp_qk_norm_workspace_bytes", [qp, i64, i64], i64),
                    ("eqtp_qk_norm_backward", [qp, i64, i64] + [vp] * 16 + [i64, vp], i32),
                    ("eqtp_route", [rp, i64] + [vp] * 5, i32),
                    ("eqtp_route_backward", [rp, i64] + [vp] * 5, i32),
                    ("eqtp_expert_plan_workspace_bytes", [i64, i32, i32], i64),
                    ("eqtp_expert_plan", [i64, i32, i32] + [vp] * 5 + [i64, vp], i32),
                    ("eqtp_expert_linear", [xp, i64] + [vp] * 7, i32),
                    ("eqtp_expert_linear_backward_workspace_bytes", [xp, i64], i64),
                    ("eqtp_expert_linear_backward", [xp, i64] + [vp] * 12 + [i64, vp], i32)):
                getattr(lib, name).argtypes = args
                getattr(lib, name).restype = res
            lib.eqtp_status_string.argtypes = [i32]
            lib.eqtp_status_string.restype = ctypes.c_char_p
            lib.eqtp_check_graph.argtypes = [i64, i64] + [vp] * 6
            lib.eqtp_check_graph.restype = i32
            lib.eqtp_set_debug.argtypes = [i32]
            lib.eqtp_set_debug.restype = i32
            lib.eqtp_test_segment_probe.argtypes = [vp, vp, i64, i64, i32, i32, i32, vp, vp, vp]
            lib.eqtp_test_segment_probe.restype = i32
            _lib = lib
    return _lib


# The per-call marshalling is on the host's critical path for small graphs (a launch takes a few µs), so
# the helpers below take the cheap route first: the raw current stream of the current device, pointers as
# plain ints (ctypes converts them for c_void_p arguments), and one combined test per tensor before the
# detailed checks that name what is wrong.
_raw_stream = None


def _stream():
    global _raw_stream
    if _raw_stream is None:
        import torch

        get_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        get_dev = getattr(torch._C, "_cuda_getDevice", None)
        if get_raw is not None and get_dev is not None:
            _raw_stream = lambda: get_raw(get_dev())
        else:
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream
    return _raw_stream()


def _ptr(t):
    return t.data_ptr() if t is not None and t.numel() > 0 else None


def _check(t, name, dtype, shape=None):
    try:
        if t.is_cuda and t.dtype is dtype and t.is_contiguous() and (shape is None or t.shape == tuple(shape)):
            return
    except AttributeError:
        pass
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device.type != "cuda":
        raise ValueError("%s must be on the GPU" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))


def _raise(rc, where):
    if rc != EQTP_OK:
        raise EqtpError(rc, where)


def eqtp_status_string(status: int) -> str:
    return load_library().eqtp_status_string(int(status)).decode()


@functools.lru_cache(maxsize=None)
def _num_paths(lmax: int, path_set: int) -> int:
    return load_library().eqtp_num_paths(lmax, path_set)


def eqtp_num_paths(lmax: int, path_set: int = EQTP_PATHS_PARITY) -> int:
    P = _num_paths(int(lmax), int(path_set))
    if P < 0:
        raise EqtpError(-P, "eqtp_num_paths")
    return P


@functools.lru_cache(maxsize=256)
def _conv_desc(lmax, C, path_set, weight_mode, order, algo, r_cut, n_basis, x_dtype, out_dtype):
    # read by the library during a call only, so one instance per distinct descriptor is shared
    return _ConvDesc(ctypes.sizeof(_ConvDesc), lmax, C, path_set, weight_mode, order, algo, r_cut, n_basis, x_dtype,
                     out_dtype)


def eqtp_path_table(lmax: int, path_set: int = EQTP_PATHS_PARITY) -> np.ndarray:
    P = eqtp_num_paths(lmax, path_set)
    out = np.zeros((P, 3), dtype=np.int32)
    rc = load_library().eqtp_path_table(lmax, path_set, out.ctypes.data_as(ctypes.c_void_p))
    if rc < 0:
        raise EqtpError(-rc, "eqtp_path_table")
    return out


def eqtp_sh(vec, lmax: int, Y=None):
    """Y [E, (lmax+1)^2] fp32 = real spherical harmonics of vec [E, 3] fp32."""
    import torch

    _check(vec, "vec", torch.float32)
    E = vec.shape[0]
    if vec.dim() != 2 or vec.shape[1] != 3:
        raise ValueError("vec must be [E, 3]")
    K = (lmax + 1) ** 2
    if Y is None:
        Y = torch.empty((E, K), dtype=torch.float32, device=vec.device)
    _check(Y, "Y", torch.float32, (E, K))
    _raise(load_library().eqtp_sh(_ptr(vec), E, lmax, _ptr(Y), _stream()), "eqtp_sh")
    return Y


def _conv_args(vec, src, x, weights, lmax, row_ptr, dst, path_set, weight_mode, r_cut, n_basis, algo, out,
               out_dtype=EQTP_F32):
    """Checks the fused convolution's tensors; returns (descriptor, N, E, out)."""
    import torch

    x_dtype = EQTP_BF16 if x.dtype == torch.bfloat16 else EQTP_F32
    _check(x, "x", torch.bfloat16 if x_dtype == EQTP_BF16 else torch.float32)
    if x.dim() != 3:
        raise ValueError("x must be [N, C, K]")
    N, C, K = x.shape
    if K != (lmax + 1) ** 2:
        raise ValueError("x has %d components, lmax %d needs %d" % (K, lmax, (lmax + 1) ** 2))
    _check(vec, "vec", torch.float32)
    E = vec.shape[0]
    _check(src, "src", torch.int32, (E,))
    _check(weights, "weights", torch.float32)
    if (row_ptr is None) == (dst is None):
        raise ValueError("give exactly one of row_ptr (dst-sorted edges) or dst (any order)")
    if row_ptr is not None:
        _check(row_ptr, "row_ptr", torch.int32, (N + 1,))
        order = EQTP_EDGES_DST_SORTED
    else:
        _check(dst, "dst", torch.int32, (E,))
        order = EQTP_EDGES_UNSORTED
    P = eqtp_num_paths(lmax, path_set)
    wshape = (P, C) if weight_mode == EQTP_W_FIXED else (n_basis, P * C)
    if tuple(weights.shape) != wshape:
        raise ValueError("weights has shape %s, expected %s" % (tuple(weights.shape), wshape))
    odt = torch.bfloat16 if out_dtype == EQTP_BF16 else torch.float32
    if out is None:
        out = torch.empty((N, C, K), dtype=odt, device=x.device)
    _check(out, "out", odt, (N, C, K))
    d = _conv_desc(lmax, C, path_set, weight_mode, order, algo, float(r_cut), n_basis, x_dtype, out_dtype)
    return d, N, E, out


def eqtp_conv_fused(vec, src, x, weights, lmax: int, row_ptr=None, dst=None, path_set: int = EQTP_PATHS_PARITY,
                    weight_mode: int = EQTP_W_FIXED, r_cut: float = 0.0, n_basis: int = 8,
                    algo: int = EQTP_ALGO_AUTO, out=None, out_dtype: int = EQTP_F32):
    """out [N, C, K] = fused harmonics -> coupling -> sum into dst.

    Give ``row_ptr`` [N+1] for dst-sorted edges, or ``dst`` [E] for any order
    (atomic accumulation).  ``weights`` is [P, C] (fixed) or [8, P*C] (radial).
    ``x`` is float32, or bfloat16 (lmax <= 3, any edge order or weights); ``out``
    is float32, or bfloat16 with ``out_dtype=EQTP_BF16`` (edges in any order:
    packed bf16 atomics).
    """
    d, N, E, out = _conv_args(vec, src, x, weights, lmax, row_ptr, dst, path_set, weight_mode, r_cut, n_basis, algo,
                              out, out_dtype)
    rc = load_library().eqtp_conv_fused(ctypes.byref(d), N, E, _ptr(vec), _ptr(src), _ptr(dst), _ptr(row_ptr),
                                        _ptr(x), _ptr(weights), _ptr(out), _stream())
    _raise(rc, "eqtp_conv_fused")
    return out


def eqtp_conv_workspace_bytes(N: int, E: int, lmax: int, C: int, edge_order: int = EQTP_EDGES_UNSORTED,
                              weight_mode: int = EQTP_W_FIXED, path_set: int = EQTP_PATHS_PARITY) -> int:
    """Device workspace eqtp_conv_fused_ws needs (bytes)."""
    d = _ConvDesc(ctypes.sizeof(_ConvDesc), lmax, C, path_set, weight_mode, edge_order, EQTP_ALGO_AUTO, 1.0, 8,
                  EQTP_F32)
    n = load_library().eqtp_conv_workspace_bytes(ctypes.byref(d), N, E)
    if n < 0:
        raise EqtpError(-n, "eqtp_conv_workspace_bytes")
    return int(n)


def eqtp_conv_fused_ws(vec, src, x, weights, lmax: int, row_ptr=None, dst=None, path_set: int = EQTP_PATHS_PARITY,
                       weight_mode: int = EQTP_W_FIXED, r_cut: float = 0.0, n_basis: int = 8,
                       algo: int = EQTP_ALGO_AUTO, out=None, workspace=None):
    """eqtp_conv_fused with a workspace: edges in any order (``dst``) are grouped by destination on the GPU
    (rows in input order) and summed without atomics.  ``workspace`` is a uint8 CUDA tensor of at least
    eqtp_conv_workspace_bytes bytes (allocated here if None)."""
    import torch

    d, N, E, out = _conv_args(vec, src, x, weights, lmax, row_ptr, dst, path_set, weight_mode, r_cut, n_basis, algo,
                              out)
    need = load_library().eqtp_conv_workspace_bytes(ctypes.byref(d), N, E)
    if need < 0:
        _raise(-need, "eqtp_conv_workspace_bytes")
    if workspace is None:
        workspace = torch.empty(max(int(need), 16), dtype=torch.uint8, device=x.device)
    _check(workspace, "workspace", torch.uint8)
    rc = load_library().eqtp_conv_fused_ws(ctypes.byref(d), N, E, _ptr(vec), _ptr(src), _ptr(dst), _ptr(row_ptr),
                                           _ptr(x), _ptr(weights), _ptr(out), _ptr(workspace), workspace.numel(),
                                           _stream())
    _raise(rc, "eqtp_conv_fused_ws")
    return out


def eqtp_conv_fused_noalloc(vec, src, x, weights, lmax: int, row_ptr=None, dst=None,
                            path_set: int = EQTP_PATHS_PARITY, weight_mode: int = EQTP_W_FIXED, r_cut: float = 0.0,
                            n_basis: int = 8, algo: int = EQTP_ALGO_AUTO, out=None):
    """eqtp_conv_fused_ws with the library's static scratch as the workspace (no device allocation by
    the library; ``out`` must be given for a call that allocates nothing at all)."""
    d, N, E, out = _conv_args(vec, src, x, weights, lmax, row_ptr, dst, path_set, weight_mode, r_cut, n_basis, algo,
                              out)
    rc = load_library().eqtp_conv_fused_noalloc(ctypes.byref(d), N, E, _ptr(vec), _ptr(src), _ptr(dst),
                                                _ptr(row_ptr), _ptr(x), _ptr(weights), _ptr(out), _stream())
    _raise(rc, "eqtp_conv_fused_noalloc")
    return out


def eqtp_conv_messages(vec, src, x, weights, lmax: int, path_set: int = EQTP_PATHS_PARITY,
                       weight_mode: int = EQTP_W_FIXED, r_cut: float = 0.0, n_basis: int = 8, out=None,
                       algo: int = EQTP_ALGO_AUTO):
    """messages [E, C, K]: one message per edge, no destination sum (lmax 4..6 or
    algo=EQTP_ALGO_EDGE_SO2: the edge-aligned form)."""
    import torch

    _check(x, "x", torch.float32)
    if x.dim() != 3:
        raise ValueError("x must be [N, C, K]")
    N, C, K = x.shape
    if K != (lmax + 1) ** 2:
        raise ValueError("x has %d components, lmax %d needs %d" % (K, lmax, (lmax + 1) ** 2))
    _check(vec, "vec", torch.float32)
    E = vec.shape[0]
    _check(src, "src", torch.int32, (E,))
    P = eqtp_num_paths(lmax, path_set)
    wshape = (P, C) if weight_mode == EQTP_W_FIXED else (n_basis, P * C)
    _check(weights, "weights", torch.float32, wshape)
    if out is None:
        out = torch.empty((E, C, K), dtype=torch.float32, device=x.device)
    _check(out, "out", torch.float32, (E, C, K))
    d = _ConvDesc(ctypes.sizeof(_ConvDesc), lmax, C, path_set, weight_mode, EQTP_EDGES_UNSORTED, algo,
                  float(r_cut), n_basis, EQTP_F32)
    rc = load_library().eqtp_conv_messages(ctypes.byref(d), N, E, _ptr(vec), _ptr(src), _ptr(x), _ptr(weights),
                                           _ptr(out), _stream())
    _raise(rc, "eqtp_conv_messages")
    return out


def eqtp_conv_backward(vec, src, x, weights, grad_out, lmax: int, row_ptr=None, dst=None,
                       path_set: int = EQTP_PATHS_PARITY, need_x: bool = True, need_w: bool = True,
                       need_vec: bool = True, algo: int = EQTP_ALGO_AUTO, weight_mode: int = EQTP_W_FIXED,
                       r_cut: float = 0.0, n_basis: int = 8):
    """(grad_x [N,C,K] | None, grad_w | None, grad_vec [E,3] | None) of
    sum(grad_out * eqtp_conv_fused(...)) for fixed weights [P, C] (grad_w
    [P, C]) or, with weight_mode=EQTP_W_RADIAL, radial weights
    [n_basis, P*C] (grad_w of the same shape)."""
    import torch

    _check(x, "x", torch.float32)
    if x.dim() != 3:
        raise ValueError("x must be [N, C, K]")
    N, C, K = x.shape
    if K != (lmax + 1) ** 2:
        raise ValueError("x has %d components, lmax %d needs %d" % (K, lmax, (lmax + 1) ** 2))
    _check(grad_out, "grad_out", torch.float32, (N, C, K))
    _check(vec, "vec", torch.float32)
    E = vec.shape[0]
    _check(src, "src", torch.int32, (E,))
    if (row_ptr is None) == (dst is None):
        raise ValueError("give exactly one of row_ptr (dst-sorted edges) or dst (any order)")
    if row_ptr is not None:
        _check(row_ptr, "row_ptr", torch.int32, (N + 1,))
        order = EQTP_EDGES_DST_SORTED
    else:
        _check(dst, "dst", torch.int32, (E,))
        order = EQTP_EDGES_UNSORTED
    P = eqtp_num_paths(lmax, path_set)
    _check(weights, "weights", torch.float32, (P, C) if weight_mode == EQTP_W_FIXED else (n_basis, P * C))
    if not (need_x or need_w or need_vec):
        raise ValueError("request at least one gradient")
    gx = torch.empty_like(x) if need_x else None
    gw = torch.empty_like(weights) if need_w else None
    gv = torch.empty((E, 3), dtype=torch.float32, device=x.device) if need_vec else None
    d = _ConvDesc(ctypes.sizeof(_ConvDesc), lmax, C, path_set, weight_mode, order, algo, float(r_cut), n_basis,
                  EQTP_F32)
    rc = load_library().eqtp_conv_backward(ctypes.byref(d), N, E, _ptr(vec), _ptr(src), _ptr(dst), _ptr(row_ptr),
                                           _ptr(x), _ptr(weights), _ptr(grad_out), _ptr(gx), _ptr(gw), _ptr(gv),
                                           _stream())
    _raise(rc, "eqtp_conv_backward")
    return gx, gw, gv


def eqtp_conv_backward_by_source(vec_s, dst_s, src_ptr, x, weights, grad_out, lmax: int,
                                 path_set: int = EQTP_PATHS_PARITY, need_x: bool = True, need_w: bool = True,
                                 need_vec: bool = False, perm=None, weight_mode: int = EQTP_W_FIXED,
                                 r_cut: float = 0.0, n_basis: int = 8, algo: int = EQTP_ALGO_AUTO):
    """(grad_x [N,C,K] | None, grad_w | None, grad_vec [E,3] | None) from the
    edges grouped by source node: src_ptr [N+1] CSR over sources, vec_s [E,3] /
    dst_s [E] in that order, perm [E] (needed for grad_vec) the caller's index of
    each grouped edge (see eqtp_sort_edges).  grad_vec is in the caller's edge
    order.  Fixed weights [P, C] or, with weight_mode=EQTP_W_RADIAL, radial
    weights [n_basis, P*C] (grad_w of the same shape)."""
    import torch

    _check(grad_out, "grad_out", torch.float32)
    if grad_out.dim() != 3:
        raise ValueError("grad_out must be [N, C, K]")
    N, C, K = grad_out.shape
    if K != (lmax + 1) ** 2:
        raise ValueError("grad_out has %d components, lmax %d needs %d" % (K, lmax, (lmax + 1) ** 2))
    _check(vec_s, "vec_s", torch.float32)
    E = vec_s.shape[0]
    _check(dst_s, "dst_s", torch.int32, (E,))
    _check(src_ptr, "src_ptr", torch.int32, (N + 1,))
    _check(x, "x", torch.float32, (N, C, K))
    P = eqtp_num_paths(lmax, path_set)
    _check(weights, "weights", torch.float32, (P, C) if weight_mode == EQTP_W_FIXED else (n_basis, P * C))
    if not (need_x or need_w or need_vec):
        raise ValueError("request at least one gradient")
    if need_vec:
        if perm is None:
            raise ValueError("grad_vec needs perm (the caller's index of each grouped edge)")
        _check(perm, "perm", torch.int32, (E,))
    gx = torch.empty_like(grad_out) if need_x else None
    gw = torch.empty_like(weights) if need_w else None
    gv = torch.empty((E, 3), dtype=torch.float32, device=grad_out.device) if need_vec else None
    d = _ConvDesc(ctypes.sizeof(_ConvDesc), lmax, C, path_set, weight_mode, EQTP_EDGES_DST_SORTED, algo,
                  float(r_cut), n_basis, EQTP_F32)
    rc = load_library().eqtp_conv_backward_by_source(ctypes.byref(d), N, E, _ptr(vec_s), _ptr(dst_s), _ptr(src_ptr),
                                                     _ptr(x), _ptr(weights), _ptr(grad_out), _ptr(gx), _ptr(gw),
                                                     _ptr(perm if need_vec else None), _ptr(gv), _stream())
    _raise(rc, "eqtp_conv_backward_by_source")
    return gx, gw, gv


def eqtp_check_graph(N: int, E: int, row_ptr=None, src=None, dst=None, vec=None, report=None):
    """Graph checks on the GPU: report [EQTP_CHECK_WORDS] int32 (counts of out-of-range src / dst,
    decreasing row_ptr steps, row_ptr endpoint faults, edges outside their dst's row, non-finite
    vectors; then the first offending edge and row, -1 if none).  Any array may be None."""
    import torch

    for t, name, dt, shape in ((row_ptr, "row_ptr", torch.int32, (N + 1,)), (src, "src", torch.int32, (E,)),
                               (dst, "dst", torch.int32, (E,)), (vec, "vec", torch.float32, (E, 3))):
        if t is not None:
            _check(t, name, dt, shape)
    dev = next((t.device for t in (row_ptr, src, dst, vec) if t is not None), torch.device("cuda"))
    rep = report if report is not None else torch.empty(EQTP_CHECK_WORDS, dtype=torch.int32, device=dev)
    _check(rep, "report", torch.int32, (EQTP_CHECK_WORDS,))
    rc = load_library().eqtp_check_graph(N, E, _ptr(row_ptr), _ptr(src), _ptr(dst), _ptr(vec), _ptr(rep), _stream())
    _raise(rc, "eqtp_check_graph")
    return rep


def eqtp_set_debug(on: bool) -> bool:
    """Switch the library's debug mode (graph checks before every launch); returns the previous setting."""
    return bool(load_library().eqtp_set_debug(1 if on else 0))


def eqtp_edge_rows(row_ptr, E: int, out=None):
    """rows [E] int32: the destination row of every edge of a dst-sorted CSR."""
    import torch

    _check(row_ptr, "row_ptr", torch.int32)
    N = row_ptr.shape[0] - 1
    rows = out if out is not None else torch.empty(E, dtype=torch.int32, device=row_ptr.device)
    _check(rows, "rows", torch.int32, (E,))
    rc = load_library().eqtp_edge_rows(N, E, _ptr(row_ptr), _ptr(rows), _stream())
    _raise(rc, "eqtp_edge_rows")
    return rows


def eqtp_sort_edges(dst, N: int, vec=None, src=None, out=None):
    """(row_ptr [N+1], perm [E], vec[perm] | None, src[perm] | None): edges grouped
    by destination (order inside a row unspecified).  ``out`` may give the four
    output tensors (the last two None when vec / src are not given)."""
    import torch

    _check(dst, "dst", torch.int32)
    E = dst.shape[0]
    dev = dst.device
    if out is None:
        out = (torch.empty(N + 1, dtype=torch.int32, device=dev), torch.empty(E, dtype=torch.int32, device=dev),
               torch.empty_like(vec) if vec is not None else None, torch.empty_like(src) if src is not None else None)
    row_ptr, perm, vs, ss = out
    _check(row_ptr, "row_ptr", torch.int32, (N + 1,))
    _check(perm, "perm", torch.int32, (E,))
    if vec is not None:
        _check(vec, "vec", torch.float32, (E, 3))
        _check(vs, "vec_sorted", torch.float32, (E, 3))
    if src is not None:
        _check(src, "src", torch.int32, (E,))
        _check(ss, "src_sorted", torch.int32, (E,))
    rc = load_library().eqtp_sort_edges(N, E, _ptr(dst), _ptr(vec), _ptr(src), _ptr(row_ptr), _ptr(perm),
                                        _ptr(vs if vec is not None else None), _ptr(ss if src is not None else None),
                                        _stream())
    _raise(rc, "eqtp_sort_edges")
    return row_ptr, perm, (vs if vec is not None else None), (ss if src is not None else None)


def eqtp_sort_workspace_bytes(N: int, E: int) -> int:
    """Device workspace eqtp_sort_edges_stable needs (bytes)."""
    n = load_library().eqtp_sort_workspace_bytes(N, E)
    if n < 0:
        raise EqtpError(-n, "eqtp_sort_workspace_bytes")
    return int(n)


def eqtp_sort_edges_stable(dst, N: int, vec=None, src=None, out=None, workspace=None):
    """eqtp_sort_edges with every row in input order (stable radix sort): the same four outputs, unique
    and identical from call to call.  ``workspace`` is a uint8 CUDA tensor of at least
    eqtp_sort_workspace_bytes bytes (allocated here if None)."""
    import torch

    _check(dst, "dst", torch.int32)
    E = dst.shape[0]
    dev = dst.device
    if out is None:
        out = (torch.empty(N + 1, dtype=torch.int32, device=dev), torch.empty(E, dtype=torch.int32, device=dev),
               torch.empty_like(vec) if vec is not None else None, torch.empty_like(src) if src is not None else None)
    row_ptr, perm, vs, ss = out
    _check(row_ptr, "row_ptr", torch.int32, (N + 1,))
    _check(perm, "perm", torch.int32, (E,))
    if vec is not None:
        _check(vec, "vec", torch.float32, (E, 3))
        _check(vs, "vec_sorted", torch.float32, (E, 3))
    if src is not None:
        _check(src, "src", torch.int32, (E,))
        _check(ss, "src_sorted", torch.int32, (E,))
    need = eqtp_sort_workspace_bytes(N, E)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    _check(workspace, "workspace", torch.uint8)
    rc = load_library().eqtp_sort_edges_stable(N, E, _ptr(dst), _ptr(vec), _ptr(src), _ptr(row_ptr), _ptr(perm),
                                               _ptr(vs if vec is not None else None),
                                               _ptr(ss if src is not None else None), _ptr(workspace),
                                               workspace.numel(), _stream())
    _raise(rc, "eqtp_sort_edges_stable")
    return row_ptr, perm, (vs if vec is not None else None), (ss if src is not None else None)


def eqtp_linear(h, W, lmax: int, dtype: int = EQTP_F32, out=None):
    """out[n, c', l m] = sum_c W[l, c', c] h[n, c, l m] (fp32 out).

    float32 h and W: dtype EQTP_F32 (fp32 products) or EQTP_BF16 / EQTP_F32_BF16 (each value rounded to
    bf16 for the products; passed to the library as EQTP_F32_BF16).  bfloat16 h and W: bf16 storage and
    products (EQTP_BF16)."""
    import torch

    if h.dtype == torch.bfloat16:
        if dtype not in (EQTP_BF16, EQTP_F32_BF16):
            raise ValueError("bfloat16 h needs dtype EQTP_BF16")
        st, cdt = torch.bfloat16, EQTP_BF16
    else:
        st = torch.float32
        cdt = EQTP_F32 if dtype == EQTP_F32 else EQTP_F32_BF16
    _check(h, "h", st)
    N, C, K = h.shape
    _check(W, "W", st, (lmax + 1, C, C))
    if out is None:
        out = torch.empty((N, C, K), dtype=torch.float32, device=h.device)
    _check(out, "out", torch.float32, (N, C, K))
    _raise(load_library().eqtp_linear(N, C, lmax, cdt, _ptr(h), _ptr(W), _ptr(out), _stream()), "eqtp_linear")
    return out


def _ix_desc(lmax, C, path_set, r_cut, norm):
    return _InteractionDesc(ctypes.sizeof(_InteractionDesc), lmax, C, path_set, float(r_cut), 8, 64, float(norm))


def eqtp_interaction_workspace_bytes(N: int, E: int, lmax: int, C: int, r_cut: float = 1.0, norm: float = 1.0,
                                     path_set: int = EQTP_PATHS_PARITY) -> int:
    d = _ix_desc(lmax, C, path_set, r_cut, norm)
    n = load_library().eqtp_interaction_workspace_bytes(ctypes.byref(d), N, E)
    if n < 0:
        _raise(int(-n), "eqtp_interaction_workspace_bytes")
    return int(n)


def eqtp_interaction(vec, src, row_ptr, h, W_up, W1, W2, W3, W_out, lmax: int, r_cut: float, norm: float = 1.0,
                     path_set: int = EQTP_PATHS_PARITY, workspace=None, out=None):
    """One interaction layer (see include/eqtp.h): out [N, C, K] fp32 from node features h [N, C, K],
    dst-sorted edges (vec, src, row_ptr) and the weights W_up, W_out [lmax+1, C, C], W1 [8, 64],
    W2 [64, 64], W3 [64, P*C].  ``workspace``: a uint8 tensor of at least
    eqtp_interaction_workspace_bytes bytes, or None to allocate one here."""
    import torch

    _check(h, "h", torch.float32)
    if h.dim() != 3:
        raise ValueError("h must be [N, C, K]")
    N, C, K = h.shape
    if K != (lmax + 1) ** 2:
        raise ValueError("h has %d components, lmax %d needs %d" % (K, lmax, (lmax + 1) ** 2))
    _check(vec, "vec", torch.float32)
    E = vec.shape[0]
    _check(src, "src", torch.int32, (E,))
    _check(row_ptr, "row_ptr", torch.int32, (N + 1,))
    P = eqtp_num_paths(lmax, path_set)
    _check(W_up, "W_up", torch.float32, (lmax + 1, C, C))
    _check(W_out, "W_out", torch.float32, (lmax + 1, C, C))
    _check(W1, "W1", torch.float32, (8, 64))
    _check(W2, "W2", torch.float32, (64, 64))
    _check(W3, "W3", torch.float32, (64, P * C))
    d = _ix_desc(lmax, C, path_set, r_cut, norm)
    need = eqtp_interaction_workspace_bytes(N, E, lmax, C, r_cut, norm, path_set)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=h.device)
    _check(workspace, "workspace", torch.uint8)
    if out is None:
        out = torch.empty((N, C, K), dtype=torch.float32, device=h.device)
    _check(out, "out", torch.float32, (N, C, K))
    rc = load_library().eqtp_interaction(ctypes.byref(d), N, E, _ptr(vec), _ptr(src), _ptr(row_ptr), _ptr(h),
                                         _ptr(W_up), _ptr(W1), _ptr(W2), _ptr(W3), _ptr(W_out), _ptr(out),
                                         _ptr(workspace), workspace.numel(), _stream())
    _raise(rc, "eqtp_interaction")
    return out


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch

        _torch_module = torch
    return _torch_module


def _like(x, code, own):
    """An empty tensor of x's shape and the type of a code; `own` is x's."""
    torch = _torch()
    return torch.empty_like(x) if code == own else torch.empty_like(x, dtype=_torch_dtype(code))


def _rows(x, name, lmax):
    """(element type code, N, C) of features [N, C, K], or [N, C] at lmax 0."""
    torch = _torch()
    try:  # the usual case in one test
        dt = x.dtype
        if x.is_cuda and x.is_contiguous() and (dt is torch.float32 or dt is torch.bfloat16):
            N, C, K = x.shape
            if K == (lmax + 1) ** 2:
                return (EQTP_F32 if dt is torch.float32 else EQTP_BF16), N, C
    except (AttributeError, ValueError):
        pass
    code = EQTP_BF16 if x.dtype is torch.bfloat16 else EQTP_F32
    _check(x, name, torch.bfloat16 if code == EQTP_BF16 else torch.float32)
    if x.dim() == 3:
        N, C, K = x.shape
        if K != (lmax + 1) ** 2:
            raise ValueError("%s has %d components, lmax %d needs %d" % (name, K, lmax, (lmax + 1) ** 2))
    elif x.dim() == 2 and lmax == 0:
        N, C = x.shape
    else:
        raise ValueError("%s must be [N, C, K] (or [N, C] at lmax 0)" % name)
    return code, N, C


def _check_rng(rng, p):
    torch = _torch()
    if p == 0.0:
        return
    if rng is None:
        raise ValueError("p > 0 needs rng, an int64 tensor (seed, offset) on the GPU")
    _check(rng, "rng", torch.int64, (2,))


@functools.lru_cache(maxsize=256)
def _norm_desc(lmax, C, x_dtype, out_dtype, eps, p):
    # read by the library during a call only, so one instance per distinct descriptor is shared
    d = _NormDesc(ctypes.sizeof(_NormDesc), lmax, C, x_dtype, out_dtype, eps, p)
    need = load_library().eqtp_layer_norm_workspace_bytes(ctypes.byref(d), 0)  # checks the descriptor
    if need < 0:
        raise EqtpError(int(-need), "eqtp_norm_desc")
    return ctypes.byref(d), d


def _check_affine(weight, bias, lmax, C):
    torch = _torch()
    if weight is not None:
        _check(weight, "weight", torch.float32, (lmax + 1, C))
    if bias is not None:
        _check(bias, "bias", torch.float32, (C,))


def _torch_dtype(code):
    torch = _torch()
    if code not in (EQTP_F32, EQTP_BF16):
        raise ValueError("out_dtype must be EQTP_F32 or EQTP_BF16")
    return torch.bfloat16 if code == EQTP_BF16 else torch.float32


def eqtp_layer_norm(x, lmax: int, weight=None, bias=None, eps: float = 1e-5, out_dtype: int = None, out=None,
                    stats=None):
    """out [N, C, K] = layer norm by degree of x (see include/eqtp.h); x float32 or bfloat16, [N, C, K] or, at
    lmax 0, [N, C].  ``weight`` [lmax+1, C], ``bias`` [C] float32.  ``out_dtype``: EQTP_F32 or EQTP_BF16 (x's by
    default).  ``stats``: a float32 [N, lmax+2] tensor to fill, for eqtp_layer_norm_backward."""
    torch = _torch()
    code, N, C = _rows(x, "x", lmax)
    ocode = code if out_dtype is None else out_dtype
    odt = _torch_dtype(ocode)
    _check_affine(weight, bias, lmax, C)
    d, _ = _norm_desc(lmax, C, code, ocode, float(eps), 0.0)
    if out is None:
        out = _like(x, ocode, code)
    else:
        _check(out, "out", odt, x.shape)
    if stats is not None:
        _check(stats, "stats", torch.float32, (N, lmax + 2))
    _raise(load_library().eqtp_layer_norm(d, N, _ptr(x), _ptr(weight), _ptr(bias), _ptr(out), _ptr(stats), _stream()),
           "eqtp_layer_norm")
    return out


def eqtp_dropout_add_norm(x, residual, rng, p: float, lmax: int, weight=None, bias=None, eps: float = 1e-5,
                          out_dtype: int = None, out=None, total=None, stats=None):
    """(out, total): total = residual + dropout(x), out = eqtp_layer_norm(total), in one pass.  ``rng``: int64
    (seed, offset) on the GPU, or None when p is 0.  The rest as for eqtp_layer_norm."""
    torch = _torch()
    code, N, C = _rows(x, "x", lmax)
    _check(residual, "residual", x.dtype, x.shape)
    ocode = code if out_dtype is None else out_dtype
    odt = _torch_dtype(ocode)
    p = float(p)
    _check_rng(rng, p)
    _check_affine(weight, bias, lmax, C)
    d, _ = _norm_desc(lmax, C, code, ocode, float(eps), p)
    if out is None:
        out = _like(x, ocode, code)
    else:
        _check(out, "out", odt, x.shape)
    if total is None:
        total = torch.empty_like(x)
    else:
        _check(total, "total", x.dtype, x.shape)
    if stats is not None:
        _check(stats, "stats", torch.float32, (N, lmax + 2))
    rc = load_library().eqtp_dropout_add_norm(d, N, _ptr(x), _ptr(residual), _ptr(rng), _ptr(weight), _ptr(bias),
                                              _ptr(total), _ptr(out), _ptr(stats), _stream())
    _raise(rc, "eqtp_dropout_add_norm")
    return out, total


def eqtp_layer_norm_workspace_bytes(N: int, C: int, lmax: int) -> int:
    """Device workspace eqtp_layer_norm_backward needs for the gradients of weight and bias (bytes)."""
    d, _ = _norm_desc(lmax, C, EQTP_F32, EQTP_F32, 1e-5, 0.0)
    n = load_library().eqtp_layer_norm_workspace_bytes(d, N)
    if n < 0:
        raise EqtpError(int(-n), "eqtp_layer_norm_workspace_bytes")
    return int(n)


def eqtp_layer_norm_backward(total, stats, grad_out, lmax: int, weight=None, grad_total=None, rng=None,
                             p: float = 0.0, need_residual: bool = True, need_x: bool = None,
                             need_weight: bool = True, need_bias: bool = True, workspace=None):
    """(grad_residual, grad_x, grad_weight, grad_bias) of eqtp_dropout_add_norm, each None if not asked for; of
    eqtp_layer_norm with ``total`` = x, whose gradient is grad_residual.  ``need_x`` defaults to p > 0.
    ``workspace``: a uint8 tensor of at least eqtp_layer_norm_workspace_bytes bytes, or None to allocate one."""
    torch = _torch()
    code, N, C = _rows(total, "total", lmax)
    ocode = EQTP_BF16 if grad_out.dtype is torch.bfloat16 else EQTP_F32
    _check(grad_out, "grad_out", _torch_dtype(ocode), total.shape)
    _check(stats, "stats", torch.float32, (N, lmax + 2))
    _check_affine(weight, None, lmax, C)
    if grad_total is not None:
        _check(grad_total, "grad_total", total.dtype, total.shape)
    p = float(p)
    if need_x is None:
        need_x = p > 0.0
    if need_x:
        _check_rng(rng, p)
    d, _ = _norm_desc(lmax, C, code, ocode, 1e-5, p)
    dev = total.device
    gr = torch.empty_like(total) if need_residual else None
    gx = torch.empty_like(total) if need_x else None
    gw = torch.empty((lmax + 1, C), dtype=torch.float32, device=dev) if need_weight else None
    gb = torch.empty((C,), dtype=torch.float32, device=dev) if need_bias else None
    if need_weight or need_bias:
        if workspace is None:
            workspace = torch.empty(load_library().eqtp_layer_norm_workspace_bytes(d, N), dtype=torch.uint8, device=dev)
        else:
            _check(workspace, "workspace", torch.uint8)
    rc = load_library().eqtp_layer_norm_backward(d, N, _ptr(total), _ptr(stats), _ptr(weight), _ptr(grad_out),
                                                 _ptr(grad_total), _ptr(rng), _ptr(gr), _ptr(gx), _ptr(gw), _ptr(gb),
                                                 _ptr(workspace), workspace.numel() if workspace is not None else 0,
                                                 _stream())
    _raise(rc, "eqtp_layer_norm_backward")
    return gr, gx, gw, gb


def eqtp_dropout(x, rng, p: float, lmax: int = 0, residual=None, out=None):
    """out [N, C, K] = residual + dropout(x) of whole channels (see include/eqtp.h); without residual dropout(x),
    which on a gradient, with the same rng, is the backward pass.  ``out`` may be x or residual."""
    torch = _torch()
    code, N, C = _rows(x, "x", lmax)
    p = float(p)
    _check_rng(rng, p)
    if residual is not None:
        _check(residual, "residual", x.dtype, x.shape)
    if out is None:
        out = torch.empty_like(x)
    else:
        _check(out, "out", x.dtype, x.shape)
    rc = load_library().eqtp_dropout(N, C, lmax, code, p, _ptr(x), _ptr(residual), _ptr(rng), _ptr(out), _stream())
    _raise(rc, "eqtp_dropout")
    return out


@functools.lru_cache(maxsize=256)
def _attention_desc(lmax, C, heads, kv_heads, x_dtype, scale):
    # read by the library during a call only, so one instance per distinct descriptor is shared
    if scale is None:
        scale = (C // heads * (lmax + 1) ** 2) ** -0.5 if heads > 0 and C >= heads else 1.0
    d = _AttentionDesc(ctypes.sizeof(_AttentionDesc), lmax, C, heads, kv_heads, x_dtype, scale)
    need = load_library().eqtp_attention_workspace_bytes(ctypes.byref(d), 0, 0, 0)  # checks the descriptor
    if need < 0:
        raise EqtpError(int(-need), "eqtp_attention_desc")
    return ctypes.byref(d), d


def _attention_args(q, k, v, src, row_ptr, lmax, heads, scale, bias):
    """Checks the attention's tensors; returns (descriptor, N, M, E)."""
    torch = _torch()
    code, N, C = _rows(q, "q", lmax)
    dt = q.dtype
    _check(k, "k", dt)
    ks = k.shape
    if len(ks) != q.dim() or (len(ks) == 3 and ks[2] != (lmax + 1) ** 2):
        raise ValueError("k must be [M, C kv_heads / heads, K] as q is [N, C, K]")
    _check(v, "v", dt, ks)
    M, Ck = ks[0], ks[1]
    if heads <= 0 or C % heads != 0:
        raise ValueError("heads must divide the %d channels of q" % C)
    width = C // heads
    if width == 0 or Ck == 0 or Ck % width != 0 or heads % (Ck // width) != 0:
        raise ValueError("k has %d channels: heads of %d channels, their number a divisor of %d" % (Ck, width, heads))
    E = src.numel()
    _check(src, "src", torch.int32, (E,))
    _check(row_ptr, "row_ptr", torch.int32, (N + 1,))
    if bias is not None:
        _check(bias, "bias", torch.float32, (E, heads))
    # the scale as a number: a tensor would be found in the descriptors' cache by its identity, whatever it holds by now
    return _attention_desc(lmax, C, heads, Ck // width, code, None if scale is None else float(scale))[0], N, M, E


def _workspace(workspace, need, dev):
    torch = _torch()
    if need < 0:
        raise EqtpError(int(-need), "workspace size")
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev) if need > 0 else None
    _check(workspace, "workspace", torch.uint8)
    return workspace


def eqtp_attention_workspace_bytes(N: int, M: int, E: int, lmax: int, C: int, heads: int, kv_heads: int = None) -> int:
    """Device workspace eqtp_attention needs (bytes; often 0)."""
    d, _ = _attention_desc(lmax, C, heads, heads if kv_heads is None else kv_heads, EQTP_F32, None)
    n = load_library().eqtp_attention_workspace_bytes(d, N, M, E)
    if n < 0:
        raise EqtpError(int(-n), "eqtp_attention_workspace_bytes")
    return int(n)


def eqtp_attention(q, k, v, src, row_ptr, lmax: int, heads: int, scale: float = None, bias=None, out=None, lse=None,
                   workspace=None):
    """out [N, C, K] = attention of q's rows over the edges of a dst-sorted graph (see include/eqtp.h).

    q [N, C, K], k and v [M, Ck, K] float32 or bfloat16 ([N, C] and [M, Ck] at lmax 0); Ck = C, or fewer heads of
    the same width that the heads of q share.  ``src`` [E], ``row_ptr`` [N+1] int32.  ``scale``: 1 / sqrt of the
    elements of a head by default.  ``bias`` [E, heads] float32, -inf to mask.  ``lse``: a float32 [N, heads]
    tensor to fill, for eqtp_attention_backward.  ``workspace``: a uint8 tensor of at least
    eqtp_attention_workspace_bytes bytes, or None to allocate one if it is needed."""
    torch = _torch()
    d, N, M, E = _attention_args(q, k, v, src, row_ptr, lmax, heads, scale, bias)
    if out is None:
        out = torch.empty_like(q)
    else:
        _check(out, "out", q.dtype, q.shape)
    if lse is not None:
        _check(lse, "lse", torch.float32, (N, heads))
    lib = load_library()
    workspace = _workspace(workspace, lib.eqtp_attention_workspace_bytes(d, N, M, E), q.device)
    rc = lib.eqtp_attention(d, N, M, E, _ptr(src), _ptr(row_ptr), _ptr(q), _ptr(k), _ptr(v), _ptr(bias), _ptr(out),
                            _ptr(lse), _ptr(workspace), workspace.numel() if workspace is not None else 0, _stream())
    _raise(rc, "eqtp_attention")
    return out


def eqtp_attention_backward_workspace_bytes(N: int, M: int, E: int, lmax: int, C: int, heads: int,
                                            kv_heads: int = None) -> int:
    """Device workspace eqtp_attention_backward needs (bytes)."""
    d, _ = _attention_desc(lmax, C, heads, heads if kv_heads is None else kv_heads, EQTP_F32, None)
    n = load_library().eqtp_attention_backward_workspace_bytes(d, N, M, E)
    if n < 0:
        raise EqtpError(int(-n), "eqtp_attention_backward_workspace_bytes")
    return int(n)


def _output_before_lse(f):
    """Lets the forward call's output stand between row_ptr and lse: perm is then where lmax is without it."""
    @functools.wraps(f)
    def call(*args, **named):
        if len(args) > 10 and (args[10] is None or isinstance(args[10], _torch().Tensor)):
            return f(*args[:5], *args[6:], out=args[5], **named)
        return f(*args, **named)
    return call


@_output_before_lse
def eqtp_attention_backward(q, k, v, src, row_ptr, lse, grad_out, src_ptr, dst_s, perm, lmax: int, heads: int,
                            scale: float = None, bias=None, need_q: bool = True, need_k: bool = True,
                            need_v: bool = True, need_bias: bool = None, workspace=None, out=None):
    """(grad_q, grad_k, grad_v, grad_bias) of eqtp_attention, each None if not asked for.  ``lse`` is the
    forward call's.  ``src_ptr`` [M+1], ``dst_s`` [E], ``perm`` [E] int32: the edges grouped by source (for grad_k
    and grad_v; e.g. autograd.attention_plan).  ``need_bias`` defaults to whether a
    bias is given.

    The forward call's output may stand between ``row_ptr`` and ``lse`` (or be given as ``out``), for programs that
    keep both.  Its shape and type are checked, its values are not read: the row sums that it could stand for are
    formed again in fp32, because a bf16 output rounds them at 2^-9."""
    torch = _torch()
    d, N, M, E = _attention_args(q, k, v, src, row_ptr, lmax, heads, scale, bias)
    if out is not None:
        _check(out, "out", q.dtype, q.shape)
    _check(lse, "lse", torch.float32, (N, heads))
    _check(grad_out, "grad_out", q.dtype, q.shape)
    if need_k or need_v:
        _check(src_ptr, "src_ptr", torch.int32, (M + 1,))
        _check(dst_s, "dst_s", torch.int32, (E,))
        _check(perm, "perm", torch.int32, (E,))
    if need_bias is None:
        need_bias = bias is not None
    gq = torch.empty_like(q) if need_q else None
    gk = torch.empty_like(k) if need_k else None
    gv = torch.empty_like(v) if need_v else None
    gb = torch.empty((E, heads), dtype=torch.float32, device=q.device) if need_bias else None
    lib = load_library()
    workspace = _workspace(workspace, lib.eqtp_attention_backward_workspace_bytes(d, N, M, E), q.device)
    rc = lib.eqtp_attention_backward(d, N, M, E, _ptr(src), _ptr(row_ptr), _ptr(q), _ptr(k), _ptr(v), _ptr(bias),
                                     _ptr(lse), _ptr(grad_out), _ptr(src_ptr), _ptr(dst_s), _ptr(perm),
                                     _ptr(gq), _ptr(gk), _ptr(gv), _ptr(gb), _ptr(workspace),
                                     workspace.numel() if workspace is not None else 0, _stream())
    _raise(rc, "eqtp_attention_backward")
    return gq, gk, gv, gb


@functools.lru_cache(maxsize=256)
def _bias_desc(heads, buckets, r_cut):
    # read by the library during a call only, so one instance per distinct descriptor is shared
    d = _BiasDesc(ctypes.sizeof(_BiasDesc), heads, buckets, r_cut)
    if r_cut != 0.0 and d.r_cut == 0.0:
        raise ValueError("r_cut = %g is 0 in float32, which would mask nothing" % r_cut)
    need = load_library().eqtp_distance_bias_workspace_bytes(ctypes.byref(d), 0)  # checks the descriptor
    if need < 0:
        raise EqtpError(int(-need), "eqtp_bias_desc")
    return ctypes.byref(d), d


def _bias_args(vec, bounds, r_cut, heads):
    torch = _torch()
    _check(vec, "vec", torch.float32)
    if vec.dim() != 2 or vec.shape[1] != 3:
        raise ValueError("vec must be [E, 3]")
    _check(bounds, "bounds", torch.float32)
    if bounds.dim() != 1:
        raise ValueError("bounds must be [B - 1]")
    return _bias_desc(int(heads), bounds.shape[0] + 1, float(r_cut))[0], vec.shape[0], bounds.shape[0] + 1


def eqtp_distance_bias(vec, bounds, table, r_cut: float = 0.0, out=None):
    """out [E, H] = the row of ``table`` [B, H] that each edge's length |vec_e| falls into (see include/eqtp.h): the
    number of ``bounds`` [B-1] (ascending) that are at most the length; -inf from ``r_cut`` on (0: no mask).  All
    float32; the result is eqtp_attention's ``bias``."""
    torch = _torch()
    _check(table, "table", torch.float32)
    if table.dim() != 2:
        raise ValueError("table must be [B, H]")
    d, E, B = _bias_args(vec, bounds, r_cut, table.shape[1])
    if table.shape[0] != B:
        raise ValueError("table has %d rows, %d bounds need %d" % (table.shape[0], B - 1, B))
    if out is None:
        out = torch.empty((E, table.shape[1]), dtype=torch.float32, device=vec.device)
    else:
        _check(out, "out", torch.float32, (E, table.shape[1]))
    _raise(load_library().eqtp_distance_bias(d, E, _ptr(vec), _ptr(bounds), _ptr(table), _ptr(out), _stream()),
           "eqtp_distance_bias")
    return out


def eqtp_distance_bias_workspace_bytes(E: int, heads: int, buckets: int) -> int:
    """Device workspace eqtp_distance_bias_backward needs (bytes)."""
    n = load_library().eqtp_distance_bias_workspace_bytes(_bias_desc(int(heads), int(buckets), 0.0)[0], E)
    if n < 0:
        raise EqtpError(int(-n), "eqtp_distance_bias_workspace_bytes")
    return int(n)


def eqtp_distance_bias_backward(vec, bounds, grad_bias, r_cut: float = 0.0, workspace=None):
    """grad_table [B, H] of eqtp_distance_bias from grad_bias [E, H] float32.  ``workspace``: a uint8 tensor of at
    least eqtp_distance_bias_workspace_bytes bytes, or None to allocate one."""
    torch = _torch()
    _check(grad_bias, "grad_bias", torch.float32)
    if grad_bias.dim() != 2:
        raise ValueError("grad_bias must be [E, H]")
    heads = grad_bias.shape[1]
    d, E, B = _bias_args(vec, bounds, r_cut, heads)
    _check(grad_bias, "grad_bias", torch.float32, (E, heads))
    grad_table = torch.empty((B, heads), dtype=torch.float32, device=vec.device)
    lib = load_library()
    workspace = _workspace(workspace, lib.eqtp_distance_bias_workspace_bytes(d, E), vec.device)
    rc = lib.eqtp_distance_bias_backward(d, E, _ptr(vec), _ptr(bounds), _ptr(grad_bias), _ptr(grad_table),
                                         _ptr(workspace), workspace.numel(), _stream())
    _raise(rc, "eqtp_distance_bias_backward")
    return grad_table


@functools.lru_cache(maxsize=256)
def _qk_norm_desc(lmax, C, heads, kv_heads, x_dtype, axes, pairs, eps):
    # read by the library during a call only, so one instance per distinct descriptor is shared
    d = _QkNormDesc(ctypes.sizeof(_QkNormDesc), lmax, C, heads, kv_heads, x_dtype, axes, pairs, eps)
    need = load_library().eqtp_qk_norm_workspace_bytes(ctypes.byref(d), 0, 0)  # checks the descriptor
    if need < 0:
        raise EqtpError(int(-need), "eqtp_qk_norm_desc")
    return ctypes.byref(d), d


def _qk_norm_args(q, k, lmax, heads, weight_q, weight_k, pos_q, pos_k, freq, eps):
    """Checks the tensors; returns (descriptor, N, M, positions of k)."""
    torch = _torch()
    code, N, C = _rows(q, "q", lmax)
    kcode, M, Ck = _rows(k, "k", lmax)
    if kcode != code:
        raise TypeError("q and k must have the same type")
    if heads <= 0 or C % heads != 0 or C == 0:
        raise ValueError("heads must divide the %d channels of q" % C)
    width = C // heads
    if Ck == 0 or Ck % width != 0:
        raise ValueError("k has %d channels: it needs heads of %d channels" % (Ck, width))
    for w, name in ((weight_q, "weight_q"), (weight_k, "weight_k")):
        if w is not None:
            _check(w, name, torch.float32, (lmax + 1, width))
    axes = pairs = 0
    if freq is not None:
        _check(freq, "freq", torch.float32)
        if freq.dim() != 2:
            raise ValueError("freq must be [axes, pairs]")
        axes, pairs = freq.shape
        if pos_k is None and M == N:
            pos_k = pos_q
        _check(pos_q, "pos_q", torch.float32, (N, axes))
        _check(pos_k, "pos_k", torch.float32, (M, axes))
    elif pos_q is not None or pos_k is not None:
        raise ValueError("positions need freq")
    return _qk_norm_desc(lmax, C, heads, Ck // width, code, axes, pairs, float(eps))[0], N, M, pos_k


def eqtp_qk_norm(q, k, lmax: int, heads: int, weight_q=None, weight_k=None, pos_q=None, pos_k=None, freq=None,
                 eps: float = 1e-5, out_q=None, out_k=None):
    """(out_q, out_k): queries and keys normed by head and degree and turned by position, in one pass (see
    include/eqtp.h).

    q [N, C, K], k [M, Ck, K] float32 or bfloat16 ([N, C] and [M, Ck] at lmax 0); Ck is a number of heads of q's
    width.  ``weight_q``, ``weight_k`` [lmax+1, C/heads] float32.  ``freq`` [axes, pairs] float32 with ``pos_q``
    [N, axes] and ``pos_k`` [M, axes] (pos_q by default where M = N), or None: no rotation.  Where space turns the
    positions, ``freq`` has to be turned, too, or logits depend on the orientation.  ``out_q`` and ``out_k`` may be q
    and k."""
    torch = _torch()
    d, N, M, pos_k = _qk_norm_args(q, k, lmax, heads, weight_q, weight_k, pos_q, pos_k, freq, eps)
    if out_q is None:
        out_q = torch.empty_like(q)
    else:
        _check(out_q, "out_q", q.dtype, q.shape)
    if out_k is None:
        out_k = torch.empty_like(k)
    else:
        _check(out_k, "out_k", k.dtype, k.shape)
    rc = load_library().eqtp_qk_norm(d, N, M, _ptr(q), _ptr(k), _ptr(weight_q), _ptr(weight_k), _ptr(pos_q), _ptr(pos_k),
                                     _ptr(freq), _ptr(out_q), _ptr(out_k), _stream())
    _raise(rc, "eqtp_qk_norm")
    return out_q, out_k


def eqtp_qk_norm_workspace_bytes(N: int, M: int, lmax: int, C: int, heads: int, kv_heads: int = None) -> int:
    """Device workspace eqtp_qk_norm_backward needs for the gradients of the weights (bytes)."""
    d = _qk_norm_desc(lmax, C, heads, heads if kv_heads is None else kv_heads, EQTP_F32, 0, 0, 1e-5)[0]
    n = load_library().eqtp_qk_norm_workspace_bytes(d, N, M)
    if n < 0:
        raise EqtpError(int(-n), "eqtp_qk_norm_workspace_bytes")
    return int(n)


def eqtp_qk_norm_backward(q, k, grad_out_q, grad_out_k, lmax: int, heads: int, weight_q=None, weight_k=None, pos_q=None,
                          pos_k=None, freq=None, eps: float = 1e-5, need_q: bool = True, need_k: bool = True,
                          need_weight_q: bool = True, need_weight_k: bool = True, need_pos: bool = False,
                          workspace=None):
    """(grad_q, grad_k, grad_weight_q, grad_weight_k, grad_pos_q, grad_pos_k) of eqtp_qk_norm, each None if not asked
    for.  A gradient of an output may be None: then nothing of its side is computed (its gradients are None).  ``workspace``: a uint8 tensor of at least
    eqtp_qk_norm_workspace_bytes bytes, or None to allocate one if it is needed."""
    torch = _torch()
    d, N, M, pos_k = _qk_norm_args(q, k, lmax, heads, weight_q, weight_k, pos_q, pos_k, freq, eps)
    if need_pos and freq is None:
        raise ValueError("gradients of positions need freq")
    sides = []
    for x, g, name, need, need_w, pos in ((q, grad_out_q, "grad_out_q", need_q, need_weight_q, pos_q),
                                          (k, grad_out_k, "grad_out_k", need_k, need_weight_k, pos_k)):
        if g is None:
            sides.append((None, None, None))
            continue
        _check(g, name, x.dtype, x.shape)
        sides.append((torch.empty_like(x) if need else None,
                      torch.empty((lmax + 1, q.shape[1] // heads), dtype=torch.float32, device=q.device) if need_w else None,
                      torch.empty_like(pos) if need_pos else None))
    (gq, gwq, gpq), (gk, gwk, gpk) = sides
    lib = load_library()
    if gwq is not None or gwk is not None:
        workspace = _workspace(workspace, max(16, lib.eqtp_qk_norm_workspace_bytes(d, N, M)), q.device)
    rc = lib.eqtp_qk_norm_backward(d, N, M, _ptr(q), _ptr(k), _ptr(weight_q), _ptr(weight_k), _ptr(pos_q), _ptr(pos_k),
                                   _ptr(freq), _ptr(grad_out_q), _ptr(grad_out_k), _ptr(gq), _ptr(gk), _ptr(gwq),
                                   _ptr(gwk), _ptr(gpq), _ptr(gpk), _ptr(workspace),
                                   workspace.numel() if workspace is not None else 0, _stream())
    _raise(rc, "eqtp_qk_norm_backward")
    return gq, gk, gwq, gwk, gpq, gpk


@functools.lru_cache(maxsize=256)
def _route_desc(experts, top_k, groups, top_groups, score, renormalise, x_dtype, scale):
    # read by the library during a call only, so one instance per distinct descriptor is shared
    d = _RouteDesc(ctypes.sizeof(_RouteDesc), experts, top_k, groups, top_groups, score, renormalise, x_dtype, scale)
    _raise(load_library().eqtp_route(ctypes.byref(d), 0, None, None, None, None, None), "eqtp_route_desc")  # checks it
    return ctypes.byref(d), d


def _logits(logits):
    torch = _torch()
    code = EQTP_BF16 if logits.dtype is torch.bfloat16 else EQTP_F32
    _check(logits, "logits", torch.bfloat16 if code == EQTP_BF16 else torch.float32)
    if logits.dim() != 2:
        raise ValueError("logits must be [N, X]")
    return code, logits.shape[0], logits.shape[1]


def eqtp_route(logits, top_k: int, score: int = EQTP_SCORE_SOFTMAX, bias=None, groups: int = 1, top_groups: int = None,
               renormalise: bool = True, scale: float = 1.0, idx=None, weight=None):
    """(idx [N, top_k] int32, weight [N, top_k] float32): each node's experts in descending order and their weights
    (see include/eqtp.h).  ``logits`` [N, X] float32 or bfloat16; ``bias`` [X] float32 steers the choice only;
    ``top_groups`` of ``groups`` groups of consecutive experts stay open (all by default)."""
    torch = _torch()
    code, N, X = _logits(logits)
    if bias is not None:
        _check(bias, "bias", torch.float32, (X,))
    d, _ = _route_desc(X, int(top_k), int(groups), int(groups if top_groups is None else top_groups), int(score),
                       int(bool(renormalise)), code, float(scale))
    if idx is None:
        idx = torch.empty((N, top_k), dtype=torch.int32, device=logits.device)
    else:
        _check(idx, "idx", torch.int32, (N, top_k))
    if weight is None:
        weight = torch.empty((N, top_k), dtype=torch.float32, device=logits.device)
    else:
        _check(weight, "weight", torch.float32, (N, top_k))
    _raise(load_library().eqtp_route(d, N, _ptr(logits), _ptr(bias), _ptr(idx), _ptr(weight), _stream()), "eqtp_route")
    return idx, weight


def eqtp_route_backward(logits, idx, grad_weight, score: int = EQTP_SCORE_SOFTMAX, renormalise: bool = True,
                        scale: float = 1.0):
    """grad_logits [N, X] (logits' type) of eqtp_route's weights, its choice ``idx`` [N, top_k] held fixed."""
    torch = _torch()
    code, N, X = _logits(logits)
    if idx.dim() != 2:
        raise ValueError("idx must be [N, top_k]")
    top_k = idx.shape[1]
    _check(idx, "idx", torch.int32, (N, top_k))
    _check(grad_weight, "grad_weight", torch.float32, (N, top_k))
    d, _ = _route_desc(X, top_k, 1, 1, int(score), int(bool(renormalise)), code, float(scale))
    out = torch.empty_like(logits)
    _raise(load_library().eqtp_route_backward(d, N, _ptr(logits), _ptr(idx), _ptr(grad_weight), _ptr(out), _stream()),
           "eqtp_route_backward")
    return out


def _choice(idx):
    _check(idx, "idx", _torch().int32)
    if idx.dim() != 2:
        raise ValueError("idx must be [N, top_k]")
    return idx.shape


def eqtp_expert_plan_workspace_bytes(N: int, top_k: int, experts: int) -> int:
    """Device workspace eqtp_expert_plan needs (bytes)."""
    n = load_library().eqtp_expert_plan_workspace_bytes(N, top_k, experts)
    if n < 0:
        raise EqtpError(int(-n), "eqtp_expert_plan_workspace_bytes")
    return int(n)


def eqtp_expert_plan(idx, experts: int, workspace=None):
    """(order [N], slots [N top_k], ptr [experts+1]) int32: a routing grouped by expert (see include/eqtp.h), for
    eqtp_expert_linear and its backward call; made once, it serves every layer that uses the routing.  Differences of
    ptr are the experts' loads.  With top_k = 1, order is slots."""
    torch = _torch()
    N, top_k = _choice(idx)
    need = eqtp_expert_plan_workspace_bytes(N, top_k, experts)
    slots = torch.empty(N * top_k, dtype=torch.int32, device=idx.device)
    order = slots if top_k == 1 else torch.empty(N, dtype=torch.int32, device=idx.device)
    ptr = torch.empty(experts + 1, dtype=torch.int32, device=idx.device)
    workspace = _workspace(workspace, need, idx.device)
    rc = load_library().eqtp_expert_plan(N, top_k, experts, _ptr(idx), None if top_k == 1 else _ptr(order), _ptr(slots),
                                         _ptr(ptr), _ptr(workspace), workspace.numel(), _stream())
    _raise(rc, "eqtp_expert_plan")
    return order, slots, ptr


@functools.lru_cache(maxsize=256)
def _expert_desc(lmax, C, experts, top_k, x_dtype, out_dtype):
    # read by the library during a call only, so one instance per distinct descriptor is shared
    d = _ExpertDesc(ctypes.sizeof(_ExpertDesc), lmax, C, experts, top_k, x_dtype, out_dtype)
    need = load_library().eqtp_expert_linear_backward_workspace_bytes(ctypes.byref(d), 0)  # checks the descriptor
    if need < 0:
        raise EqtpError(int(-need), "eqtp_expert_desc")
    return ctypes.byref(d), d


def _expert_args(h, W, idx, lmax, weight, plan, out_dtype):
    """Checks the tensors; returns (descriptor, N, order, slots, ptr)."""
    torch = _torch()
    code, N, C = _rows(h, "h", lmax)
    _check(W, "W", h.dtype)
    if W.dim() != 4 or W.shape[1:] != (lmax + 1, C, C):
        raise ValueError("W must be [experts, %d, %d, %d]" % (lmax + 1, C, C))
    X = W.shape[0]
    rows, top_k = _choice(idx)
    if rows != N:
        raise ValueError("idx has %d rows, h %d" % (rows, N))
    if weight is not None:
        _check(weight, "weight", torch.float32, (N, top_k))
    order = slots = ptr = None
    if plan is not None:
        order, slots, ptr = plan
        _check(order, "order", torch.int32, (N,))
        _check(slots, "slots", torch.int32, (N * top_k,))
        _check(ptr, "ptr", torch.int32, (X + 1,))
    ocode = code if out_dtype is None else out_dtype
    _torch_dtype(ocode)
    return _expert_desc(lmax, C, X, top_k, code, ocode)[0], N, order, slots, ptr


def eqtp_expert_linear(h, W, idx, lmax: int, weight=None, plan=None, out_dtype: int = None, out=None):
    """out [N, C, K]: per-degree channel linears by expert, each node's summed under ``weight`` (see include/eqtp.h).

    h [N, C, K], W [X, lmax+1, C, C] float32 or bfloat16 (C = 8, 16, 32, 64 or 128); ``idx`` [N, top_k] int32, outside
    [0, X) for none; ``weight`` [N, top_k] float32 or None (ones).  ``plan``: eqtp_expert_plan's result, which only
    makes it faster, or None.  ``out_dtype``: EQTP_F32 or EQTP_BF16 (h's by default)."""
    torch = _torch()
    d, N, order, _, _ = _expert_args(h, W, idx, lmax, weight, plan, out_dtype)
    odt = h.dtype if out_dtype is None else _torch_dtype(out_dtype)
    if out is None:
        out = torch.empty_like(h, dtype=odt)
    else:
        _check(out, "out", odt, h.shape)
    _raise(load_library().eqtp_expert_linear(d, N, _ptr(h), _ptr(W), _ptr(idx), _ptr(weight), _ptr(order), _ptr(out),
                                             _stream()), "eqtp_expert_linear")
    return out


def eqtp_expert_linear_backward_workspace_bytes(N: int, lmax: int, C: int, experts: int, top_k: int,
                                                x_dtype: int = EQTP_F32) -> int:
    """Device workspace eqtp_expert_linear_backward needs (bytes)."""
    n = load_library().eqtp_expert_linear_backward_workspace_bytes(
        _expert_desc(lmax, C, experts, top_k, x_dtype, x_dtype)[0], N)
    if n < 0:
        raise EqtpError(int(-n), "eqtp_expert_linear_backward_workspace_bytes")
    return int(n)


def eqtp_expert_linear_backward(h, W, idx, grad_out, lmax: int, weight=None, plan=None, need_h: bool = True,
                                need_W: bool = True, need_weight: bool = None, workspace=None):
    """(grad_h, grad_W float32, grad_weight) of eqtp_expert_linear, each None if not asked for; ``grad_out`` [N, C, K]
    in h's type.  ``need_weight`` defaults to whether a weight is given.  ``plan``: eqtp_expert_plan's result, made
    here if it is None and grad_W is asked for.  ``workspace``: a uint8 tensor of at least
    eqtp_expert_linear_backward_workspace_bytes bytes, or None to allocate one."""
    torch = _torch()
    if plan is None and need_W:
        plan = eqtp_expert_plan(idx, W.shape[0])
    d, N, order, slots, ptr = _expert_args(h, W, idx, lmax, weight, plan, None)
    _check(grad_out, "grad_out", h.dtype, h.shape)
    if need_weight is None:
        need_weight = weight is not None
    gh = torch.empty_like(h) if need_h else None
    gW = torch.empty(W.shape, dtype=torch.float32, device=h.device) if need_W else None
    gw = torch.empty(idx.shape, dtype=torch.float32, device=h.device) if need_weight else None
    lib = load_library()
    workspace = _workspace(workspace, lib.eqtp_expert_linear_backward_workspace_bytes(d, N), h.device)
    rc = lib.eqtp_expert_linear_backward(d, N, _ptr(h), _ptr(W), _ptr(idx), _ptr(weight), _ptr(order), _ptr(slots),
                                         _ptr(ptr), _ptr(grad_out), _ptr(gh), _ptr(gW), _ptr(gw), _ptr(workspace),
                                         workspace.numel(), _stream())
    _raise(rc, "eqtp_expert_linear_backward")
    return gh, gW, gw


def eqtp_test_segment_probe(row_ptr, src, C: int, lmax: int, algo: int = EQTP_ALGO_NODE_MFMA):
    """(count [N] int32, src_sum [N] int64) walked with the conv kernel's schedule."""
    import torch

    _check(row_ptr, "row_ptr", torch.int32)
    _check(src, "src", torch.int32)
    N = row_ptr.shape[0] - 1
    E = src.shape[0]
    count = torch.empty(N, dtype=torch.int32, device=row_ptr.device)
    src_sum = torch.empty(N, dtype=torch.int64, device=row_ptr.device)
    rc = load_library().eqtp_test_segment_probe(_ptr(row_ptr), _ptr(src), N, E, C, lmax, algo, _ptr(count),
                                                _ptr(src_sum), _stream())
    _raise(rc, "eqtp_test_segment_probe")
    return count, src_sum
