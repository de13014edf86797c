"""The attention binding without a GPU: what reaches the library is recorded
by a stand-in, so ways to call it can be compared argument by argument."""
import pytest

from test_abi_host import _lib


class _Recorder:
    """Answers size queries with 0 and keeps the arguments of the calls."""

    def __init__(self, lib):
        self._lib, self.calls, self.scales = lib, [], []

    def eqtp_attention_workspace_bytes(self, *a):
        return self._lib.eqtp_attention_workspace_bytes(*a)

    def eqtp_attention_backward_workspace_bytes(self, *a):
        return 0

    def eqtp_attention(self, d, *a):
        self.scales.append(d._obj.scale)
        return 0

    def eqtp_attention_backward(self, d, *a):
        # the addresses of the results differ from call to call: whether there is one
        self.calls.append((d._obj.scale,) + a[:14] + tuple(p is not None for p in a[14:18]) + a[18:])
        return 0


@pytest.fixture
def recorded(monkeypatch):
    import torch

    e = _lib()
    rec = _Recorder(e.load_library())
    monkeypatch.setattr(e, "load_library", lambda: rec)
    monkeypatch.setattr(e, "_stream", lambda: 0)

    def check(t, name, dtype, shape=None):  # as the binding's own, but for the device
        if not isinstance(t, torch.Tensor) or t.dtype != dtype or (shape is not None and tuple(t.shape) != tuple(shape)):
            raise ValueError("%s is not as it should be" % name)

    monkeypatch.setattr(e, "_check", check)
    e._attention_desc.cache_clear()
    yield e, rec
    e._attention_desc.cache_clear()


def _tensors():
    import torch

    N, M, E, heads, C, K = 3, 5, 7, 2, 8, 4
    f = lambda *s: torch.zeros(s)
    i = lambda n: torch.zeros(n, dtype=torch.int32)
    return dict(q=f(N, C, K), k=f(M, C, K), v=f(M, C, K), src=i(E), row_ptr=i(N + 1), out=f(N, C, K), lse=f(N, heads),
                grad_out=f(N, C, K), src_ptr=i(M + 1), dst_s=i(E), perm=i(E), bias=f(E, heads))


def test_attention_backward_takes_the_output_before_lse(recorded):
    """(.., row_ptr, out, lse, ..) and (.., row_ptr, lse, ..) are the same call."""
    e, rec = recorded
    t = _tensors()
    head = [t[n] for n in ("q", "k", "v", "src", "row_ptr")]
    tail = [t[n] for n in ("lse", "grad_out", "src_ptr", "dst_s", "perm")] + [1, 2]
    e.eqtp_attention_backward(*head, *tail, bias=t["bias"])
    e.eqtp_attention_backward(*head, t["out"], *tail, bias=t["bias"])
    e.eqtp_attention_backward(*head, *tail, bias=t["bias"], out=t["out"])
    e.eqtp_attention_backward(*head, t["out"], *tail[:5], lmax=1, heads=2, bias=t["bias"])
    assert len(rec.calls) == 4 and all(c == rec.calls[0] for c in rec.calls[1:])
    # without the grouping by source, where the place of perm holds None
    none = [t["lse"], t["grad_out"], None, None, None, 1, 2, 0.5, t["bias"], True, False, False, True]
    e.eqtp_attention_backward(*head, *none)
    e.eqtp_attention_backward(*head, t["out"], *none)
    assert rec.calls[4] == rec.calls[5] and rec.calls[4][0] == 0.5 and rec.calls[4] != rec.calls[0]


def test_attention_backward_checks_the_output(recorded):
    e, _ = recorded
    t = _tensors()
    rest = [t[n] for n in ("lse", "grad_out", "src_ptr", "dst_s", "perm")] + [1, 2]
    head = [t[n] for n in ("q", "k", "v", "src", "row_ptr")]
    with pytest.raises(ValueError, match="out"):
        e.eqtp_attention_backward(*head, t["out"][:2], *rest)
    with pytest.raises(ValueError, match="out"):
        e.eqtp_attention_backward(*head, t["out"].double(), *rest)
    with pytest.raises(TypeError):  # given twice
        e.eqtp_attention_backward(*head, t["out"], *rest, out=t["out"])


def test_attention_scale_is_taken_by_value(recorded):
    """A scale held in a tensor (a learned one) counts as it is at the call, not as it was at an earlier one."""
    import numpy as np
    import torch

    e, rec = recorded
    t = _tensors()
    head = [t[n] for n in ("q", "k", "v", "src", "row_ptr")]
    back = [t[n] for n in ("lse", "grad_out", "src_ptr", "dst_s", "perm")] + [1, 2]
    s = torch.tensor(0.5)
    for value in (0.5, 0.25, -2.0):
        s.fill_(value)
        e.eqtp_attention(*head, 1, 2, scale=s)
        e.eqtp_attention_backward(*head, *back, scale=s)
        assert rec.scales[-1] == value and rec.calls[-1][0] == value
    a = np.array(0.125)  # not hashable
    e.eqtp_attention(*head, 1, 2, scale=a)
    assert rec.scales[-1] == 0.125
    e.eqtp_attention(*head, 1, 2)
    assert rec.scales[-1] == 0.25  # 1 / sqrt(4 channels of 4 components)
