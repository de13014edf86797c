"""Workspace sizes of the attention, and what is refused with too little of
it: answered before any HIP call, so no GPU is needed."""
import ctypes

from test_abi_host import FAKE, NULL, _lib
from test_block_host import _attn_desc


def test_few_long_rows_need_a_workspace():
    e = _lib()
    lib = e.load_library()
    d = ctypes.byref(_attn_desc(e))
    need = lib.eqtp_attention_workspace_bytes(d, 1, 100000, 100000)
    assert need > 0
    call = lambda space, size: lib.eqtp_attention(d, 1, 100000, 100000, *[FAKE] * 8, space, size, NULL)
    assert call(NULL, need) == 1 and call(FAKE, need - 1) == 1
    assert call(ctypes.c_void_p(0x10008), need) == 1
    assert lib.eqtp_attention_workspace_bytes(d, 100000, 100000, 100000) == 0


def test_workspace_sizes():
    """Partial results of S pieces a row: D sums and two numbers for each head; backward two tables of E heads numbers
    and the larger of the rows' and the sources' partial results."""
    e = _lib()
    lib = e.load_library()
    H, G = 4, 2
    d = ctypes.byref(_attn_desc(e, lmax=0, C=64, heads=H, kv_heads=G))
    D = 16

    def pieces(rows, E):
        s = min(-(-2048 // rows), E // rows // 32, 1024) if 0 < rows < 2048 else 1
        return s if s >= 2 else 1

    for N, M, E in ((1, 5, 64), (1, 5, 63), (7, 50000, 50000), (2047, 3, 2047 * 64), (2048, 3, 1 << 20), (3, 7, 1 << 20),
                    (1, 1, (1 << 31) - 1)):
        S, Z = pieces(N, E), pieces(M, E)
        fwd = 4 * N * S * H * (D + 2) if S > 1 else 0
        rows = 4 * N * H * (S * (2 * D + 2) + 2) if S > 1 else 0
        sources = 4 * M * Z * G * 2 * D if Z > 1 else 0
        tables = (8 * E * H + 15) // 16 * 16
        assert lib.eqtp_attention_workspace_bytes(d, N, M, E) == fwd
        assert lib.eqtp_attention_backward_workspace_bytes(d, N, M, E) == tables + max(rows, sources)
