"""The fast-sums flag of the 8-bit product, without a GPU."""

import ctypes

import pytest

pytest.importorskip("newton_schulz_dmuon_amd")
from newton_schulz_dmuon_amd import _lib  # noqa: E402

A, B, C, D, E, W = (0x7F0000000000 + i * 0x100000000 for i in range(6))


@pytest.mark.parametrize("dt,rows,want", [
    (_lib.BF16 | _lib.Q8_FAST_SUMS, 0, _lib.OK), (_lib.F32 | _lib.Q8_FAST_SUMS, 8, _lib.ERR_UNSUPPORTED_DTYPE),
    (2 | _lib.Q8_FAST_SUMS, 8, _lib.ERR_UNSUPPORTED_DTYPE), (1 << 9, 8, _lib.ERR_UNSUPPORTED_DTYPE),
    (-1, 8, _lib.ERR_UNSUPPORTED_DTYPE)])
def test_out_dtype(dt, rows, want):
    lib = _lib.load()
    assert lib.dmuon_q8_matmul(A, B, rows, C, D, 256, 512, E, dt, W, 1 << 40, None) == want
    size = ctypes.c_size_t(7)
    assert lib.dmuon_q8_matmul_workspace_bytes(rows, 256, 512, dt, ctypes.byref(size)) == want
    if want == _lib.OK:
        assert size.value == 0


def test_the_sizes_bytes_are_checked_with_the_results_type():
    """A bf16 result with the flag is a bf16 result: out may end where the next
    buffer begins."""
    lib = _lib.load()
    out = W - 8 * 256 * 2
    dt = _lib.BF16 | _lib.Q8_FAST_SUMS
    assert lib.dmuon_q8_matmul(A, B, 8, W, D, 256, 512, out + 16, dt, None, 0, None) == _lib.ERR_ALIAS
    assert lib.dmuon_q8_matmul(A, B, 8, W, D, 256, 512, out + 8, dt, None, 0, None) == _lib.ERR_MISALIGNED


@pytest.mark.parametrize("t,n,k", [(1, 4096, 4096), (300, 512, 2048), (2048, 4096, 8192), (8192, 14336, 4096)])
def test_workspace_bytes(t, n, k):
    lib = _lib.load()
    for dt in (_lib.BF16, _lib.F32, _lib.BF16 | _lib.Q8_FAST_SUMS):
        size = ctypes.c_size_t(7)
        assert lib.dmuon_q8_matmul_workspace_bytes(t, n, k, dt, ctypes.byref(size)) == _lib.OK
        assert size.value % 256 == 0
    exact = [ctypes.c_size_t(0) for _ in range(2)]
    for dt, out in zip((_lib.BF16, _lib.F32), exact):
        lib.dmuon_q8_matmul_workspace_bytes(t, n, k, dt, ctypes.byref(out))
    assert exact[0].value == exact[1].value  # the same sums, the same plan
