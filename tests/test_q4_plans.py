"""The sizes of the GPU tests reach every kernel of the 4-bit products that any sizes
reach, without a GPU: each streaming work-group's shape, and each tile with its sums
whole, split, and both."""

import ctypes
import random

import pytest

_lib = pytest.importorskip("newton_schulz_dmuon_amd")._lib
import test_gpu_q4 as q4  # noqa: E402
import test_gpu_q4_plans as more  # noqa: E402


@pytest.fixture(scope="module")
def kernel():
    """(bf16 rows, rows, outputs, columns) -> what runs."""
    fn = _lib.load().dmuon_q4_choice
    i64 = ctypes.c_int64
    fn.argtypes, fn.restype = [ctypes.c_int32, i64, i64, i64, ctypes.POINTER(i64)], ctypes.c_int
    choice = (i64 * 9)()

    def ask(bf16_rows, t, n, k):
        assert fn(bf16_rows, t, n, k, choice) == _lib.OK
        row_blocks, out_blocks, waves, rows, ta, tb, whole, tail, pieces = choice
        if row_blocks:
            assert ta == tb == whole == tail == pieces == 0
            return "streamed", row_blocks, out_blocks, waves, rows
        assert whole + tail == -(-n // ta) * -(-t // tb) and (tail > 0) == (pieces > 1)
        return "tiles", ta, tb, "whole" if pieces == 1 else "both" if whole else "split"

    return ask


@pytest.fixture(scope="module")
def reached(kernel):
    rng = random.Random(1)

    def size():
        return int(round(65536 ** rng.random()))

    sizes = [(size(), size(), size()) for _ in range(40000)]
    return [{kernel(bf16_rows, *s) for s in sizes} for bf16_rows in (0, 1)]


@pytest.mark.parametrize("bf16_rows", [0, 1])
def test_every_kernel_is_run(kernel, reached, bf16_rows):
    run = {kernel(bf16_rows, *s) for s in q4.EVERY_KERNEL + more.MORE_SIZES}
    assert len(reached[bf16_rows]) > 20 and not reached[bf16_rows] - run


def test_every_kernel_reads_rows_where_they_lie(kernel, reached):
    sizes = q4.CHUNK_SIZES + more.MORE_CHUNK_SIZES
    assert all(k % 8 == 0 for _, _, k in sizes)
    assert not reached[1] - {kernel(1, *s) for s in sizes}


def test_bad_sizes_are_refused(kernel):
    fn = _lib.load().dmuon_q4_choice
    for bf16_rows in (0, 1):
        assert fn(bf16_rows, 1, 0, 1, (ctypes.c_int64 * 9)()) == _lib.ERR_INVALID_ARG
