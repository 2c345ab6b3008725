"""Refusals of the 4-bit block products, without a GPU: every argument error is
reported before any HIP call (fake device pointers are never dereferenced), and
the binding refuses tensors the kernels could not read."""

import ctypes

import pytest
import torch

nsd = pytest.importorskip("newton_schulz_dmuon_amd")
from newton_schulz_dmuon_amd import _lib  # noqa: E402

A, B, C, D, E, F, W = (0x7F0000000000 + i * 0x100000000 for i in range(7))
BAD, DT, MIS, ALIAS = _lib.ERR_INVALID_ARG, _lib.ERR_UNSUPPORTED_DTYPE, _lib.ERR_MISALIGNED, _lib.ERR_ALIAS


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def source(**kw):
    d = dict(x=A, dtype=_lib.BF16, reserved=0, rows=64, cols=256, random=None, codes=B, scales=C, codes_t=D, scales_t=E)
    d.update(kw)
    return _lib.Q4SourceDesc(*[d[n] for n, _ in _lib.Q4SourceDesc._fields_])


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=7), DT), (dict(rows=-1), BAD), (dict(rows=(1 << 22) + 1, cols=1), BAD),
    (dict(rows=(1 << 29) + 1, cols=1, codes_t=None, scales_t=None), BAD), (dict(cols=0), BAD),
    (dict(cols=(1 << 22) + 1), BAD), (dict(rows=1 << 22, cols=(1 << 15) + 1), BAD), (dict(reserved=1), BAD),
    (dict(x=None), BAD), (dict(codes=None), BAD), (dict(scales=None), BAD), (dict(codes_t=None), BAD),
    (dict(scales_t=None), BAD), (dict(codes=None, scales=None, codes_t=None, scales_t=None), BAD),
    (dict(x=A + 8), MIS), (dict(codes=B + 8), MIS), (dict(scales=C + 4), MIS), (dict(codes_t=D + 8), MIS),
    (dict(scales_t=E + 8), MIS), (dict(random=F + 8), MIS), (dict(codes=A), ALIAS), (dict(codes_t=B + 16), ALIAS),
    (dict(scales=B + 64 * 128 - 16), ALIAS), (dict(random=B), ALIAS), (dict(random=C), ALIAS),
    (dict(rows=0), _lib.OK), (dict(rows=0, x=None, codes=None, scales=None), _lib.OK)])
def test_quantize_refusals(lib, kw, want):
    arr = (_lib.Q4SourceDesc * 1)(source(**kw))
    assert lib.dmuon_q4_quantize(arr, 1, None) == want
    assert want == _lib.OK or lib.dmuon_last_error()


def test_quantize_counts(lib):
    assert lib.dmuon_q4_quantize(None, 0, None) == _lib.OK
    assert lib.dmuon_q4_quantize(None, 1, None) == BAD
    assert lib.dmuon_q4_quantize(None, -1, None) == BAD
    two = (_lib.Q4SourceDesc * 2)(source(), source())  # the second writes the first's results
    assert lib.dmuon_q4_quantize(two, 2, None) == ALIAS
    assert ctypes.sizeof(_lib.Q4SourceDesc) == 72


def dequantize(lib, codes=A, scales=B, rows=4, cols=256, out=C, dt=_lib.BF16):
    return lib.dmuon_q4_dequantize(codes, scales, rows, cols, out, dt, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=2), DT), (dict(rows=-1), BAD), (dict(cols=0), BAD), (dict(cols=(1 << 22) + 1), BAD),
    (dict(rows=(1 << 29) + 1, cols=1), BAD), (dict(rows=1 << 29, cols=257), BAD), (dict(codes=None), BAD),
    (dict(scales=None), BAD), (dict(out=None), BAD), (dict(codes=A + 8), MIS), (dict(scales=B + 8), MIS),
    (dict(out=C + 2), MIS), (dict(out=A), ALIAS), (dict(out=B + 16), ALIAS), (dict(rows=0, codes=None), _lib.OK)])
def test_dequantize_refusals(lib, kw, want):
    assert dequantize(lib, **kw) == want


def matmul(lib, codes=A, scales=B, rows=8, codes_b=C, scales_b=D, outs=256, inner=512, base=None, out=E, dt=_lib.BF16,
           ws=W, nws=1 << 40):
    return lib.dmuon_q4_matmul(codes, scales, rows, codes_b, scales_b, outs, inner, base, out, dt, ws, nws, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=2), DT), (dict(dt=_lib.BF16 | _lib.Q8_FAST_SUMS), DT), (dict(rows=-1), BAD), (dict(outs=0), BAD),
    (dict(inner=-1), BAD), (dict(outs=(1 << 22) + 1), BAD), (dict(inner=1 << 23), BAD),
    (dict(rows=1 << 24, outs=1 << 20), BAD), (dict(rows=(1 << 29) + 1, outs=1, inner=1), BAD), (dict(codes=None), BAD),
    (dict(scales=None), BAD), (dict(codes_b=None), BAD), (dict(scales_b=None), BAD), (dict(out=None), BAD),
    (dict(codes=A + 1), MIS), (dict(codes_b=C + 8), MIS), (dict(scales=B + 4), MIS), (dict(scales_b=D + 2), MIS),
    (dict(out=E + 2), MIS), (dict(base=F + 2), MIS), (dict(out=A), ALIAS), (dict(out=C + 512), ALIAS), (dict(out=B), ALIAS),
    (dict(base=E + 16), ALIAS), (dict(base=E - 16), ALIAS), (dict(rows=0), _lib.OK),
    (dict(rows=0, codes=None, out=None), _lib.OK), (dict(inner=0, codes=None, out=None), BAD)])
def test_matmul_refusals(lib, kw, want):
    assert matmul(lib, **kw) == want


def rows_matmul(lib, x=A, rows=8, codes_b=C, scales_b=D, outs=256, inner=512, out=E, dt=_lib.BF16, ws=W, nws=1 << 40):
    return lib.dmuon_q4_rows_matmul(x, rows, codes_b, scales_b, outs, inner, out, dt, ws, nws, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=2), DT), (dict(rows=-1), BAD), (dict(outs=0), BAD), (dict(inner=0), BAD), (dict(inner=1 << 23), BAD),
    (dict(rows=1 << 24, outs=1 << 20), BAD), (dict(x=None), BAD), (dict(codes_b=None), BAD), (dict(scales_b=None), BAD),
    (dict(out=None), BAD), (dict(x=A + 2), MIS), (dict(codes_b=C + 8), MIS), (dict(scales_b=D + 2), MIS),
    (dict(out=E + 2), MIS), (dict(out=A), ALIAS), (dict(out=C + 512), ALIAS), (dict(rows=0, x=None), _lib.OK)])
def test_rows_matmul_refusals(lib, kw, want):
    assert rows_matmul(lib, **kw) == want


@pytest.mark.parametrize("call", ["dmuon_q4_matmul", "dmuon_q4_rows_matmul"])
def test_workspaces(lib, call):
    """Sizes are bounded, and a workspace that is too small, misaligned or
    overlapping is refused."""
    fn = getattr(lib, call + "_workspace_bytes")
    out = ctypes.c_size_t(7)
    ref = ctypes.byref(out)
    assert fn(16, 256, 256, None) == BAD
    assert fn(-1, 256, 256, ref) == BAD and fn(16, 0, 256, ref) == BAD and fn(16, 256, -1, ref) == BAD
    assert fn(1 << 29, 256, 256, ref) == _lib.OK
    assert fn((1 << 29) + 1, 1, 1, ref) == BAD and fn(1 << 29, 257, 1, ref) == BAD
    assert fn(1, 1 << 22, (1 << 15) + 1, ref) == BAD
    run = matmul if call == "dmuon_q4_matmul" else rows_matmul
    tried = 0
    for t in (0, 1, 16, 17, 100, 1000, 8192, 100_000):
        for n, k in ((1, 1), (128, 128), (1024, 4096), (14336, 4096), (1001, 513), (300, 100_000)):
            assert fn(t, n, k, ref) == _lib.OK
            # at most 16 pieces of fewer tiles than fill the chip, and a padded copy of bf16 rows
            assert out.value % 256 == 0 and out.value <= 16 * 512 * 128 * 128 * 4 + 2 * t * (k + 256)
            if out.value:
                tried += 1
                sizes = dict(rows=t, outs=n, inner=k, nws=out.value)
                assert run(lib, **dict(sizes, nws=out.value - 1)) == _lib.ERR_WORKSPACE_TOO_SMALL
                assert run(lib, **dict(sizes, ws=W + 16)) == MIS
                assert run(lib, **dict(sizes, ws=None)) == BAD
                assert run(lib, **dict(sizes, ws=E)) == ALIAS


def status(fn, *a, **kw):
    with pytest.raises(nsd.DmuonError) as e:
        fn(*a, **kw)
    return e.value.status


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    q, w = nsd.Q4Matrix.empty(4, 256, "cpu"), nsd.Q4Matrix.empty(128, 256, "cpu")
    assert status(nsd.q4_quantize, x) == BAD
    assert status(nsd.q4_quantize_weights, [x]) == BAD
    assert status(nsd.q4_dequantize, q) == BAD
    assert status(nsd.q4_matmul, q, w) == BAD and status(nsd.q4_matmul, x, w) == BAD
    assert status(nsd.q4_weight_grad, q, q) == BAD


def test_binding_refuses_a_missing_form():
    q = nsd.Q4Matrix.empty(4, 256, "cpu", transposed=False)
    t = nsd.Q4Matrix.empty(4, 256, "cpu", plain=False)
    for fn, args, kw in ((nsd.q4_dequantize, (t,), {}), (nsd.q4_dequantize, (q,), dict(transpose=True)),
                         (nsd.q4_matmul, (q, t), {}), (nsd.q4_matmul, (q, q), dict(transpose=True)),
                         (nsd.q4_weight_grad, (q, t), {}), (nsd.q4_weight_grad, (t, q), {})):
        with pytest.raises(nsd.DmuonError, match="GPU|no codes|no transposed codes"):
            fn(*args, **kw)


def test_binding_shapes():
    q = nsd.Q4Matrix.empty(5, 130, "cpu")
    assert q.codes.shape == (5, 128) and q.scales.shape == (8, 16)
    assert q.codes_t.shape == (130, 128) and q.scales_t.shape == (8, 144)
    assert q.nbytes() == 5 * 128 + 8 * 16 + 130 * 128 + 8 * 144
    assert nsd.Q4Matrix.empty(130, 300, "cpu", transposed=False).codes_t is None
    assert nsd.Q4Matrix.empty(130, 300, "cpu", plain=False).nbytes() == 300 * 128 + 8 * 304
    assert nsd.q4_quantize_weights([]) == []


def tracked(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16, requires_grad=True)


CALLS = [lambda x: nsd.q4_quantize(x), lambda x: nsd.q4_quantize(x * 2),
         lambda x: nsd.q4_quantize_weights([x * 2]), lambda x: nsd.q4_quantize_weights([x.detach(), x * 2])]


@pytest.mark.parametrize("call", CALLS)
def test_tracked_inputs_are_refused(call):
    x = tracked(4, 256)
    with pytest.raises(nsd.DmuonError, match="gradient"):
        call(x)
    with torch.no_grad(), pytest.raises(nsd.DmuonError, match="GPU"):
        call(x)


def test_a_parameter_may_be_quantised():
    with pytest.raises(nsd.DmuonError, match="GPU"):
        nsd.q4_quantize_weights([torch.nn.Parameter(torch.zeros(128, 256))])


def test_rows_of_whole_chunks_need_no_copy(lib):
    """A workspace holds a padded copy of bf16 rows only where 16-byte chunks do not
    make up a row."""
    out = ctypes.c_size_t(7)
    for k in (8, 24, 72, 1000, 1416):
        assert lib.dmuon_q4_rows_matmul_workspace_bytes(4, 256, k, ctypes.byref(out)) == _lib.OK and out.value == 0
        assert lib.dmuon_q4_rows_matmul_workspace_bytes(4, 256, k + 1, ctypes.byref(out)) == _lib.OK
        assert out.value == (4 * (k + 8) * 2 + 255) // 256 * 256
