"""Refusals of the 8-bit block products, without a GPU: every argument error
is reported before any HIP call (fake device pointers are never dereferenced),
and the binding refuses tensors the kernels could not read."""

import ctypes

import pytest
import torch

nsd = pytest.importorskip("newton_schulz_dmuon_amd")
from newton_schulz_dmuon_amd import _lib  # noqa: E402

A, B, C, D, E, W = (0x7F0000000000 + i * 0x100000000 for i in range(6))


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def quantize(lib, x=A, dt=_lib.BF16, rows=4, cols=256, codes=B, scales=C):
    return lib.dmuon_q8_quantize(x, dt, rows, cols, codes, scales, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=7), _lib.ERR_UNSUPPORTED_DTYPE), (dict(rows=-1), _lib.ERR_INVALID_ARG),
    (dict(cols=0), _lib.ERR_INVALID_ARG), (dict(cols=(1 << 22) + 1), _lib.ERR_INVALID_ARG),
    (dict(rows=1 << 31), _lib.ERR_INVALID_ARG), (dict(rows=1 << 30, cols=1 << 20), _lib.ERR_INVALID_ARG),
    (dict(x=None), _lib.ERR_INVALID_ARG), (dict(codes=None), _lib.ERR_INVALID_ARG),
    (dict(scales=None), _lib.ERR_INVALID_ARG), (dict(x=A + 8), _lib.ERR_MISALIGNED),
    (dict(codes=B + 4), _lib.ERR_MISALIGNED), (dict(scales=C + 1), _lib.ERR_MISALIGNED),
    (dict(codes=A + 16), _lib.ERR_ALIAS), (dict(scales=B + 1020), _lib.ERR_ALIAS),
    (dict(rows=0), _lib.OK)])
def test_quantize_refusals(lib, kw, want):
    assert quantize(lib, **kw) == want
    assert want == _lib.OK or lib.dmuon_last_error()


def weight(**kw):
    d = dict(param=A, param_dtype=_lib.BF16, reserved=0, rows=256, cols=128, codes=B, scales=C, codes_t=D,
             scales_t=E)
    d.update(kw)
    return _lib.Q8WeightDesc(*[d[n] for n, _ in _lib.Q8WeightDesc._fields_])


@pytest.mark.parametrize("kw,want", [
    (dict(param=None), _lib.ERR_INVALID_ARG), (dict(rows=0), _lib.ERR_INVALID_ARG),
    (dict(cols=(1 << 22) + 1), _lib.ERR_INVALID_ARG), (dict(reserved=1), _lib.ERR_INVALID_ARG),
    (dict(param_dtype=3), _lib.ERR_UNSUPPORTED_DTYPE), (dict(codes_t=None), _lib.ERR_INVALID_ARG),
    (dict(scales_t=None), _lib.ERR_INVALID_ARG), (dict(codes=B + 8), _lib.ERR_MISALIGNED),
    (dict(scales=C + 2), _lib.ERR_MISALIGNED), (dict(codes_t=B), _lib.ERR_ALIAS),
    (dict(codes=A), _lib.ERR_ALIAS)])
def test_quantize_weights_refusals(lib, kw, want):
    arr = (_lib.Q8WeightDesc * 1)(weight(**kw))
    assert lib.dmuon_q8_quantize_weights(arr, 1, None) == want


def test_quantize_weights_counts(lib):
    assert lib.dmuon_q8_quantize_weights(None, 0, None) == _lib.OK
    assert lib.dmuon_q8_quantize_weights(None, 1, None) == _lib.ERR_INVALID_ARG
    assert lib.dmuon_q8_quantize_weights(None, -1, None) == _lib.ERR_INVALID_ARG
    two = (_lib.Q8WeightDesc * 2)(weight(), weight())  # the second writes the first's results
    assert lib.dmuon_q8_quantize_weights(two, 2, None) == _lib.ERR_ALIAS
    assert ctypes.sizeof(_lib.Q8WeightDesc) == 64


def matmul(lib, codes=A, scales=B, rows=8, codes_b=C, scales_b=D, outs=256, inner=512, out=E, dt=_lib.BF16, ws=W,
           nws=1 << 40):
    return lib.dmuon_q8_matmul(codes, scales, rows, codes_b, scales_b, outs, inner, out, dt, ws, nws, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=2), _lib.ERR_UNSUPPORTED_DTYPE), (dict(rows=-1), _lib.ERR_INVALID_ARG),
    (dict(outs=0), _lib.ERR_INVALID_ARG), (dict(inner=0), _lib.ERR_INVALID_ARG),
    (dict(outs=(1 << 22) + 1), _lib.ERR_INVALID_ARG), (dict(inner=1 << 23), _lib.ERR_INVALID_ARG),
    (dict(rows=1 << 24, outs=1 << 20), _lib.ERR_INVALID_ARG), (dict(codes=None), _lib.ERR_INVALID_ARG),
    (dict(scales=None), _lib.ERR_INVALID_ARG), (dict(codes_b=None), _lib.ERR_INVALID_ARG),
    (dict(scales_b=None), _lib.ERR_INVALID_ARG), (dict(out=None), _lib.ERR_INVALID_ARG),
    (dict(codes=A + 1), _lib.ERR_MISALIGNED), (dict(codes_b=C + 8), _lib.ERR_MISALIGNED),
    (dict(scales=B + 2), _lib.ERR_MISALIGNED), (dict(scales_b=D + 2), _lib.ERR_MISALIGNED),
    (dict(out=E + 2), _lib.ERR_MISALIGNED), (dict(out=A), _lib.ERR_ALIAS), (dict(out=C + 512), _lib.ERR_ALIAS),
    (dict(out=B), _lib.ERR_ALIAS), (dict(rows=0), _lib.OK), (dict(rows=0, codes=None, out=None), _lib.OK)])
def test_matmul_refusals(lib, kw, want):
    assert matmul(lib, **kw) == want


def wgrad(lib, dy=A, codes=B, scales=C, rows=64, outs=256, cols=512, base=None, out=E, dt=_lib.BF16, ws=W,
          nws=1 << 40):
    return lib.dmuon_q8_weight_grad(dy, codes, scales, rows, outs, cols, base, out, dt, ws, nws, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=2), _lib.ERR_UNSUPPORTED_DTYPE), (dict(rows=-1), _lib.ERR_INVALID_ARG),
    (dict(outs=0), _lib.ERR_INVALID_ARG), (dict(cols=0), _lib.ERR_INVALID_ARG),
    (dict(dy=None), _lib.ERR_INVALID_ARG), (dict(codes=None), _lib.ERR_INVALID_ARG),
    (dict(scales=None), _lib.ERR_INVALID_ARG), (dict(out=None), _lib.ERR_INVALID_ARG),
    (dict(dy=A + 2), _lib.ERR_MISALIGNED), (dict(codes=B + 8), _lib.ERR_MISALIGNED),
    (dict(scales=C + 2), _lib.ERR_MISALIGNED), (dict(out=E + 2), _lib.ERR_MISALIGNED),
    (dict(base=D + 2), _lib.ERR_MISALIGNED), (dict(out=A), _lib.ERR_ALIAS), (dict(out=B), _lib.ERR_ALIAS),
    (dict(base=E + 16), _lib.ERR_ALIAS), (dict(base=E - 16), _lib.ERR_ALIAS)])
def test_weight_grad_refusals(lib, kw, want):
    assert wgrad(lib, **kw) == want


@pytest.mark.parametrize("call,extra", [("dmuon_q8_matmul_workspace_bytes", (_lib.BF16,)),
                                        ("dmuon_q8_matmul_workspace_bytes", (_lib.F32,)),
                                        ("dmuon_q8_weight_grad_workspace_bytes", ())])
def test_workspace_bytes(lib, call, extra):
    fn = getattr(lib, call)
    out = ctypes.c_size_t(7)
    ref = ctypes.byref(out)
    assert fn(16, 256, 256, *extra, None) == _lib.ERR_INVALID_ARG
    assert fn(-1, 256, 256, *extra, ref) == _lib.ERR_INVALID_ARG
    assert fn(16, 0, 256, *extra, ref) == _lib.ERR_INVALID_ARG
    assert fn(16, 256, 0, *extra, ref) == _lib.ERR_INVALID_ARG
    for t in (0, 1, 16, 17, 100, 1000, 8192, 100_000):
        for n, k in ((1, 1), (128, 128), (1024, 4096), (14336, 4096), (1001, 513)):
            assert fn(t, n, k, *extra, ref) == _lib.OK
            # at most 16 pieces of fewer tiles than fill the chip, and a padded dy
            assert out.value % 256 == 0 and out.value <= (16 * 512 * 128 * 128 * 4) + 2 * t * (n + 263)


def status(fn, *a, **kw):
    with pytest.raises(nsd.DmuonError) as e:
        fn(*a, **kw)
    return e.value.status


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    q = nsd.Q8Rows.empty(4, 256, "cpu")
    w = nsd.Q8Weight.empty(128, 256, "cpu")
    assert status(nsd.q8_quantize, x) == _lib.ERR_INVALID_ARG
    assert status(nsd.q8_quantize_weights, [x]) == _lib.ERR_INVALID_ARG
    assert status(nsd.q8_matmul, q, w) == _lib.ERR_INVALID_ARG
    assert status(nsd.q8_weight_grad, x, q) == _lib.ERR_INVALID_ARG


def test_binding_shapes():
    q = nsd.Q8Rows.empty(5, 130, "cpu")
    assert q.codes.shape == (5, 256) and q.scales.shape == (2, 8) and q.nbytes() == 5 * 256 + 16
    w = nsd.Q8Weight.empty(130, 300, "cpu")
    assert w.codes.shape == (130, 384) and w.scales.shape == (2, 3)
    assert w.codes_t.shape == (300, 256) and w.scales_t.shape == (3, 2)
    assert nsd.Q8Weight.empty(130, 300, "cpu", transposed=False).codes_t is None
    assert nsd.q8_quantize_weights([]) == []


def test_size_limits(lib):
    """Sizes that a launch could not count are refused: rows beyond 2^29, and
    buffers of more than 2^37 elements."""
    ref = ctypes.byref(ctypes.c_size_t(0))
    assert quantize(lib, rows=(1 << 29) + 1, cols=1) == _lib.ERR_INVALID_ARG
    assert quantize(lib, rows=(1 << 27) + 1, cols=1000) == _lib.ERR_INVALID_ARG
    big = (_lib.Q8WeightDesc * 1)(weight(rows=1 << 22, cols=(1 << 15) + 1))
    assert lib.dmuon_q8_quantize_weights(big, 1, None) == _lib.ERR_INVALID_ARG
    for fn, extra in ((lib.dmuon_q8_matmul_workspace_bytes, (_lib.BF16,)),
                      (lib.dmuon_q8_weight_grad_workspace_bytes, ())):
        assert fn(1 << 29, 256, 256, *extra, ref) == _lib.OK
        assert fn((1 << 29) + 1, 1, 1, *extra, ref) == _lib.ERR_INVALID_ARG
        assert fn(1 << 29, 257, 1, *extra, ref) == _lib.ERR_INVALID_ARG
        assert fn(1, 1 << 22, (1 << 15) + 1, *extra, ref) == _lib.ERR_INVALID_ARG
