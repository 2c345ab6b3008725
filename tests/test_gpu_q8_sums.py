"""How a product of 8-bit operands sums: in fp32 unless the caller asks for fast
sums, whose error the bound of test_gpu_q8 (CUT) covers."""

import numpy as np
import pytest
import torch

import newton_schulz_dmuon_amd as nsd
from newton_schulz_dmuon_amd import _lib
from test_gpu_q8 import (BF16, CUT, F32, PRODUCT_SIZES, check_sum, host, layer_inputs, ref, rows_of, status,
                         weight_of)

pytestmark = pytest.mark.gpu

# (the streaming kernel's work-groups with a ring that turns several times, and
# every tile shape, whole and split)
MORE_SIZES = [(16, 1000, 3900), (7, 300, 8200), (1, 5001, 4301), (39, 2767, 4301), (45, 4239, 4301), (1505, 2801, 131),
              (1500, 1000, 9001), (2230, 3602, 903), (2309, 3424, 133)]


def operands_that_cancel(t, n, k):
    """Rows and weights of +-256 in about one place of eight, +-1 and +-3
    elsewhere, in blocks of scale 1: every product is an integer, and so is every
    sum, below 2^24 (asserted), so fp32 sums are exact in any order.  Next to a
    product of 2^16 the 8-bit instruction drops products below 2^3."""
    rng = np.random.default_rng(t * 3 + n * 5 + k * 7)
    kp, kb, t4, nb = ref.up(k, 128), ref.up(k, 128) // 128, ref.up(t, 4), ref.up(n, 128) // 128

    def draw(rows):
        v = rng.choice([-3.0, -1.0, 1.0, 3.0], (rows, kp))
        v = np.where(rng.random((rows, kp)) < 0.125, 256.0 * np.sign(v), v)
        v[:, k:] = 0
        return v

    a, b = draw(t), draw(n)
    want, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    assert mag.max() < 2.0 ** 24
    f8 = lambda v: torch.from_numpy(v).float().to(torch.float8_e4m3fn).cuda()  # noqa: E731
    one = lambda *s: torch.full(s, 127, dtype=torch.uint8, device="cuda")  # noqa: E731
    return nsd.Q8Rows(f8(a), one(kb, t4), k), nsd.Q8Weight(f8(b), one(nb, kb), None, None, n, k), want, mag


@pytest.mark.parametrize("t,n,k", PRODUCT_SIZES + MORE_SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sums_are_fp32(t, n, k, dtype):
    """The result is the exact sum, rounded once, where large products cancel."""
    print(f"fp32 sums {t} {n} {k} {dtype}", flush=True)
    a, w, want, _ = operands_that_cancel(t, n, k)
    got = host(nsd.q8_matmul(a, w, dtype=dtype))
    want = torch.from_numpy(want).to(dtype).double().numpy()
    assert np.array_equal(got, want), (np.argwhere(got != want)[:4], got[got != want][:4], want[got != want][:4])


@pytest.mark.parametrize("t,n,k", PRODUCT_SIZES + MORE_SIZES)
@pytest.mark.parametrize("transpose", [False, True])
def test_fast_sums(t, n, k, transpose):
    print(f"fast sums {t} {n} {k} {transpose}", flush=True)
    a, w, want, mag = operands_that_cancel(t, n, k)
    if transpose:
        w = nsd.Q8Weight(w.codes, w.scales, w.codes, w.scales, k, n)
    got = nsd.q8_matmul(a, w, transpose=transpose, fast_sums=True)
    check_sum(got, want, mag, k, (t, n, k, transpose), CUT)


@pytest.mark.parametrize("t,n,k", [(1, 1001, 513), (33, 300, 640), (257, 520, 1030), (1100, 1500, 700), (60, 8200, 260)])
def test_fast_sums_of_quantised_values(t, n, k):
    """Over scales that differ from block to block, and at both ends of their
    range."""
    print(f"fast sums of values {t} {n} {k}", flush=True)
    rng = np.random.default_rng(t)
    w, wv = weight_of(rng, n, k)
    a, av = rows_of(rng, t, k)
    check_sum(nsd.q8_matmul(a, w, fast_sums=True), *ref.matmul(av, wv), k, (t, n, k), CUT)
    x = rng.standard_normal((t, k)).astype(np.float32)
    x[:, :128] *= 2.0 ** -110
    x[:, 128:] = np.finfo(np.float32).min * np.sign(x[:, 128:])
    v = rng.standard_normal((n, k)).astype(np.float32)
    v[:, :128] *= 2.0 ** 100
    v[:, 128:] *= 2.0 ** -100
    xv = ref.row_values(*ref.quantize_rows(x.astype(np.float64)))[:, :k]
    vv = ref.weight_values(*ref.quantize_weight(v.astype(np.float64))[:2])[:, :k]
    q, p = nsd.q8_quantize(torch.from_numpy(x).cuda()), nsd.q8_quantize_weights([torch.from_numpy(v).cuda()])[0]
    check_sum(nsd.q8_matmul(q, p, fast_sums=True), *ref.matmul(xv, vv), k, "range", CUT)


@pytest.mark.parametrize("t", [1, 40, 300, 2048])
def test_fast_sums_in_a_graph(t):
    print(f"fast sums in a graph {t}", flush=True)
    x, _, w, _ = layer_inputs(3, t)
    ws, eager = nsd.Workspace(), nsd.Workspace()

    def product(x, w, ws):
        return nsd.q8_matmul(nsd.q8_quantize(x), nsd.q8_quantize_weights([w])[0], workspace=ws, fast_sums=True)

    product(x, w, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = product(x, w, ws)
    for i in range(3):
        nx, _, nw, _ = layer_inputs(30 + i, t)
        x.copy_(nx)
        w.copy_(nw)
        graph.replay()
        want = product(nx, nw, eager)
        torch.cuda.synchronize()
        assert torch.equal(y, want), i


def test_fast_sums_of_an_fp32_result_are_refused():
    print("fast sums refused", flush=True)
    a, w, _, _ = operands_that_cancel(8, 128, 128)
    assert status(nsd.q8_matmul, a, w, dtype=F32, fast_sums=True) == _lib.ERR_UNSUPPORTED_DTYPE
    out = torch.zeros(8, 128, device="cuda")
    assert status(nsd.q8_matmul, a, w, out=out, fast_sums=True) == _lib.ERR_UNSUPPORTED_DTYPE
