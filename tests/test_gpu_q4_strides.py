"""Codes and scales that lie otherwise than the format says: every call that reads
them gives, bit for bit, what it gives on their contiguous copies."""

import numpy as np
import pytest
import torch

import newton_schulz_dmuon_amd as nsd
from test_gpu_q4 import BF16, F32, values

pytestmark = pytest.mark.gpu


def transposed(t):
    return t.t().contiguous().t()


def rows_of_a_wider_buffer(t):
    wide = torch.full((t.shape[0], t.shape[1] + 40), 0x77, dtype=t.dtype, device=t.device)
    wide[:, 16:16 + t.shape[1]] = t
    return wide[:, 16:16 + t.shape[1]]


def every_second_row(t):
    wide = torch.full((2 * t.shape[0], t.shape[1]), 0x77, dtype=t.dtype, device=t.device)
    wide[::2] = t
    return wide[::2]


def every_second_column(t):
    wide = torch.full((t.shape[0], 2 * t.shape[1]), 0x77, dtype=t.dtype, device=t.device)
    wide[:, ::2] = t
    return wide[:, ::2]


def transposed_at_an_odd_place(t):
    """Columns an odd number of bytes apart, the first at an odd address."""
    step = t.shape[0] | 1
    raw = torch.full((1 + t.shape[1] * step,), 0x77, dtype=t.dtype, device=t.device)
    view = raw[1:].view(t.shape[1], step)[:, :t.shape[0]]
    view.copy_(t.t())
    return view.t()


LAYOUTS = [transposed, rows_of_a_wider_buffer, every_second_row, every_second_column, transposed_at_an_odd_place]


def laid_out(q, layout):
    return nsd.Q4Matrix(q.rows, q.cols, *(layout(t) for t in q.tensors()))


def calls(x, w, d, rows, base, **kw):
    """Every call that reads codes."""
    return [nsd.q4_matmul(x, w, dtype=F32, **kw), nsd.q4_matmul(d, w, transpose=True, dtype=BF16, **kw),
            nsd.q4_matmul(rows, w, dtype=F32, **kw), nsd.q4_weight_grad(d, x, base=base, **kw),
            nsd.q4_dequantize(w, **kw), nsd.q4_dequantize(x, transpose=True, dtype=F32, **kw)]


def operands(t, n, k, seed=0):
    rng = np.random.default_rng(t + 3 * n + 5 * k + seed)
    x, w, dy = (values(rng, *s, BF16).cuda() for s in ((t, k), (n, k), (t, n)))
    x4, d4 = nsd.q4_quantize(x, transposed=True), nsd.q4_quantize(dy, transposed=True)
    return x4, nsd.q4_quantize_weights([w])[0], d4, x, values(rng, n, k, F32).cuda()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("t,n,k", [(1, 1, 1), (1, 130, 257), (5, 256, 512), (33, 129, 1000), (130, 300, 260), (700, 515, 1030)])
def test_any_strides(layout, t, n, k):
    print(f"strides {layout.__name__} {t} {n} {k}", flush=True)
    x, w, d, rows, base = operands(t, n, k)
    want = calls(x, w, d, rows, base)
    x2, w2, d2 = (laid_out(q, layout) for q in (x, w, d))
    kept = [[v.clone() for v in q.tensors()] for q in (x2, w2, d2)]
    got = calls(x2, w2, d2, rows, base)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for q, c in zip((x2, w2, d2), kept) for a, b in zip(q.tensors(), c))


def test_broadcast_codes():
    """One row's codes for every row: a step of zero."""
    print("broadcast", flush=True)
    x, w = operands(1, 130, 300)[:2]
    q = nsd.Q4Matrix(70, 300, x.codes.expand(70, -1), x.scales[:, :1].expand(-1, 80))
    y = nsd.q4_matmul(q, w, dtype=F32)
    dense = nsd.q4_matmul(nsd.Q4Matrix(70, 300, *(v.contiguous() for v in q.tensors()[:2])), w, dtype=F32)
    torch.cuda.synchronize()
    assert torch.equal(y, dense) and torch.equal(y[0], y[69])


@pytest.mark.parametrize("layout", [transposed, every_second_column])
def test_another_stream_and_graphs(layout):
    print(f"streams and graphs {layout.__name__}", flush=True)
    x, w, d, rows, base = operands(200, 384, 1000)
    want = calls(x, w, d, rows, base)
    given = [laid_out(q, layout) for q in (x, w, d)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = calls(*given, rows, base, stream=s)
    junk = [torch.full((1 << 20,), 3.0, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del junk
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(*given, rows, base)
    for seed in range(3):
        new = operands(200, 384, 1000, seed)
        for to, q in zip(given, new):
            for p, v in zip(to.tensors(), q.tensors()):
                p.copy_(v)
        rows.copy_(new[3])
        base.copy_(new[4])
        graph.replay()
        want = calls(*new)
        torch.cuda.synchronize()
        assert all(torch.equal(p, v) for p, v in zip(got, want))


def test_results_must_be_contiguous():
    print("results", flush=True)
    x, w, _, rows, _ = operands(40, 130, 300)
    for q in (laid_out(x, every_second_row), nsd.Q4Matrix(40, 300, x.codes, every_second_column(x.scales))):
        with pytest.raises(nsd.DmuonError, match="contiguous"):
            nsd.q4_quantize(rows, out=q)
        with pytest.raises(nsd.DmuonError, match="contiguous"):
            nsd.q4_quantize_weights([rows], out=[q])


def test_offsets_beyond_32_bits():
    """More than 2^32 bytes of transposed codes, read where they lie first and last."""
    rows, cols = (1 << 21) + 5, 4100
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("not enough memory")
    print("offsets beyond 32 bits", flush=True)
    torch.manual_seed(3)
    raw = torch.randint(0, 256, (2176, rows), dtype=torch.uint8, device="cuda")
    scales = torch.randint(100, 150, (136, (rows + 15) // 16 * 16), dtype=torch.uint8, device="cuda")
    got = nsd.q4_dequantize(nsd.Q4Matrix(rows, cols, raw.t(), scales))
    for lo, hi in ((0, 300), (rows // 2, rows // 2 + 300), (rows - 300, rows)):
        s = scales[:, lo:hi]
        s = torch.nn.functional.pad(s, (0, -s.shape[1] % 16), value=2).contiguous()
        want = nsd.q4_dequantize(nsd.Q4Matrix(hi - lo, cols, raw[:, lo:hi].t().contiguous(), s))
        assert torch.equal(got[lo:hi], want)
    del got, raw
    torch.cuda.empty_cache()
