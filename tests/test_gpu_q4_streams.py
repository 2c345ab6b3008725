"""The 4-bit block products on streams and in graphs: whose stream a call's memory
belongs to, calls in flight at once, captures replayed beside eager work."""

import numpy as np
import pytest
import torch

import newton_schulz_dmuon_amd as nsd
from test_gpu_q4 import BF16, F32, values

pytestmark = pytest.mark.gpu


def inputs(seed, t=300, n=384, k=1536):
    rng = np.random.default_rng(seed)
    r = torch.from_numpy(rng.integers(0, 256, (t, n)).astype(np.uint8)).cuda()
    return (values(rng, t, k, BF16).cuda(), values(rng, t, n, BF16, 1e-2).cuda(), values(rng, n, k, BF16, 0.02).cuda(),
            values(rng, n, k, F32, 0.1).cuda(), r)


def layer(x, dy, w, grad, r, workspace=None, stream=None):
    """One linear layer's training step, every product of it, and its serving."""
    kw = dict(workspace=workspace, stream=stream)
    w4 = nsd.q4_quantize_weights([w], stream=stream)[0]
    x4 = nsd.q4_quantize(x, transposed=True, stream=stream)
    y = nsd.q4_matmul(x4, w4, **kw)
    d4 = nsd.q4_quantize(dy, transposed=True, random=r, stream=stream)
    dx = nsd.q4_matmul(d4, w4, transpose=True, dtype=F32, **kw)
    nsd.q4_weight_grad(d4, x4, out=grad, base=grad, **kw)
    # a row length that is padded first
    z = nsd.q4_matmul(x, w4, **kw)
    return y, dx, z, nsd.q4_dequantize(w4, transpose=True, stream=stream)


def same(a, b):
    return len(a) == len(b) and all(torch.equal(p, q) for p, q in zip(a, b))


SIZES = [(1, 384, 1536), (40, 390, 1500), (300, 384, 1536), (2048, 384, 1536), (2048, 1000, 1000)]


@pytest.mark.parametrize("size", SIZES)
def test_another_stream(size):
    print(f"another stream {size}", flush=True)
    x, dy, w, g0, r = inputs(1, *size)
    g = g0.clone()
    want = layer(x, dy, w, g, r)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g2 = g0.clone()
    torch.cuda.synchronize()
    got = layer(x, dy, w, g2, r, stream=s)
    # churn of the current stream's allocator while the other stream works
    junk = [torch.full((1 << 20,), 3.0, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert same(got, want) and torch.equal(g, g2)
    del junk


@pytest.mark.parametrize("own_workspaces", [False, True])
def test_two_streams_at_once(own_workspaces):
    """Calls in flight on two streams, and a graph replaying beside them, give the
    results of calls one after the other."""
    print(f"two streams {own_workspaces}", flush=True)
    given = [inputs(20 + i, t) for i, t in enumerate((300, 2048))]
    want = []
    for x, dy, w, g, r in given:
        g = g.clone()
        want.append(layer(x, dy, w, g, r) + (g,))
    ws = [nsd.Workspace() if own_workspaces else None for _ in range(3)]
    x, dy, w, g0, r = given[1]
    gg = g0.clone()
    layer(x, dy, w, gg, r, workspace=ws[2])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = layer(x, dy, w, gg, r, workspace=ws[2])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        gg.copy_(g0)
        grads = [i[3].clone() for i in given]
        torch.cuda.synchronize()
        graph.replay()
        got = [layer(*i[:3], g, i[4], stream=s, workspace=v) for i, g, s, v in zip(given, grads, streams, ws)]
        torch.cuda.synchronize()
        for a, g, b in zip(got, grads, want):
            assert same(a + (g,), b)
        assert same(captured + (gg,), want[1])


@pytest.mark.parametrize("size", SIZES)
def test_graph_replays(size):
    """Captured with a workspace of its own and replayed on changing inputs, the
    eager calls running in between on theirs."""
    print(f"graph {size}", flush=True)
    given = inputs(2, *size)
    ws, eager = nsd.Workspace(), nsd.Workspace()
    x, dy, w, g, r = given
    with torch.cuda.stream(torch.cuda.Stream()):
        layer(x, dy, w, g.clone(), r, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(x, dy, w, g, r, workspace=ws)
    for i in range(4):
        new = inputs(10 + i, *size)
        for a, b in zip(given, new):
            a.copy_(b)
        graph.replay()
        want = layer(*new, workspace=eager)
        torch.cuda.synchronize()
        assert same(got, want) and torch.equal(g, new[3]), i


def test_a_capture_that_forks():
    """A backward pass captured with the weight's gradient on a stream of its own,
    nothing passed in and the temporaries dropped, replayed on changing inputs
    beside eager calls."""
    print("a forked capture", flush=True)
    x, dy, w, _, r = inputs(60, 2048)
    s = torch.cuda.Stream()

    def backward(x, dy, w, r, stream):
        x4, w4 = nsd.q4_quantize(x, transposed=True, plain=False), nsd.q4_quantize_weights([w])[0]
        d4 = nsd.q4_quantize(dy, transposed=True, random=r)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        dx = nsd.q4_matmul(d4, w4, transpose=True)
        dw = nsd.q4_weight_grad(d4, x4, stream=stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        return dx, dw

    backward(x, dy, w, r, s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = backward(x, dy, w, r, s)
    for i in range(4):
        nx, ndy, nw, _, nr = inputs(61 + i, 2048)
        for a, b in zip((x, dy, w, r), (nx, ndy, nw, nr)):
            a.copy_(b)
        graph.replay()
        want = backward(nx, ndy, nw, nr, None)
        torch.cuda.synchronize()
        assert same(got, want), i


def freed_block(nbytes):
    """The address of a block of the current stream, free again, that the next
    allocation of this size on it takes (asserted)."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    t = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    at = t.data_ptr()
    del t
    t = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    assert t.data_ptr() == at
    del t
    return at


def test_results_on_another_stream_take_no_block_of_the_current_one():
    print("results' blocks", flush=True)
    t, n, k = 2048, 2048, 4096
    s = torch.cuda.Stream()
    x, w, dy = (torch.ones(a, b, dtype=BF16, device="cuda") for a, b in ((t, k), (n, k), (t, n)))
    x4, w4 = nsd.q4_quantize(x, transposed=True), nsd.q4_quantize_weights([w])[0]
    d4 = nsd.q4_quantize(dy, transposed=True)
    calls = [(lambda: nsd.q4_quantize(x, transposed=True, stream=s), lambda q: q.tensors(), t * k // 2),
             (lambda: nsd.q4_quantize_weights([w], stream=s)[0], lambda q: q.tensors(), n * k // 2),
             (lambda: nsd.q4_dequantize(w4, stream=s), lambda y: (y,), 2 * n * k),
             (lambda: nsd.q4_matmul(x4, w4, stream=s), lambda y: (y,), 2 * t * n),
             (lambda: nsd.q4_matmul(x, w4, dtype=F32, stream=s), lambda y: (y,), 4 * t * n),
             (lambda: nsd.q4_weight_grad(d4, x4, stream=s), lambda g: (g,), 2 * n * k)]
    for call, tensors, nbytes in calls:
        at = freed_block(nbytes)
        result = call()
        assert at not in {v.untyped_storage().data_ptr() for v in tensors(result)}
        # and the block is still the current stream's
        assert torch.empty(nbytes, dtype=torch.uint8, device="cuda").data_ptr() == at
        torch.cuda.synchronize()


def test_inputs_may_be_dropped_after_a_call():
    """Operands made on the current stream, used on another behind pending work
    there, and dropped: their memory goes to no new tensor before it is done."""
    print("dropped inputs", flush=True)
    s = torch.cuda.Stream()
    cur = torch.cuda.current_stream()
    x, dy, w, _, r = inputs(3, 1024, 1024, 2000)
    want = None
    for i in range(6):
        a, b = nsd.q4_quantize(x, transposed=True), nsd.q4_quantize_weights([w])[0]
        d, xx = nsd.q4_quantize(dy, transposed=True, random=r), x.clone()
        if i:
            s.wait_stream(cur)
            with torch.cuda.stream(s):
                torch.cuda._sleep(int(2e7))
        kw = dict(stream=s) if i else {}
        got = (nsd.q4_matmul(a, b, **kw), nsd.q4_matmul(xx, b, **kw), nsd.q4_weight_grad(d, a, **kw), nsd.q4_dequantize(b, **kw),
               nsd.q4_quantize(xx, **kw).codes)
        del a, b, d, xx
        junk = [torch.full((1024, 2048), 255, dtype=torch.uint8, device="cuda") for _ in range(12)]
        torch.cuda.synchronize()
        want = want or got
        assert same(got, want)
        del junk


def test_a_captured_workspace_outlives_a_larger_call():
    """Captured with a warmed Workspace, which a larger product then uses eagerly:
    the graph's scratch (rows of 1001 elements are copied there) goes to no new
    tensor, and its replays stay right."""
    print("captured workspace", flush=True)
    rng = np.random.default_rng(5)
    w = nsd.q4_quantize_weights([values(rng, 700, 1001, BF16, 0.02).cuda()])[0]
    small, large = values(rng, 300, 1001, BF16).cuda(), values(rng, 5000, 1001, BF16).cuda()
    want, want_large = nsd.q4_matmul(small, w), nsd.q4_matmul(large, w)
    ws = nsd.Workspace()
    nsd.q4_matmul(small, w, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = nsd.q4_matmul(small, w, workspace=ws)
    scratch, nbytes = ws.buf.data_ptr(), ws.buf.numel()
    for _ in range(3):
        assert torch.equal(nsd.q4_matmul(large, w, workspace=ws), want_large)
        assert ws.buf.numel() > nbytes
        torch.cuda.synchronize()
        held = [torch.full((nbytes,), 7, dtype=torch.uint8, device="cuda") for _ in range(4)]
        assert all(h.data_ptr() != scratch for h in held)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and all((h == 7).all() for h in held)


def test_no_rows_on_another_stream():
    print("no rows on a stream", flush=True)
    s = torch.cuda.Stream()
    w4 = nsd.q4_quantize_weights([torch.ones(130, 200, dtype=BF16, device="cuda")], stream=s)[0]
    empty = torch.empty(0, 200, dtype=BF16, device="cuda")
    x4 = nsd.q4_quantize(empty, transposed=True, stream=s)
    assert nsd.q4_matmul(x4, w4, stream=s).shape == (0, 130) and nsd.q4_matmul(empty, w4, stream=s).shape == (0, 130)
    d4 = nsd.q4_quantize(torch.empty(0, 130, dtype=BF16, device="cuda"), transposed=True, stream=s)
    grad = nsd.q4_weight_grad(d4, x4, stream=s)
    torch.cuda.synchronize()
    assert grad.shape == (130, 200) and not grad.any()
