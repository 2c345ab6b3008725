"""Memory of the 8-bit block products' calls on another stream than the current
one.  A block that was freed on the current stream may still be in use by work
there, so nothing that another stream writes may lie in it."""

import numpy as np
import pytest
import torch

import newton_schulz_dmuon_amd as nsd
from test_gpu_q8 import BF16, F32, layer_inputs, values

pytestmark = pytest.mark.gpu


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


def addresses(*tensors):
    return {t.untyped_storage().data_ptr() for t in tensors}


def test_results_on_another_stream_take_no_block_of_the_current_one():
    print("results' blocks", flush=True)
    t, n, k = 2048, 2048, 4096
    s = torch.cuda.Stream()
    x, w, dy = (torch.ones(r, c, dtype=BF16, device="cuda") for r, c in ((t, k), (n, k), (t, n)))
    x8, w8 = nsd.q8_quantize(x), nsd.q8_quantize_weights([w])[0]
    calls = [(lambda: nsd.q8_quantize(x, stream=s), lambda q: (q.codes, q.scales), t * k),
             (lambda: nsd.q8_quantize_weights([w], stream=s)[0], lambda q: (q.codes, q.codes_t, q.scales, q.scales_t), n * k),
             (lambda: nsd.q8_matmul(x8, w8, stream=s), lambda y: (y,), 2 * t * n),
             (lambda: nsd.q8_matmul(x8, w8, dtype=F32, stream=s), lambda y: (y,), 4 * t * n),
             (lambda: nsd.q8_weight_grad(dy, x8, stream=s), lambda g: (g,), 2 * n * k)]
    for call, tensors, nbytes in calls:
        at = freed_block(nbytes)
        result = call()
        assert at not in addresses(*tensors(result))
        # and the block is still the current stream's
        assert torch.empty(nbytes, dtype=torch.uint8, device="cuda").data_ptr() == at
        torch.cuda.synchronize()


def test_workspaces_on_another_stream_take_no_block_of_the_current_one():
    print("workspaces' blocks", flush=True)
    t, n, k = 4096, 1024, 4096
    s = torch.cuda.Stream()
    x8 = nsd.q8_quantize(torch.ones(t, k, dtype=BF16, device="cuda"))
    dy, grad = torch.ones(t, n, dtype=BF16, device="cuda"), torch.zeros(n, k, device="cuda")
    ws = nsd.Workspace()
    nsd.q8_weight_grad(dy, x8, out=grad, workspace=ws)
    nbytes = ws.buf.numel()
    assert nbytes > 1 << 20  # the sum is split
    del ws
    ws = nsd.Workspace()
    at = freed_block(nbytes)
    nsd.q8_weight_grad(dy, x8, out=grad, workspace=ws, stream=s)
    assert at not in addresses(ws.buf)
    torch.cuda.synchronize()
    params = [torch.ones(512, 512, dtype=BF16, device="cuda")]
    args = (params, [params[0] * 0.5], [torch.zeros(512, 512, device="cuda")], [1.0])
    steps = nsd.Workspace()
    nsd.muon_step(*args, workspace=steps)
    nbytes = steps.buf.numel()
    del steps
    steps = nsd.Workspace()
    at = freed_block(nbytes)
    nsd.muon_step(*args, workspace=steps, stream=s)
    assert at not in addresses(steps.buf)
    torch.cuda.synchronize()


def test_a_workspace_is_kept_for_every_stream_that_used_it():
    """Made for one stream, used on a second and replaced by a larger one: the
    old buffer's memory goes to nobody before the second stream is done."""
    print("a workspace on two streams", flush=True)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    device = torch.device("cuda", torch.cuda.current_device())
    ws = nsd.Workspace()
    at = ws.get(8 << 20, device, a).data_ptr()
    assert ws.get(8 << 20, device, b).data_ptr() == at
    with torch.cuda.stream(b):
        torch.cuda._sleep(int(2e8))
    ws.get(64 << 20, device, a)
    with torch.cuda.stream(a):
        t = torch.empty(8 << 20, dtype=torch.uint8, device="cuda")
    assert not b.query() and t.data_ptr() != at
    torch.cuda.synchronize()


def test_products_of_a_backward_pass_on_two_streams():
    """The input's gradient on the current stream, the weight's on another, with
    neither results nor workspaces passed in, and temporaries dropped at once."""
    print("backward on two streams", flush=True)
    s = torch.cuda.Stream()
    cur = torch.cuda.current_stream()
    for t, n, k in ((2048, 384, 1536), (300, 512, 1536), (4096, 1024, 2048)):
        x, dy, w, _ = layer_inputs(40 + t, t, n, k)
        x8, w8 = nsd.q8_quantize(x), nsd.q8_quantize_weights([w])[0]
        want = nsd.q8_matmul(nsd.q8_quantize(dy), w8, transpose=True), nsd.q8_weight_grad(dy, x8)
        torch.cuda.synchronize()
        for _ in range(20):
            s.wait_stream(cur)
            dx = nsd.q8_matmul(nsd.q8_quantize(dy), w8, transpose=True)
            dw = nsd.q8_weight_grad(dy, x8, stream=s)
            cur.wait_stream(s)
            assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


def test_work_pending_on_a_freed_block():
    """Long work on the current stream whose result is freed before it runs, then
    a call on another stream with a result of the same size."""
    print("pending work", flush=True)
    s = torch.cuda.Stream()
    rng = np.random.default_rng(2)
    x = values(rng, 1024, 2048, BF16).cuda()
    w8 = nsd.q8_quantize_weights([values(rng, 1024, 2048, BF16, 0.02).cuda()])[0]
    x8 = nsd.q8_quantize(x)
    want = nsd.q8_matmul(x8, w8)
    torch.cuda.synchronize()
    for _ in range(5):
        tmp = torch.empty(1024, 1024, dtype=BF16, device="cuda")
        torch.cuda._sleep(int(2e7))
        tmp.fill_(7.0)
        del tmp
        y = nsd.q8_matmul(x8, w8, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_inputs_may_be_dropped_after_a_call():
    """Operands made on the current stream, used on another behind pending work
    there, and dropped: their memory goes to no new tensor before it is done."""
    print("dropped inputs", flush=True)
    s = torch.cuda.Stream()
    cur = torch.cuda.current_stream()
    rng = np.random.default_rng(3)
    x = values(rng, 1024, 2048, BF16).cuda()
    w = values(rng, 1024, 2048, BF16, 0.02).cuda()
    want = nsd.q8_matmul(nsd.q8_quantize(x), nsd.q8_quantize_weights([w])[0])
    torch.cuda.synchronize()
    for _ in range(5):
        a, b = nsd.q8_quantize(x), nsd.q8_quantize_weights([w])[0]
        s.wait_stream(cur)
        with torch.cuda.stream(s):
            torch.cuda._sleep(int(2e7))
        y = nsd.q8_matmul(a, b, stream=s)
        del a, b
        junk = [torch.full((1024, 2048), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        del junk


def test_a_captured_workspace_outlives_a_larger_call():
    """Captured with a warmed Workspace, which a larger layer then uses eagerly:
    the graph's scratch goes to no new tensor, and its replays stay right."""
    print("captured workspace", flush=True)
    small, large = layer_inputs(50, 2048, 384, 1536), layer_inputs(51, 8192, 1024, 2048)
    ws = nsd.Workspace()

    def grad(inputs, ws):
        x, dy, _, base = inputs
        return nsd.q8_weight_grad(dy, nsd.q8_quantize(x), base=base, workspace=ws)

    want, want_large = grad(small, None), grad(large, None)
    grad(small, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = grad(small, ws)
    scratch, nbytes = ws.buf.data_ptr(), ws.buf.numel()
    for _ in range(3):
        assert torch.equal(grad(large, ws), want_large)
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
    w8 = nsd.q8_quantize_weights([torch.ones(130, 200, dtype=BF16, device="cuda")], stream=s)[0]
    x8 = nsd.q8_quantize(torch.empty(0, 200, dtype=BF16, device="cuda"), stream=s)
    assert nsd.q8_matmul(x8, w8, stream=s).shape == (0, 130)
    grad = nsd.q8_weight_grad(torch.empty(0, 130, dtype=BF16, device="cuda"), x8, stream=s)
    torch.cuda.synchronize()
    assert grad.shape == (130, 200) and not grad.any()


def test_a_capture_that_forks():
    """A backward pass captured with the weight's gradient on a stream of its own,
    nothing passed in and the temporaries dropped, replayed on changing inputs
    beside eager calls."""
    print("a forked capture", flush=True)
    t, n, k = 2048, 384, 1536
    x, dy, w, _ = layer_inputs(60, t, n, k)
    s = torch.cuda.Stream()

    def backward(x, dy, w, stream):
        x8, w8 = nsd.q8_quantize(x), nsd.q8_quantize_weights([w])[0]
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        dx = nsd.q8_matmul(nsd.q8_quantize(dy), w8, transpose=True)
        dw = nsd.q8_weight_grad(dy, x8, stream=stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        return dx, dw

    backward(x, dy, w, s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx, dw = backward(x, dy, w, s)
    for i in range(4):
        nx, ndy, nw, _ = layer_inputs(61 + i, t, n, k)
        x.copy_(nx)
        dy.copy_(ndy)
        w.copy_(nw)
        graph.replay()
        want = backward(nx, ndy, nw, None)
        torch.cuda.synchronize()
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1]), i
