"""8-bit block products over torch tensors: the linear layers around the step.

``q8_quantize`` turns activations (or output gradients) into 8-bit rows,
``q8_quantize_weights`` the params into 8-bit weights, ``q8_matmul`` multiplies
the two, forward or (``transpose=True``) for the gradient of the input, and
``q8_weight_grad`` makes the weight gradient that ``muon_step`` reads from the
8-bit rows the forward pass kept.  The format is described in
``include/dmuon.h``: E4M3 codes, one power-of-two scale per block of 128.

A training step of one linear layer::

    w8, = nsd.q8_quantize_weights([w])
    x8 = nsd.q8_quantize(x)                          # kept for the backward pass
    y = nsd.q8_matmul(x8, w8)                        # x w^T
    dx = nsd.q8_matmul(nsd.q8_quantize(dy), w8, transpose=True)   # dy w
    nsd.q8_weight_grad(dy, x8, out=grad)             # dy^T x
    nsd.muon_step([w], [grad], [momentum], [scale])

The functions enqueue kernels on ``stream`` (the current one by default) and
record no gradients: the backward pass is the last two calls.  An input that
requires one is refused while gradients are recorded (parameters that
``q8_quantize_weights`` reads excepted), and so is one with a tangent of
forward-mode differentiation.  Results that are not passed in are new tensors;
without ``workspace`` a call that needs scratch allocates it.  On a ``stream`` of
its own a call's results and scratch belong to that stream, and all its tensors may
be dropped as soon as it returns; the caller only orders the streams (``stream``
after the work that makes the inputs, the readers of the results after
``stream``).  A ``Workspace`` serves any number of calls on one stream; work that
may overlap (calls on two streams, a call and a replayed graph, two graphs) needs
one each, and a graph's has to live as long as the graph.  Every call can be
captured into a graph, and the same call gives the same bits.
"""

from __future__ import annotations

import ctypes
from typing import List, Optional, Sequence

from . import _lib
from ._lib import DmuonError, Q8WeightDesc, check, load
from .api import Workspace, _allocating, _current_device, _dtype_code, _mark_used, _ptr, _raw_stream

BLOCK = 128


def _up(n: int, a: int) -> int:
    return -(-n // a) * a


class Q8Rows:
    """8-bit rows of a ``[rows, cols]`` matrix: ``codes`` ``[rows, cols up to
    128]`` (``torch.float8_e4m3fn``) and ``scales`` ``[cols up to 128 / 128,
    rows up to 4]`` (``torch.uint8``, exponent + 127)."""

    __slots__ = ("codes", "scales", "cols")

    def __init__(self, codes, scales, cols: int):
        self.codes, self.scales, self.cols = codes, scales, cols

    @classmethod
    def empty(cls, rows: int, cols: int, device) -> "Q8Rows":
        import torch
        kp = _up(cols, BLOCK)
        return cls(torch.empty(rows, kp, dtype=torch.float8_e4m3fn, device=device),
                   torch.empty(kp // BLOCK, _up(rows, 4), dtype=torch.uint8, device=device), cols)

    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()


class Q8Weight:
    """8-bit weights of a ``[rows, cols]`` matrix: ``codes`` ``[rows, cols up
    to 128]`` and ``scales``, one per 128 x 128 block; ``codes_t`` ``[cols,
    rows up to 128]`` and ``scales_t``, the same transposed, or None."""

    __slots__ = ("codes", "scales", "codes_t", "scales_t", "rows", "cols")

    def __init__(self, codes, scales, codes_t=None, scales_t=None, rows: Optional[int] = None,
                 cols: Optional[int] = None):
        self.codes, self.scales, self.codes_t, self.scales_t = codes, scales, codes_t, scales_t
        self.rows = codes.shape[0] if rows is None else rows
        # without the transposed codes the padding of cols cannot be told
        self.cols = cols if cols is not None else \
            (codes_t.shape[0] if codes_t is not None else codes.shape[1])

    @classmethod
    def empty(cls, rows: int, cols: int, device, transposed: bool = True) -> "Q8Weight":
        import torch
        np_, kp = _up(rows, BLOCK), _up(cols, BLOCK)
        nb, kb = np_ // BLOCK, kp // BLOCK
        f8, u8 = torch.float8_e4m3fn, torch.uint8
        return cls(torch.empty(rows, kp, dtype=f8, device=device),
                   torch.empty(nb, kb, dtype=u8, device=device),
                   torch.empty(cols, np_, dtype=f8, device=device) if transposed else None,
                   torch.empty(kb, nb, dtype=u8, device=device) if transposed else None, rows, cols)


def _invalid(message: str) -> DmuonError:
    return DmuonError(_lib.ERR_INVALID_ARG, message)


def _check_tensor(t, what: str, shape, dtype, device, contiguous: bool = True) -> None:
    """The checks that the C call cannot make: a kernel would read another
    device's memory, or past the end of a smaller tensor."""
    if t.device != device:
        raise _invalid(f"{what} is on {t.device}, not on {device}")
    if t.dtype != dtype:
        raise DmuonError(_lib.ERR_UNSUPPORTED_DTYPE, f"{what} has dtype {t.dtype}, not {dtype}")
    if t.shape != shape:
        raise _invalid(f"{what} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if contiguous and not t.is_contiguous():
        raise _invalid(f"{what} must be contiguous")


def _check_rows(q: Q8Rows, rows: int) -> None:
    import torch
    kp = _up(q.cols, BLOCK)
    _check_tensor(q.codes, "codes", (rows, kp), torch.float8_e4m3fn, q.codes.device)
    _check_tensor(q.scales, "scales", (kp // BLOCK, _up(rows, 4)), torch.uint8, q.codes.device)


_forward_ad = None


def _check_no_tangent(t, what: str) -> None:
    """The same of forward-mode differentiation, whose tensors require no gradient
    and which torch.no_grad() does not switch off."""
    global _forward_ad
    if _forward_ad is None:
        from torch.autograd import forward_ad
        _forward_ad = forward_ad
    # without an open level no tensor has a tangent (nor is it looked for, half a
    # microsecond a tensor)
    if getattr(_forward_ad, "_current_level", 0) >= 0 and _forward_ad.unpack_dual(t).tangent is not None:
        raise _invalid(f"{what} has a tangent, which this call does not carry on; call it in an "
                       "autograd.Function or on a detached tensor")


def _check_untracked(t, what: str) -> None:
    """No result carries a gradient on: an input that autograd tracks would leave
    its graph without a word."""
    _check_no_tangent(t, what)
    if not t.requires_grad:
        return
    import torch
    if torch.is_grad_enabled():
        raise _invalid(f"{what} requires a gradient, which this call does not record; call it under "
                       "torch.no_grad(), in an autograd.Function or on a detached tensor")


def _matrix(t, what: str):
    """``t``'s device, rows and columns; any leading dimensions are rows."""
    _check_untracked(t, what)
    if t.dim() < 1 or t.shape[-1] < 1:
        raise _invalid(f"{what} needs at least one column")
    if not t.is_cuda:
        raise _invalid(f"{what} is on {t.device}, not on a GPU")
    cols = t.shape[-1]
    return t.device, t.numel() // cols, cols


def _run(fn, device, stream, *args) -> None:
    """One C call on ``stream`` (by default ``device``'s current one), with
    ``device`` current, since kernels are loaded per device."""
    index = device.index
    if stream is None:
        handle = _raw_stream(index)
    else:
        handle = stream.cuda_stream
    if _current_device() == index:
        status = fn(*args, handle)
    else:
        import torch
        with torch.cuda.device(device):
            status = fn(*args, handle)
    if status:
        check(status)


def _check_stream(device, stream) -> None:
    if stream.device != device:
        raise _invalid(f"the stream is on {stream.device}, the tensors on {device}")


def _keep(device, stream, results, made: bool, inputs) -> None:
    """For a call on a stream of its own: the memory of every tensor of it stays
    theirs until the stream is done with it, and that of results made for the
    call (which belongs to ``stream``) until the current stream is."""
    import torch
    _mark_used(stream, *results, *inputs)
    if made:
        _mark_used(torch.cuda.current_stream(device), *results)


def q8_quantize(x, out: Optional[Q8Rows] = None, stream=None) -> Q8Rows:
    """8-bit rows of ``x`` (bf16 or fp32, ``[..., cols]``; the leading
    dimensions are flattened), one scale per 1 x 128 block."""
    device, rows, cols = _matrix(x, "x")
    if stream is not None:
        _check_stream(device, stream)
    dt = _dtype_code(x)
    made = out is None
    if made:
        with _allocating(stream):
            out = Q8Rows.empty(rows, cols, device)
    else:
        if out.cols != cols or out.codes.device != device:
            raise _invalid("out does not fit x")
        _check_rows(out, rows)
    if stream is not None:
        _keep(device, stream, (out.codes, out.scales), made, (x,))
    _run(load().dmuon_q8_quantize, device, stream, _ptr(x), dt, rows, cols, out.codes.data_ptr(),
         out.scales.data_ptr())
    return out


def q8_quantize_weights(params: Sequence, out: Optional[Sequence[Q8Weight]] = None,
                        transposed: bool = True, stream=None) -> List[Q8Weight]:
    """8-bit weights of each matrix (bf16 or fp32, ``[rows, cols]``), one scale
    per 128 x 128 block; without ``transposed`` only what the forward product
    reads.  All matrices lie on one device.  ``out`` takes an earlier call's
    results, with or without their transposed codes, and overwrites them, their
    ``rows`` and ``cols`` too (columns that round up to the same 128 fit)."""
    import torch
    n = len(params)
    if n == 0:
        return []
    for i, p in enumerate(params):
        if p.is_leaf:  # a parameter may be quantised, as the step may update it
            _check_no_tangent(p, f"matrix {i}")
        else:
            _check_untracked(p, f"matrix {i}")
    device = params[0].device
    for i, p in enumerate(params):
        if p.dim() != 2:
            raise _invalid(f"matrix {i} is not 2-D")
        if not p.is_cuda or p.device != device:
            raise _invalid(f"matrix {i} is on {p.device}, not on {device} (a GPU)")
    if stream is not None:
        _check_stream(device, stream)
    made = out is None
    if made:
        with _allocating(stream):
            out = [Q8Weight.empty(p.shape[0], p.shape[1], device, transposed) for p in params]
    else:
        out = list(out)
        if len(out) != n:
            raise _invalid(f"{len(out)} results for {n} matrices")
        f8, u8 = torch.float8_e4m3fn, torch.uint8
        for p, q in zip(params, out):
            r, c = p.shape
            np_, kp = _up(r, BLOCK), _up(c, BLOCK)
            _check_tensor(q.codes, "codes", (r, kp), f8, device)
            _check_tensor(q.scales, "scales", (np_ // BLOCK, kp // BLOCK), u8, device)
            if (q.codes_t is None) != (q.scales_t is None):
                raise _invalid("codes_t and scales_t go together")
            if q.codes_t is not None:
                _check_tensor(q.codes_t, "codes_t", (c, np_), f8, device)
                _check_tensor(q.scales_t, "scales_t", (kp // BLOCK, np_ // BLOCK), u8, device)
    arr = (Q8WeightDesc * n)()
    for i, (p, q) in enumerate(zip(params, out)):
        arr[i] = Q8WeightDesc(_ptr(p), _dtype_code(p), 0, p.shape[0], p.shape[1],
                              q.codes.data_ptr(), q.scales.data_ptr(), _ptr(q.codes_t),
                              _ptr(q.scales_t))
        if stream is not None:
            _keep(device, stream, (q.codes, q.scales, q.codes_t, q.scales_t), made, (p,))
    _run(load().dmuon_q8_quantize_weights, device, stream, arr, n)
    for p, q in zip(params, out):
        q.rows, q.cols = p.shape
    return out


def _workspace(call, sizes, workspace: Optional[Workspace], device, stream):
    """Device scratch for a product of these sizes: (address, bytes, tensor);
    the tensor keeps the memory until the launches are enqueued."""
    need = ctypes.c_size_t(0)
    check(call(*sizes, ctypes.byref(need)))
    return _scratch(need.value, workspace, device, stream)


def _scratch(need: int, workspace: Optional[Workspace], device, stream):
    """``_workspace`` of ``need`` bytes."""
    if need == 0:
        return None, 0, None
    if workspace is not None:
        buf = workspace.get(need, device, stream)
    else:
        import torch
        with _allocating(stream):
            buf = torch.empty(need, dtype=torch.uint8, device=device)
    return buf.data_ptr(), buf.numel(), buf


def q8_matmul(a: Q8Rows, w: Q8Weight, transpose: bool = False, out=None, dtype=None,
              workspace: Optional[Workspace] = None, stream=None, fast_sums: bool = False):
    """``a w^T`` (``[rows, w.rows]``) or, with ``transpose``, ``a w``
    (``[rows, w.cols]``), bf16 (the default) or fp32: exact products, fp32 sums,
    one rounding.  ``out`` takes the result; its dtype is then the result's.

    With ``fast_sums``, for a bf16 result, the sums are the 8-bit matrix
    instruction's, twice as fast for many rows: products are added in groups of
    eight, each cut toward zero at 2^-13 of the group's largest.  That adds an
    error of 1.5e-5 of the result's norm on Gaussian operands, 4e-5 with outlier
    channels, and at most 7 * 2^-13 of the products' sum of magnitudes."""
    import torch
    rows, device = a.codes.shape[0], a.codes.device
    codes, scales = (w.codes_t, w.scales_t) if transpose else (w.codes, w.scales)
    if codes is None or scales is None:
        raise _invalid("the weight has no transposed codes")
    outs, inner = (w.cols, w.rows) if transpose else (w.rows, w.cols)
    if not a.codes.is_cuda:
        raise _invalid(f"codes are on {device}, not on a GPU")
    if stream is not None:
        _check_stream(device, stream)
    if a.cols != inner:
        raise _invalid(f"rows of {a.cols} columns against a weight of {inner}")
    _check_rows(a, rows)
    kp = _up(inner, BLOCK)
    _check_tensor(codes, "the weight's codes", (outs, kp), torch.float8_e4m3fn, device)
    _check_tensor(scales, "the weight's scales", (_up(outs, BLOCK) // BLOCK, kp // BLOCK),
                  torch.uint8, device)
    made = out is None
    if made:
        with _allocating(stream):
            out = torch.empty(rows, outs, dtype=dtype or torch.bfloat16, device=device)
    else:
        if dtype is not None and dtype != out.dtype:
            raise _invalid(f"out has dtype {out.dtype}, not {dtype}")
        _check_tensor(out, "out", (rows, outs), out.dtype, device)
    lib = load()
    dt = _dtype_code(out)
    if fast_sums:
        dt |= _lib.Q8_FAST_SUMS
    ws, nws, keep = _workspace(lib.dmuon_q8_matmul_workspace_bytes, (rows, outs, inner, dt),
                               workspace, device, stream)
    if stream is not None:
        _keep(device, stream, (out,), made, (a.codes, a.scales, codes, scales))
    _run(lib.dmuon_q8_matmul, device, stream, a.codes.data_ptr(), a.scales.data_ptr(), rows,
         codes.data_ptr(), scales.data_ptr(), outs, inner, out.data_ptr(), dt, ws, nws)
    return out


def q8_weight_grad(dy, x: Q8Rows, out=None, dtype=None, base=None,
                   workspace: Optional[Workspace] = None, stream=None):
    """``base + dy^T x`` (``[dy's columns, x.cols]``): the weight gradient of
    ``y = x w^T`` from the bf16 gradient ``dy`` (``[..., outs]``) and the 8-bit
    rows of ``x``.  The result is ``out`` (for instance the ``grads`` entry of
    ``muon_step``) or a new tensor of ``dtype`` (bf16 by default, else fp32).
    ``base`` has the result's dtype and may be ``out`` itself, which adds to
    the gradient in place."""
    import torch
    device, rows, outs = _matrix(dy, "dy")
    if stream is not None:
        _check_stream(device, stream)
    if dy.dtype != torch.bfloat16:
        raise DmuonError(_lib.ERR_UNSUPPORTED_DTYPE, f"dy has dtype {dy.dtype}, not torch.bfloat16")
    if not dy.is_contiguous():
        raise _invalid("dy must be contiguous")
    if x.codes.device != device:
        raise _invalid(f"codes are on {x.codes.device}, not on {device}")
    _check_rows(x, rows)
    cols = x.cols
    made = out is None
    if made:
        with _allocating(stream):
            out = torch.empty(outs, cols, device=device,
                              dtype=dtype or (base.dtype if base is not None else torch.bfloat16))
    else:
        if dtype is not None and dtype != out.dtype:
            raise _invalid(f"out has dtype {out.dtype}, not {dtype}")
        _check_tensor(out, "out", (outs, cols), out.dtype, device)
    if base is not None:
        _check_untracked(base, "base")
        _check_tensor(base, "base", (outs, cols), out.dtype, device)
    lib = load()
    ws, nws, keep = _workspace(lib.dmuon_q8_weight_grad_workspace_bytes, (rows, outs, cols),
                               workspace, device, stream)
    if stream is not None:
        _keep(device, stream, (out,), made, (dy, x.codes, x.scales, base))
    _run(lib.dmuon_q8_weight_grad, device, stream, dy.data_ptr(), x.codes.data_ptr(),
         x.scales.data_ptr(), rows, outs, cols, base.data_ptr() if base is not None else None,
         out.data_ptr(), _dtype_code(out), ws, nws)
    return out
