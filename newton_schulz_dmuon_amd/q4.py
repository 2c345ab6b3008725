"""4-bit block products over torch tensors: the linear layers around the step
with microscaled 4-bit operands (E2M1 codes, one power-of-two scale per 32).

``q4_quantize`` turns activations or output gradients into 4-bit matrices,
``q4_quantize_weights`` the params, ``q4_dequantize`` reads one back,
``q4_matmul`` multiplies 4-bit rows, or bf16 rows, by 4-bit weights, forward or
(``transpose=True``) for the gradient of the input, and ``q4_weight_grad`` makes
the weight gradient that ``muon_step`` reads.  The format is described in
``include/dmuon.h``.  Its blocks lie along the direction that a product sums over,
so a matrix has two forms of other codes: ``codes`` for sums along its rows and
``codes_t`` for sums along its columns.

A training step of one linear layer::

    w4, = nsd.q4_quantize_weights([w])               # both forms
    x4 = nsd.q4_quantize(x, transposed=True)         # codes_t is kept for the backward pass
    y = nsd.q4_matmul(x4, w4)                        # x w^T
    r = torch.randint(0, 256, dy.shape, dtype=torch.uint8, device=dy.device)
    dy4 = nsd.q4_quantize(dy, transposed=True, random=r)
    dx = nsd.q4_matmul(dy4, w4, transpose=True)      # dy w
    nsd.q4_weight_grad(dy4, x4, out=grad)            # dy^T x
    nsd.muon_step([w], [grad], [momentum], [scale])

Serving with a weight in 4 bits and activations in bf16: ``nsd.q4_matmul(x, w4)``.

Gradients, streams, workspaces, graphs and reproducibility are as for the 8-bit
products (``q8.py``): no gradients are recorded and inputs that would lose one are
refused, a call's results and scratch belong to its ``stream``, work that may
overlap needs a ``Workspace`` each, every call can be captured, and the same call
gives the same bits.
"""

from __future__ import annotations

import ctypes
import functools
from typing import List, Optional, Sequence

from . import _lib
from ._lib import DmuonError, Q4SourceDesc, check, load
from .api import Workspace, _allocating, _dtype_code, _mark_used, _ptr
from .q8 import (_check_no_tangent, _check_stream, _check_tensor, _check_untracked, _invalid, _keep, _matrix, _run,
                 _scratch, _up)

BLOCK = 32
PAD = 256


def _form(rows: int, cols: int, device):
    import torch
    cp = _up(cols, PAD)
    return (torch.empty(rows, cp // 2, dtype=torch.uint8, device=device),
            torch.empty(cp // BLOCK, _up(rows, 16), dtype=torch.uint8, device=device))


class Q4Matrix:
    """A ``[rows, cols]`` matrix in 4 bits, ``torch.uint8`` throughout: ``codes``
    ``[rows, cols up to 256 / 2]``, two to a byte, with ``scales`` ``[cols up to
    256 / 32, rows up to 16]`` (exponent + 127), for sums along its rows; and
    ``codes_t`` ``[cols, rows up to 256 / 2]`` with ``scales_t``, the same of its
    transpose.  Either form may be None, and dropped when no product needs it any
    more.  Codes and scales that a call reads may have any strides and begin anywhere
    (what is not contiguous, or begins at no multiple of 16 bytes, is copied first, on
    the call's stream); those that one writes may not."""

    __slots__ = ("rows", "cols", "codes", "scales", "codes_t", "scales_t")

    def __init__(self, rows: int, cols: int, codes=None, scales=None, codes_t=None, scales_t=None):
        self.rows, self.cols = rows, cols
        self.codes, self.scales, self.codes_t, self.scales_t = codes, scales, codes_t, scales_t

    @classmethod
    def empty(cls, rows: int, cols: int, device, plain: bool = True, transposed: bool = True) -> "Q4Matrix":
        return cls(rows, cols, *(_form(rows, cols, device) if plain else (None, None)),
                   *(_form(cols, rows, device) if transposed else (None, None)))

    def tensors(self):
        return self.codes, self.scales, self.codes_t, self.scales_t

    def nbytes(self) -> int:
        return sum(t.numel() for t in self.tensors() if t is not None)


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(call: str, rows: int, outs: int, inner: int) -> int:
    """A function of the sizes alone."""
    need = ctypes.c_size_t(0)
    check(getattr(load(), call + "_workspace_bytes")(rows, outs, inner, ctypes.byref(need)))
    return need.value


_uint8 = None


def _check_form(codes, scales, rows: int, cols: int, what: str, device, strided: bool = False) -> bool:
    """Whether both are contiguous, which they have to be unless ``strided``."""
    global _uint8
    cp = _up(cols, PAD)
    if (codes.shape == (rows, cp // 2) and scales.shape == (cp // BLOCK, _up(rows, 16)) and
            codes.dtype is _uint8 and scales.dtype is _uint8 and codes.device == device and scales.device == device and
            codes.is_contiguous() and scales.is_contiguous()):
        return True
    import torch
    _uint8 = torch.uint8  # at first None, which no type is
    _check_tensor(codes, f"{what}'s codes", (rows, cp // 2), torch.uint8, device, not strided)
    _check_tensor(scales, f"{what}'s scales", (cp // BLOCK, _up(rows, 16)), torch.uint8, device, not strided)
    return codes.is_contiguous() and scales.is_contiguous()


def _dense(t, stream):
    """``t``, or a copy that is contiguous and aligned and belongs to the call's
    stream."""
    if t.is_contiguous() and t.data_ptr() % 16 == 0:
        return t
    import torch
    with _allocating(stream):
        out = torch.empty(t.shape, dtype=t.dtype, device=t.device)
    if stream is not None:
        _mark_used(stream, t)
    _run(load().dmuon_q4_copy, t.device, stream, t.data_ptr(), *t.shape, *t.stride(), out.data_ptr())
    return out


def _dense_form(codes, scales, stream):
    codes, scales = _dense(codes, stream), _dense(scales, stream)
    return codes, scales, codes.data_ptr(), scales.data_ptr()


def _form_of(q: Q4Matrix, transposed: bool, what: str):
    """The codes and scales of one form, its rows and its columns, and their
    addresses: None if they do not lie as the kernels read them, who then get
    ``_dense_form``."""
    codes, scales = (q.codes_t, q.scales_t) if transposed else (q.codes, q.scales)
    if codes is None or scales is None:
        raise _invalid(f"{what} has no {'transposed ' if transposed else ''}codes")
    if not codes.is_cuda:
        raise _invalid(f"{what}'s codes are on {codes.device}, not on a GPU")
    rows, cols = (q.cols, q.rows) if transposed else (q.rows, q.cols)
    if _check_form(codes, scales, rows, cols, what, codes.device, True):
        p, ps = codes.data_ptr(), scales.data_ptr()
        if not (p | ps) & 15:
            return codes, scales, rows, cols, p, ps
    return codes, scales, rows, cols, None, None


def _check_out(q: Q4Matrix, rows: int, cols: int, device) -> None:
    if (q.codes is None) != (q.scales is None) or (q.codes_t is None) != (q.scales_t is None):
        raise _invalid("codes and scales go together")
    if q.codes is None and q.codes_t is None:
        raise _invalid("out has neither form")
    if q.codes is not None:
        _check_form(q.codes, q.scales, rows, cols, "out", device)
    if q.codes_t is not None:
        _check_form(q.codes_t, q.scales_t, cols, rows, "out's transpose", device)


def _source(x, dt: int, rows: int, cols: int, random, q: Q4Matrix) -> Q4SourceDesc:
    """The descriptor of a matrix whose arguments have been checked."""
    codes, codes_t = q.codes, q.codes_t
    return Q4SourceDesc(x.data_ptr(), dt, 0, rows, cols, None if random is None else random.data_ptr(),
                        None if codes is None else codes.data_ptr(), None if codes is None else q.scales.data_ptr(),
                        None if codes_t is None else codes_t.data_ptr(),
                        None if codes_t is None else q.scales_t.data_ptr())


def q4_quantize(x, transposed: bool = False, random=None, plain: bool = True, out: Optional[Q4Matrix] = None,
                stream=None) -> Q4Matrix:
    """The 4-bit form of ``x`` (bf16 or fp32, ``[..., cols]``; the leading
    dimensions are flattened) for sums along its rows (``plain``), along its
    columns (``transposed``), or both, which reads it once.  ``random``
    (``torch.uint8`` of ``x``'s shape) rounds each element by its random byte in
    place of to nearest, in both forms alike.  ``out`` takes the result, in the
    forms that it has; a matrix of other columns that round up to the same sizes
    fits."""
    import torch
    device, rows, cols = _matrix(x, "x")
    if stream is not None:
        _check_stream(device, stream)
    if random is not None:
        _check_tensor(random, "random", x.shape, torch.uint8, device)
    dt = _dtype_code(x)
    _ptr(x)
    made = out is None
    if made:
        if not plain and not transposed:
            raise _invalid("neither form is asked for")
        with _allocating(stream):
            out = Q4Matrix.empty(rows, cols, device, plain, transposed)
    else:
        _check_out(out, rows, cols, device)
    if stream is not None:
        _keep(device, stream, [t for t in out.tensors() if t is not None], made, (x, random))
    _run(load().dmuon_q4_quantize, device, stream, ctypes.byref(_source(x, dt, rows, cols, random, out)), 1)
    out.rows, out.cols = rows, cols
    return out


def q4_quantize_weights(params: Sequence, out: Optional[Sequence[Q4Matrix]] = None, transposed: bool = True,
                        stream=None) -> List[Q4Matrix]:
    """The 4-bit form of each matrix (bf16 or fp32, ``[rows, cols]``) for sums
    along its rows and, if ``transposed``, along its columns (the gradient of the
    input).  All matrices lie on one device.  ``out`` takes an earlier call's
    results and overwrites them, in the forms that they have."""
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
        if p.dim() != 2 or p.shape[1] < 1:
            raise _invalid(f"matrix {i} is not 2-D, or has no columns")
        if not p.is_cuda or p.device != device:
            raise _invalid(f"matrix {i} is on {p.device}, not on {device} (a GPU)")
        _dtype_code(p)
        _ptr(p)
    if stream is not None:
        _check_stream(device, stream)
    made = out is None
    if made:
        with _allocating(stream):
            out = [Q4Matrix.empty(p.shape[0], p.shape[1], device, True, transposed) for p in params]
    else:
        out = list(out)
        if len(out) != n:
            raise _invalid(f"{len(out)} results for {n} matrices")
        for p, q in zip(params, out):
            _check_out(q, p.shape[0], p.shape[1], device)
    arr = (Q4SourceDesc * n)()
    for i, (p, q) in enumerate(zip(params, out)):
        arr[i] = _source(p, _dtype_code(p), p.shape[0], p.shape[1], None, q)
        if stream is not None:
            _keep(device, stream, [t for t in q.tensors() if t is not None], made, (p,))
    _run(load().dmuon_q4_quantize, device, stream, arr, n)
    for p, q in zip(params, out):
        q.rows, q.cols = p.shape
    return out


def _result(out, shape, dtype, device, stream):
    """The result tensor, and whether it was made for the call."""
    import torch
    if out is None:
        with _allocating(stream):
            return torch.empty(shape, dtype=dtype or torch.bfloat16, device=device), True
    if dtype is not None and dtype != out.dtype:
        raise _invalid(f"out has dtype {out.dtype}, not {dtype}")
    _check_tensor(out, "out", shape, out.dtype, device)
    return out, False


def q4_dequantize(q: Q4Matrix, transpose: bool = False, out=None, dtype=None, stream=None):
    """The values of ``q``'s codes, ``[rows, cols]``, or of its transposed codes,
    ``[cols, rows]``: bf16 (the default) or fp32, both exact (``4 * 2^126``, which
    the types' largest values round to, becomes infinite)."""
    codes, scales, rows, cols, p, ps = _form_of(q, transpose, "q")
    device = codes.device
    if stream is not None:
        _check_stream(device, stream)
    out, made = _result(out, (rows, cols), dtype, device, stream)
    dt = _dtype_code(out)
    if p is None:
        codes, scales, p, ps = _dense_form(codes, scales, stream)
    if stream is not None:
        _keep(device, stream, (out,), made, (codes, scales))
    if cols:
        _run(load().dmuon_q4_dequantize, device, stream, p, ps, rows, cols, out.data_ptr(), dt)
    return out


def q4_matmul(a, w: Q4Matrix, transpose: bool = False, out=None, dtype=None,
              workspace: Optional[Workspace] = None, stream=None):
    """``a w^T`` (``[rows, w.rows]``) or, with ``transpose``, ``a w``
    (``[rows, w.cols]``), bf16 (the default) or fp32: exact products, fp32 sums,
    one rounding.  ``a`` is a ``Q4Matrix`` or a bf16 tensor ``[..., cols]``, whose
    leading dimensions are flattened.  ``out`` takes the result; its dtype is then
    the result's."""
    import torch
    codes, scales, outs, inner, p, ps = _form_of(w, transpose, "the weight")
    device = codes.device
    if stream is not None:
        _check_stream(device, stream)
    if isinstance(a, Q4Matrix):
        a_codes, a_scales, rows, cols, a_p, a_ps = _form_of(a, False, "a")
        on = a_codes.device
    else:
        on, rows, cols = _matrix(a, "a")
        if a.dtype != torch.bfloat16:
            raise DmuonError(_lib.ERR_UNSUPPORTED_DTYPE, f"a has dtype {a.dtype}, not torch.bfloat16")
        _ptr(a)
    if on != device:
        raise _invalid(f"a is on {on}, not on {device}")
    if cols != inner:
        raise _invalid(f"rows of {cols} columns against a weight of {inner}")
    out, made = _result(out, (rows, outs), dtype, device, stream)
    dt = _dtype_code(out)
    lib = load()
    if p is None:
        codes, scales, p, ps = _dense_form(codes, scales, stream)
    if isinstance(a, Q4Matrix):
        if a_p is None:
            a_codes, a_scales, a_p, a_ps = _dense_form(a_codes, a_scales, stream)
        need = _workspace_bytes("dmuon_q4_matmul", rows, outs, inner)
        ws, nws, keep = _scratch(need, workspace, device, stream)
        if stream is not None:
            _keep(device, stream, (out,), made, (a_codes, a_scales, codes, scales))
        _run(lib.dmuon_q4_matmul, device, stream, a_p, a_ps, rows, p, ps, outs, inner, None, out.data_ptr(), dt, ws, nws)
    else:
        need = _workspace_bytes("dmuon_q4_rows_matmul", rows, outs, inner)
        ws, nws, keep = _scratch(need, workspace, device, stream)
        if stream is not None:
            _keep(device, stream, (out,), made, (a, codes, scales))
        _run(lib.dmuon_q4_rows_matmul, device, stream, a.data_ptr(), rows, p, ps, outs, inner, out.data_ptr(), dt, ws, nws)
    return out


def q4_weight_grad(dy: Q4Matrix, x: Q4Matrix, out=None, dtype=None, base=None,
                   workspace: Optional[Workspace] = None, stream=None):
    """``base + dy^T x`` (``[dy.cols, x.cols]``): the weight gradient of
    ``y = x w^T`` from the transposed codes of both, exact products, fp32 sums, one
    rounding.  The result is ``out`` (for instance the ``grads`` entry of
    ``muon_step``) or a new tensor of ``dtype`` (``base``'s, or bf16).  ``base``
    has the result's dtype and may be ``out`` itself, which adds to the gradient
    in place."""
    codes, scales, rows, tokens, p, ps = _form_of(dy, True, "dy")
    x_codes, x_scales, outs, x_tokens, x_p, x_ps = _form_of(x, True, "x")
    device = codes.device
    if stream is not None:
        _check_stream(device, stream)
    if x_codes.device != device:
        raise _invalid(f"x is on {x_codes.device}, not on {device}")
    if tokens != x_tokens:
        raise _invalid(f"dy has {tokens} rows, x {x_tokens}")
    if base is not None:
        _check_untracked(base, "base")
        if dtype is None and out is None:
            dtype = base.dtype
    out, made = _result(out, (rows, outs), dtype, device, stream)
    if base is not None:
        _check_tensor(base, "base", (rows, outs), out.dtype, device)
    dt = _dtype_code(out)
    lib = load()
    if p is None:
        codes, scales, p, ps = _dense_form(codes, scales, stream)
    if x_p is None:
        x_codes, x_scales, x_p, x_ps = _dense_form(x_codes, x_scales, stream)
    ws, nws, keep = _scratch(_workspace_bytes("dmuon_q4_matmul", rows, outs, tokens), workspace, device, stream)
    if stream is not None:
        _keep(device, stream, (out,), made, (codes, scales, x_codes, x_scales, base))
    _run(lib.dmuon_q4_matmul, device, stream, p, ps, rows, x_p, x_ps, outs, tokens,
         base.data_ptr() if base is not None else None, out.data_ptr(), dt, ws, nws)
    return out
