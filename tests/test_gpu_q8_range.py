"""The 8-bit block products at the ends of the scales' range, and beside rows
there, against float64 products of the values that the codes stand for.  Bounds
as in test_gpu_q8."""

import numpy as np
import pytest
import torch

import newton_schulz_dmuon_amd as nsd
from test_gpu_q8 import BF16, CUT, F32, check_sum

pytestmark = pytest.mark.gpu


def power(byte):
    """2^(byte - 127) as float64."""
    return (byte.to(torch.int64) - 127 + 1023 << 52).view(torch.float64)


def row_values(q):
    t = q.codes.shape[0]
    return (q.codes.double() * power(q.scales[:, :t].t()).repeat_interleave(128, 1))[:, :q.cols].contiguous()


def check_weight_grad(dy, q, what):
    xv, dv = row_values(q), dy.double().t().contiguous()
    want, mag = (dv @ xv).cpu().numpy(), (dv.abs() @ xv.abs()).cpu().numpy()
    assert np.isfinite(want).all()
    for dtype in (BF16, F32):
        check_sum(nsd.q8_weight_grad(dy, q, dtype=dtype), want, mag, dy.shape[0], (what, dtype))


# (rows that leave one to three rows in the last word of a scale table, and end
# inside a step; every tile shape of the weight gradient)
LAST_ROWS = [(2, 130, 300), (3, 130, 300), (67, 130, 300), (70, 1846, 2187), (1602, 2049, 2051), (450, 8200, 2100)]


@pytest.mark.parametrize("t,n,k", LAST_ROWS)
def test_a_large_row_beside_the_last(t, n, k):
    """A row near fp32's largest value next to an ordinary last row: its scale
    reaches its own codes only."""
    print(f"large row beside the last {t} {n} {k}", flush=True)
    torch.manual_seed(t)
    x = torch.randn(t, k, device="cuda")
    x[t - 2] = 0
    x[t - 2, 0] = 3.0e38
    dy = 0.01 * torch.randn(t, n, device="cuda")
    dy[t - 2] *= 2.0 ** -60
    q = nsd.q8_quantize(x)
    assert q.scales[0, t - 2] == 247 and (q.codes[t - 1].float().abs() >= 256).any()
    check_weight_grad(dy.to(BF16), q, (t, n, k))


@pytest.mark.parametrize("t,n,k", [(1, 130, 300), (65, 130, 300), (70, 1846, 2187)])
def test_bytes_behind_the_last_row_are_not_read_as_scales(t, n, k):
    print(f"bytes behind the last row {t} {n} {k}", flush=True)
    torch.manual_seed(t)
    q = nsd.q8_quantize(torch.randn(t, k, device="cuda"))
    q.scales[:, t:] = 255
    check_weight_grad((0.01 * torch.randn(t, n, device="cuda")).to(BF16), q, (t, n, k))


def weight_values(q, transpose):
    codes, scales = (q.codes_t, q.scales_t) if transpose else (q.codes, q.scales)
    n, k = (q.cols, q.rows) if transpose else (q.rows, q.cols)
    s = power(scales).repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)
    return (codes.double() * s)[:, :k].t().contiguous()


def check_product(a, w, transpose, what):
    av, wv = row_values(a), weight_values(w, transpose)
    want, mag = (av @ wv).cpu().numpy(), (av.abs() @ wv.abs()).cpu().numpy()
    assert np.isfinite(want).all()
    for dtype in (BF16, F32):
        check_sum(nsd.q8_matmul(a, w, transpose=transpose, dtype=dtype), want, mag, a.cols, (what, dtype),
                  CUT if dtype == BF16 else 0.0)


# (the streaming kernel's block shapes and the tiles)
EXTREME_PRODUCTS = [(1, 300, 700), (24, 300, 700), (60, 8200, 260), (257, 520, 1030), (1505, 2801, 131), (2309, 3424, 260)]


@pytest.mark.parametrize("t,n,k", EXTREME_PRODUCTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("other", [0.0, 2.0 ** -100])
@pytest.mark.parametrize("transpose", [False, True])
def test_lowest_values_in_a_product(t, n, k, dtype, other, transpose):
    """Columns of the type's lowest value (code 256 at 2^120, more than bf16 or
    fp32 hold) against weights of zero, or small enough for a finite result; and
    the other way round."""
    print(f"lowest values {t} {n} {k} {dtype} {other} {transpose}", flush=True)
    torch.manual_seed(t)
    last = (k - 1) // 128 * 128  # the last block's columns
    lowest = torch.finfo(dtype).min
    x, w = torch.randn(t, k, device="cuda"), 0.02 * torch.randn(n, k, device="cuda")
    x[:, last::2], w[:, last:] = lowest, w[:, last:] * other
    y, v = torch.randn(t, k, device="cuda"), 0.02 * torch.randn(n, k, device="cuda")
    y[:, last:], v[:, last::2] = y[:, last:] * other, lowest
    for a, b in ((x, w), (y, v)):
        b = b.t().contiguous() if transpose else b
        q, p = nsd.q8_quantize(a.to(dtype)), nsd.q8_quantize_weights([b.to(dtype)])[0]
        assert bool((q.scales == 247).any() | (p.scales == 247).any())
        check_product(q, p, transpose, (t, n, k))


@pytest.mark.parametrize("t,n,k", LAST_ROWS + [(64, 130, 300)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("other", [0.0, 2.0 ** -100])
def test_lowest_values_in_a_weight_grad(t, n, k, dtype, other):
    """Rows with the type's lowest value whose gradient is zero, or small."""
    print(f"lowest values in a gradient {t} {n} {k} {dtype} {other}", flush=True)
    torch.manual_seed(t)
    x = torch.randn(t, k, device="cuda")
    dy = 0.01 * torch.randn(t, n, device="cuda")
    x[1::3, ::5] = torch.finfo(dtype).min
    x[t - 1, k - 1] = torch.finfo(dtype).min
    dy[1::3] *= other
    dy[t - 1] *= other
    check_weight_grad(dy.to(BF16), nsd.q8_quantize(x.to(dtype)), (t, n, k))


def test_smallest_codes_are_kept():
    """Blocks at the smallest scale, 2^-117, down to the code 2^-9, against
    operands large enough for an ordinary result: an expansion or product that
    flushed subnormals would lose them."""
    print("smallest codes", flush=True)
    torch.manual_seed(3)
    for t, n, k in ((5, 140, 260), (300, 700, 390), (1505, 2801, 131)):
        small = torch.randint(-7, 8, (t, k), device="cuda").float() * 2.0 ** -126
        q = nsd.q8_quantize(small)
        assert (q.scales == 10).all()
        w = nsd.q8_quantize_weights([torch.randn(n, k, device="cuda") * 2.0 ** 110])[0]
        check_product(q, w, False, (t, n, k))
        p = nsd.q8_quantize_weights([torch.randint(-7, 8, (n, k), device="cuda").float() * 2.0 ** -126])[0]
        check_product(nsd.q8_quantize(torch.randn(t, k, device="cuda") * 2.0 ** 110), p, False, (t, n, k))
        check_weight_grad((torch.randn(t, n, device="cuda") * 2.0 ** 110).to(BF16), q, (t, n, k))
