"""The 8-bit block products at the ends of the scales' range, and beside rows
there, against float64 products of the values that the codes stand for.  Bounds
as in test_gpu_q8."""

import numpy as np
import pytest
import torch

import newton_schulz_dmuon_amd as nsd
from test_gpu_q8 import BF16, F32, check_sum

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
