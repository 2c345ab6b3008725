"""4-bit block products whose sums lie in fp32's subnormal range, and operands at its
edge.

Operands are codes with scales 2^e, 2^(e + 1) and 2^(e + 2) and integers times 2^e,
so every product and sum is a multiple of 2^(ea + eb - 2) (of half of it where bf16
rows' sums are halved, whose codes are multiples of a half) below 2^24 of them
(asserted): fp32 holds it exactly, also below 2^-126, if nothing is flushed to zero
and the unit is at least 2^-149.  The result is then the exact sum rounded once."""

import numpy as np
import pytest
import torch

import newton_schulz_dmuon_amd as nsd
from oracle import q4 as ref
from test_gpu_q4 import BF16, F32, device, host

pytestmark = pytest.mark.gpu

# (rows, outputs, columns): streamed, small tiles, both large tiles, split along the sum
SIZES = [(1, 130, 300), (5, 4100, 1100), (16, 300, 2000), (70, 500, 520), (200, 640, 1024), (600, 4100, 700), (1500, 1000, 3001),
         (2309, 3424, 133)]
# the operands' exponents: sums of 2^-146 to about 2^-132; over both sides of 2^-126;
# the weight at its smallest scale, whose expansion to bf16 is subnormal; rows that
# are subnormal as bf16 values
EXPONENTS = [(-73, -73), (-66, -66), (100, -125), (-40, -100)]


def codes(rng, rows, cols, e):
    cp = ref.up(cols, ref.PAD)
    c = rng.integers(0, 16, (rows, cp)).astype(np.uint8)
    c[:, cols:] = 0
    s = rng.integers(127 + e, 130 + e, (cp // 32, ref.up(rows, 16))).astype(np.uint8)
    return device(c, s), torch.from_numpy(ref.values(c, s)[:, :cols]).cuda()


def check(got, a, b, unit, base=None):
    """a b^T (+ base), exact: their products are multiples of the unit."""
    assert (a.abs() @ b.t().contiguous().abs()).max().item() + (0 if base is None else base.abs().max().item()) < 2.0 ** 24 * unit
    want = a @ b.t().contiguous()
    if base is not None:
        want = want + base.double()
    want = want.cpu().to(F32)  # exact
    want = want.to(got.dtype).double().numpy()
    g = host(got)
    assert np.array_equal(g, want), (got.dtype, np.argwhere(g != want)[:4], g[g != want][:4], want[g != want][:4])
    return np.abs(want)


@pytest.mark.parametrize("t,n,k", SIZES)
@pytest.mark.parametrize("ea,eb", EXPONENTS)
def test_small_sums_are_exact(t, n, k, ea, eb):
    print(f"small sums {t} {n} {k} {ea} {eb}", flush=True)
    rng = np.random.default_rng(t + n + k)
    a, av = codes(rng, t, k, ea)
    b, bv = codes(rng, n, k, eb)
    w = nsd.Q4Matrix(n, k, *b)
    x = torch.from_numpy(np.rint(rng.standard_normal((t, k)) * 3) * 2.0 ** ea).to(BF16).cuda()
    unit = 2.0 ** (ea + eb - 2)
    for dtype in (BF16, F32):
        size = check(nsd.q4_matmul(nsd.Q4Matrix(t, k, *a), w, dtype=dtype), av, bv, unit)
        if dtype == F32 and ea + eb < -130:
            assert ((size > 0) & (size < 2.0 ** -126)).any()
        check(nsd.q4_matmul(x, w, dtype=dtype), x.double(), bv, unit)
        # onto a base of the same size, as a weight gradient over k tokens
        base = torch.from_numpy(np.rint(rng.standard_normal((t, n)) * 99) * 4 * unit).to(dtype).cuda()
        if ea + eb < -140 and dtype == BF16:
            base = base * 0  # bf16 holds no multiple of the unit there
        got = nsd.q4_weight_grad(nsd.Q4Matrix(k, t, None, None, *a), nsd.Q4Matrix(k, n, None, None, *b), base=base)
        check(got, av, bv, unit, base)


@pytest.mark.parametrize("t,n,k", SIZES)
def test_subnormal_rows(t, n, k):
    """bf16's subnormal numbers as rows, against weights of 2^20."""
    print(f"subnormal rows {t} {n} {k}", flush=True)
    rng = np.random.default_rng(t + k)
    b, bv = codes(rng, n, k, 20)
    x = torch.from_numpy(np.rint(rng.standard_normal((t, k)) * 3) * 2.0 ** -133).to(BF16).cuda()
    assert x.any()
    for dtype in (BF16, F32):
        check(nsd.q4_matmul(x, nsd.Q4Matrix(n, k, *b), dtype=dtype), x.double(), bv, 2.0 ** (20 - 133 - 2))
