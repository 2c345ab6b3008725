"""Rounding by random bytes where rows of bytes begin at no multiple of a word: codes
and scales bit for bit, in patches of whole rows whose last words would end behind the
bytes, and beside them."""

import numpy as np
import pytest
import torch

import newton_schulz_dmuon_amd as nsd
from test_gpu_q4 import BF16, F32, check_matrix, host, values

pytestmark = pytest.mark.gpu

ROWS = [1, 7, 8, 9, 16, 40, 96, 128, 136, 168, 256, 264]
COLS = [8, 9, 15, 17, 19, 34, 67, 83, 114, 127, 131, 257, 321]


@pytest.mark.parametrize("t", ROWS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_random_bytes_at_every_edge(t, dtype):
    print(f"random bytes at edges {t} {dtype}", flush=True)
    for k in COLS:
        rng = np.random.default_rng(t * 1009 + k)
        x = values(rng, t, k, dtype)
        r = rng.integers(0, 256, (t, k)).astype(np.uint8)
        rt = torch.from_numpy(r).cuda()
        for plain, transposed in ((True, True), (True, False), (False, True)):
            q = nsd.q4_quantize(x.cuda(), transposed=transposed, plain=plain, random=rt)
            torch.cuda.synchronize()
            check_matrix(q, host(x), r, plain, transposed)


@pytest.mark.parametrize("t,k", [(4288, 114), (2208, 722), (96, 10234), (5752, 67), (856, 321)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_random_bytes_of_larger_matrices(t, k, dtype):
    print(f"random bytes {t} {k} {dtype}", flush=True)
    rng = np.random.default_rng(t + k)
    x = values(rng, t, k, dtype)
    r = rng.integers(0, 256, (t, k)).astype(np.uint8)
    q = nsd.q4_quantize(x.cuda(), transposed=True, random=torch.from_numpy(r).cuda())
    torch.cuda.synchronize()
    check_matrix(q, host(x), r)
