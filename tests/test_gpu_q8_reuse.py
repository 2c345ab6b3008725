"""Results of the 8-bit block products that are passed in to be overwritten."""

import pytest
import torch

import newton_schulz_dmuon_amd as nsd
from test_gpu_q8 import BF16, F32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("before,after", [(250, 256), (256, 250), (1, 128), (300, 300)])
def test_weights_of_another_width(before, after):
    """Widths that round up to the same 128, without transposed codes: the
    overwritten weight has the new matrix's columns."""
    print(f"another width {before} {after}", flush=True)
    torch.manual_seed(before)
    old, new = (torch.randn(130, c, device="cuda").to(BF16) for c in (before, after))
    x8 = nsd.q8_quantize(torch.randn(9, after, device="cuda").to(BF16))
    fresh = nsd.q8_quantize_weights([new], transposed=False)
    out = nsd.q8_quantize_weights([old], transposed=False)
    got = nsd.q8_quantize_weights([new], out=out)
    assert got[0] is out[0] and (got[0].rows, got[0].cols) == (130, after)
    assert torch.equal(nsd.q8_matmul(x8, got[0], dtype=F32), nsd.q8_matmul(x8, fresh[0], dtype=F32))
    if before != after:
        with pytest.raises(nsd.DmuonError):
            nsd.q8_matmul(nsd.q8_quantize(torch.randn(9, before, device="cuda")), got[0])


def test_weights_that_do_not_know_their_columns():
    """Codes without transposed ones and without cols: told by the matrix that
    is written."""
    print("unknown columns", flush=True)
    w = torch.randn(130, 200, device="cuda")
    q = nsd.Q8Weight(torch.empty(130, 256, dtype=torch.float8_e4m3fn, device="cuda"),
                     torch.empty(2, 2, dtype=torch.uint8, device="cuda"))
    assert q.cols == 256
    nsd.q8_quantize_weights([w], out=[q])
    x8 = nsd.q8_quantize(torch.randn(3, 200, device="cuda"))
    assert torch.equal(nsd.q8_matmul(x8, q), nsd.q8_matmul(x8, nsd.q8_quantize_weights([w])[0]))
