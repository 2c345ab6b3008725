"""4-bit products in the kernels that the other size lists do not reach: large tiles of
which all are split along the sum, and bf16 rows of whole 16-byte chunks in small tiles
that are."""

import pytest

import test_gpu_q4 as q4

pytestmark = pytest.mark.gpu

MORE_SIZES = [(1738, 1195, 18225), (2224, 2177, 27432)]
MORE_CHUNK_SIZES = [(9, 1, 14928)]


@pytest.mark.parametrize("t,n,k", MORE_SIZES)
def test_more_kernels(t, n, k):
    q4.test_every_kernel(t, n, k)


@pytest.mark.parametrize("t,n,k", MORE_CHUNK_SIZES)
def test_more_rows_of_whole_chunks(t, n, k):
    q4.test_rows_of_whole_chunks(t, n, k)
