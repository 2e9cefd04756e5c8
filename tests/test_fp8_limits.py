"""Argument checks of the 8-bit operators at extents whose products pass 64 bits, on the host (no GPU: every call
returns before any CUDA work)."""
import pytest

from conv_activation_epilogue_gb300 import build, mmact

P = 0x7f0000000000          # never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return mmact.load()


@pytest.mark.parametrize("M,N,K", [(1 << 22, 1 << 22, 1 << 22), (1 << 21, 1 << 22, 1 << 21), (1 << 24, 1 << 20, 1 << 20)])
def test_a_missing_weight_is_refused_whatever_the_sizes(lib, M, N, K):
    """M N K is a multiple of 2^64 here; no tensor is empty."""
    for codes, scales in ((None, P), (P, None)):
        assert lib.mmact_linear_fp8_backward(P, P, codes, scales, P, P, P, M, N, K, 1, 5, 6, 2, P, None) == mmact.MMACT_ERR_INVALID_ARG


@pytest.mark.parametrize("M,N,K", [(0, 4, 4), (4, 0, 4), (4, 4, 0)])
def test_a_missing_weight_of_an_empty_product_is_not(lib, M, N, K):
    """Nothing else is asked for and the product is empty; a null dx asks for nothing at all."""
    assert lib.mmact_linear_fp8_backward(P, P, None, None, None, None, None, M, N, K, 1, 5, 6, 2, P, None) == mmact.MMACT_OK
