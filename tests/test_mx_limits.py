"""Sizes of the mixture of experts near the end of 32-bit counting, on the host (no GPU)."""
import ctypes

import pytest

from conv_activation_epilogue_gb300 import build, mmact


@pytest.fixture(scope="module")
def lib():
    build.build()
    return mmact.load()


@pytest.mark.parametrize("H,I,ok", [((1 << 31) - 8, 8, False), ((1 << 31) - 256, 8, False), ((1 << 31) - 512, 8, True),
                                    (8, (1 << 30) - 8, False), (8, (1 << 30) - 128, False), (8, (1 << 30) - 256, True)])
def test_extents_that_do_not_round_up_in_32_bits_are_refused(lib, H, I, ok):
    """H and I are padded to multiples of 256, and a tile's rows run up to 128 past the last."""
    out = ctypes.c_int64(-1)
    got = lib.mmact_moe_workspace_bytes(1, H, I, 1, 1, ctypes.byref(out))
    assert got == (mmact.MMACT_OK if ok else mmact.MMACT_ERR_UNSUPPORTED)
    assert (out.value > 8 * H) if ok else out.value == -1
