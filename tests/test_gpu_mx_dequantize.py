"""Values of MXFP4 matrices in 16 bits, rows that begin anywhere: every element is written, once and
with its own value, and nothing beside them."""
import numpy as np
import pytest
import torch

import mx_reference as ref
from conv_activation_epilogue_gb300 import build, mmact
from parity import TORCH
from test_gpu_mxfp4 import host64, quantized

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    mmact.load()


@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 2), (1, 3), (2, 1), (3, 1), (5, 3), (17, 7), (2, 31), (3, 33), (4, 127), (5, 129),
                                    (3, 130), (7, 131), (129, 255), (200, 257), (77, 1001), (9, 4098), (5447, 1283), (3001, 3659)])
def test_every_element_once(rows, K, out):
    """The large ones take the form with four sets of rows in flight, the small ones the other."""
    g = torch.Generator(device="cuda").manual_seed(rows * 31 + K)
    x = torch.randn((rows, K), generator=g, device="cuda") * torch.exp2(torch.randint(-4, 5, (rows, 1), generator=g, device="cuda").float())
    codes, scales = quantized(x)
    guard = 64                                                 # untouched values on both sides (16 bytes apart at least)
    full = torch.full((rows * K + 2 * guard,), 77.0, dtype=TORCH[out], device="cuda")
    y = full[guard:guard + rows * K].view(rows, K)
    mmact.mmact_dequantize_mxfp4(codes, scales, y)
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
    want = ref.quantize(host64(x))[2]                          # up to 2^10: exact in all three types
    assert np.array_equal(host64(y), want)
    assert torch.all(full[:guard] == 77.0) and torch.all(full[guard + rows * K:] == 77.0)
