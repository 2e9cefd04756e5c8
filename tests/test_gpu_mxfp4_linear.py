"""Few rows of x, quantised inside the product's kernel, over K so long that its ring goes round
many times: bit for bit what mmact_quantize_mxfp4 and mmact_gemm_mxfp4 give on the same kernel."""
import numpy as np
import pytest
import torch

import mx_reference as ref
from conv_activation_epilogue_gb300 import build, mmact
from parity import TORCH
from test_gpu_mxfp4 import host64, quantized, spread

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    mmact.load()
    mmact.mmact_set_gemm_mxfp4_kernel(1)                       # the kernel for few rows
    yield
    mmact.mmact_set_gemm_mxfp4_kernel(0)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M", [1, 7, 8])
@pytest.mark.parametrize("N,K", [(136, 16384), (264, 20001), (10000, 8192), (10000, 8200), (9985, 8191), (10000, 1283)])
def test_few_rows_long_k(dtype, M, N, K):
    """N of 136 and 264: K shared by clusters of eight CTAs, 8 and 10 stages of 256 for each; of about
    10000: 32 stages and more for one CTA (and 6: the first turn of the ring)."""
    rng = np.random.default_rng(M * K)
    x = torch.from_numpy(spread(rng, M, K, dtype).astype(np.float32)).to(TORCH[dtype]).cuda()
    g = torch.Generator(device="cuda").manual_seed(K)
    wc, ws = quantized(torch.empty((N, K), device="cuda").normal_(0, K ** -0.5, generator=g))
    bias = torch.empty(N, device="cuda").normal_(0, 1, generator=g)
    work = torch.full((mmact.mmact_linear_mxfp4_workspace_bytes(M, K),), 0xFF, dtype=torch.uint8, device="cuda")
    got = torch.full((M, N), float("nan"), dtype=torch.float32, device="cuda")
    mmact.mmact_linear_mxfp4(x, wc, ws, bias, got, work, "leaky_relu", 0.2)
    xc, xs = quantized(x)
    want = torch.empty_like(got)
    mmact.mmact_gemm_mxfp4(xc, xs, wc, ws, bias, want, K, "leaky_relu", 0.2)
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
    assert torch.equal(got, want)
    if N == 136:                                               # and the formula, once
        w = torch.empty((N, K), dtype=torch.float32, device="cuda")
        mmact.mmact_dequantize_mxfp4(wc, ws, w)
        z, bound = ref.gemm(ref.quantize(host64(x))[2], host64(w), host64(bias), "leaky_relu", 0.2)
        assert np.all(np.abs(host64(got) - z) <= bound + ref.ulp(np.abs(z) + bound, "f32"))
