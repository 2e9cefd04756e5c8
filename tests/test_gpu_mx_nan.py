"""A NaN goes through every activation of the MXFP4 products and of the mixture of
experts: what the quantiser marked, and NaN in x, weights and biases."""
import numpy as np
import pytest
import torch

import mx_reference as ref
from conv_activation_epilogue_gb300 import build, mmact
from test_gpu_moe import TYPES, layer, run
from test_gpu_mxfp4 import host64, random_mx, tensor

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "leaky_relu", "tanh", "sigmoid", "gelu", "silu"]


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    mmact.load()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("mode,M", [(1, 2), (1, 140), (2, 300)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_gemm_nan_scales(act, mode, M, out):
    rng = np.random.default_rng(M)
    N, K = 200, 192
    (ac, as_, _), (bc, bs, _) = random_mx(rng, M, K), random_mx(rng, N, K)
    bs[ref.scale_place(150, 3, ref.tiles_of(N, K)[1])] = 255
    as_[ref.scale_place(1, 5, ref.tiles_of(M, K)[1])] = 255
    C = torch.empty((M, N), dtype=out, device="cuda")
    mmact.mmact_set_gemm_mxfp4_kernel(mode)
    try:
        mmact.mmact_gemm_mxfp4(ac, as_, bc, bs, None, C, K, act, 0.3)
    finally:
        mmact.mmact_set_gemm_mxfp4_kernel(0)
    want = np.zeros((M, N), dtype=bool)
    want[1, :] = want[:, 150] = True
    assert np.array_equal(np.isnan(host64(C)), want)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [5, 40])
def test_linear_nan_rows(act, M):
    rng = np.random.default_rng(M)
    N, K = 130, 320
    x = rng.normal(0, 1, (M, K))
    x[1, 7], x[3, 300] = np.inf, np.nan
    wc, ws, _ = random_mx(rng, N, K, K ** -0.5)
    work = torch.empty(mmact.mmact_linear_mxfp4_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    C = torch.empty((M, N), dtype=torch.float32, device="cuda")
    mmact.mmact_linear_mxfp4(tensor(x, "bf16"), wc, ws, None, C, work, act, 0.3)
    assert np.array_equal(np.isnan(host64(C)).all(axis=1), np.isin(np.arange(M), [1, 3]))
    assert np.array_equal(np.isnan(host64(C)).any(axis=1), np.isin(np.arange(M), [1, 3]))


@pytest.mark.parametrize("act", ACTS)
def test_a_nan_bias_of_an_empty_product(act):
    e = torch.empty(0, dtype=torch.uint8, device="cuda")
    bias = torch.tensor([1.0, float("nan"), -1.0], device="cuda")
    C = torch.empty((2, 3), dtype=torch.float32, device="cuda")
    mmact.mmact_gemm_mxfp4(e.view(2, 0), e, e.view(3, 0), e, bias, C, 0, act, 0.3)
    assert torch.isnan(C).tolist() == [[False, True, False]] * 2


@pytest.mark.parametrize("dtype,weights", TYPES)
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("act", ["relu", "leaky_relu", "gelu"])
def test_moe_nan_token_and_nan_expert(dtype, weights, gated, act):
    L = layer(8, 12, 64, 32, 6, dtype, weights, gated)
    L["b1"] = np.zeros((6, 64 if gated else 32))
    y, experts, _, _, _ = run(L, 2, dtype, weights, act, 0.3, gated=gated)
    ids = experts.cpu().numpy()
    e = int(ids[0, 0])
    L["b1"][e, 5] = np.nan                                     # one row of the up product
    got, ids2, _, _, _ = run(L, 2, dtype, weights, act, 0.3, gated=gated)
    hit = (ids == e).any(axis=1)
    assert np.array_equal(ids2.cpu().numpy(), ids)
    assert np.array_equal(np.isnan(host64(got)).all(axis=1), hit) and torch.equal(got[~hit], y[~hit])
    L["b1"][e, 5] = 0.0
    L["x"][3, 10] = np.nan
    got = run(L, 2, dtype, weights, act, 0.3, gated=gated)[0]
    assert np.array_equal(np.isnan(host64(got)).all(axis=1), np.arange(12) == 3)
    assert torch.equal(got[np.arange(12) != 3], y[np.arange(12) != 3])
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
