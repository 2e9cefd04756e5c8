"""What the mixture-of-experts layer keeps of h, its intermediate, on the GPU: the down
product takes differences of values of h that agree in their first 16 bits, so that y
shows the bits that follow."""
import numpy as np
import pytest
import torch

import mx_reference as ref
from conv_activation_epilogue_gb300 import build, mmact
from test_gpu_moe import run
from test_gpu_mxfp4 import host64, tensor

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    mmact.load()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,I", [(1, 272), (12, 272), (24, 48), (64, 640)])
def test_h_keeps_the_bits_of_fp32(dtype, T, I):
    """h[i] = (1 + a 2^-12 + b 2^-23) s, whole a and b, the same a for h[2 r] and h[2 r + 1];
    y[r] = h[2 r] - h[2 r + 1].  Bound: h is a sum of three products and y one of two values,
    in at most three parts each (sum_error)."""
    rng = np.random.default_rng(T + I)
    H, E = I // 2, 3
    L = {"x": np.zeros((T, H)), "router": np.zeros((E, H)), "rb": np.array([0.0, 2.0, 1.0]), "b1": None, "b2": None,
         "w1": np.zeros((E, I, H)), "w2": np.zeros((E, H, I))}
    s = np.exp2(rng.integers(0, 2, T))                         # one in fp16 has 2^-23 as a subnormal
    L["x"][:, 0], L["x"][:, 1], L["x"][:, 2] = s, s * 2.0 ** -12, s * 2.0 ** -23
    a, b = rng.integers(-127, 128, (E, H)).repeat(2, axis=1), rng.integers(-127, 128, (E, I))
    L["w1"][:, :, 0], L["w1"][:, :, 1], L["w1"][:, :, 2] = 1.0, a, b
    r = np.arange(H)
    L["w2"][:, r, 2 * r], L["w2"][:, r, 2 * r + 1] = 1.0, -1.0
    y, experts, _, _, _ = run(L, 1, dtype, dtype, "none", gated=False)
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
    assert torch.all(experts == 1)
    want = s[:, None] * (b[1, 0::2] - b[1, 1::2]) * 2.0 ** -23
    mag = 1.0 + 127 * 2.0 ** -12 + 127 * 2.0 ** -23
    bound = s[:, None] * mag * 2.0 * (ref.sum_error(3) + ref.sum_error(6))
    err = np.abs(host64(y) - want)
    assert np.all(err <= bound + ref.ulp(np.abs(want) + bound, dtype)), float((err / bound).max())


def sum_bound(products: np.ndarray, instructions: int) -> np.ndarray:
    """Bound on a sum of positive products along the last axis that is taken in pieces of 32: each
    piece by that many instructions of the tensor core, each off by at most two units of 2^-23 of the
    piece, each running sum by half a unit."""
    n = products.shape[-1]
    assert n % 32 == 0
    running = products.reshape(*products.shape[:-1], n // 32, 32).sum(axis=-1).cumsum(axis=-1)
    return 2.0 ** -23 * (2 * instructions * running[..., -1] + 0.5 * running.sum(axis=-1))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T", [1, 12, 24])
@pytest.mark.parametrize("product", ["up", "down"])
def test_long_sums_are_not_truncated(dtype, T, product):
    """4096 products of one sign, and a bias of their sum, negative, rounded to fp32: what is left is
    the sum's error (a sum that is truncated in every step loses 100 to 200 units of 2^-23)."""
    K, R = 4096, 64
    rng = np.random.default_rng(T)
    a = host64(tensor(rng.uniform(0.5, 2.0, K), dtype))
    w = host64(tensor(rng.uniform(0.5, 2.0, (R, K)), dtype))
    exact = w @ a
    bias = -exact.astype(np.float32).astype(np.float64)
    if product == "up":
        H, I = K, R
        L = {"x": np.tile(a, (T, 1)), "w1": w[None], "b1": bias[None], "w2": np.zeros((1, H, I)), "b2": None}
        L["w2"][0, np.arange(R), np.arange(R)] = 1.0
        instructions = 2
    else:
        H, I = R, K
        L = {"x": np.zeros((T, H)), "w1": np.zeros((1, I, H)), "b1": None, "w2": w[None], "b2": bias[None]}
        L["x"][:, 0], L["w1"][0, :, 0] = 1.0, a
        instructions = 10                                      # h in three parts, an fp16 weight in two
    L["router"], L["rb"] = np.zeros((1, H)), None
    y = run(L, 1, dtype, dtype, "none", gated=False)[0]
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
    want, bound = exact + bias, sum_bound(w * a, instructions)
    got = host64(y)[:, :R]
    lim = bound + ref.ulp(np.abs(want) + bound, dtype)
    assert np.all(np.abs(got - want) <= lim), float((np.abs(got - want) / lim).max())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T", [2, 20])
def test_infinite_h_and_weights_give_what_the_formula_gives(dtype, T):
    """h from a bias of infinities (an h that overflowed), weights that are infinite: y is the
    infinity of the formula, or NaN where that has 0 x inf or inf - inf."""
    H, I, inf = 16, 24, np.inf
    L = {"x": np.zeros((T, H)), "router": np.zeros((1, H)), "rb": None, "w1": np.zeros((1, I, H)), "b1": np.zeros((1, I)),
         "w2": np.zeros((1, H, I)), "b2": None}
    L["x"][:, 0] = 1.0
    L["w1"][0, :, 0] = np.array([1.0, -2.0, 0.0, 0.5, 1.2578125, -1.0] * 4)       # h, with b1
    w2 = L["w2"][0]
    w2[:, 0] = np.arange(H) - 3.0
    w2[0, 0], w2[1, 0], w2[2, 1], w2[3, 1], w2[4, 4] = inf, -inf, inf, -inf, inf
    w2[5, 0], w2[5, 1] = inf, inf                              # inf - inf
    w2[6, 2] = inf                                             # inf x 0
    w2[7, 1], w2[7, 4] = -inf, inf
    for case in range(3):
        if case == 1:                                          # from here on two values of h are infinite
            L["b1"][0, 8], L["b1"][0, 9] = inf, -inf
        if case == 2:
            w2[:, 8], w2[:, 9] = 1.0 / 3.0, -0.125              # f16: with lo halves
            w2[8, 9], w2[9, 8], w2[10, 8], w2[10, 9] = 0.0, -100.3, inf, -inf
            w2[11, 8], w2[11, 9] = 3.0e-5, -60001.0
        for k in ("w1", "w2"):
            L[k] = host64(tensor(L[k], dtype))
        w2 = L["w2"][0]
        y = host64(run(L, 1, dtype, dtype, "none", gated=False)[0])
        with np.errstate(invalid="ignore"):
            h = L["w1"][0] @ L["x"][0] + L["b1"][0]
            want = (w2 * h).sum(axis=1)
        assert np.isnan(want).any() and np.isinf(want).any() == (case != 1)
        for t in range(T):
            assert np.array_equal(np.isnan(y[t]), np.isnan(want)), (case, t, y[t], want)
            bad = ~np.isfinite(want)
            assert np.array_equal(y[t][bad & ~np.isnan(want)], want[bad & ~np.isnan(want)])
            assert np.all(np.abs(y[t][~bad] - want[~bad]) <= ref.ulp(want[~bad], dtype))
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
