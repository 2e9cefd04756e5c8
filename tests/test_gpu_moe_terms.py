"""The mixture with MXFP4 experts holds x and h as sums of eight 4-bit terms: here the last
ones show.  One value of every block of 32 is much larger than the rest, so that the rest are what
the last terms hold, and the products only pick single values, so that nothing hides them."""
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


def picking(rng, E, rows, K):
    """One value in each row, +-1, 1.5 or 2 times a power of two; block b's places only take from block b."""
    assert rows == K
    w = np.zeros((E, rows, K))
    for e in range(E):
        for k0 in range(0, K, 32):
            n = min(32, K - k0)
            w[e, np.arange(k0, k0 + n), k0 + rng.permutation(n)] = rng.choice([-2.0, -1.0, 1.0, 1.5], n) * np.exp2(rng.integers(-3, 4))
    return w


def mxfp4(L, name, w):
    E, rows, K = w.shape
    L[name + "_codes"], L[name + "_scales"], v = ref.quantize(w.reshape(E * rows, K))
    L[name] = v.reshape(E, rows, K)
    assert np.array_equal(L[name], w)                          # the picked values are exact in 4 bits


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,H,top", [(1, 64, 1), (3, 520, 2), (17, 264, 1), (64, 160, 3), (40, 1032, 1)])
def test_small_values_beside_large_ones(dtype, gated, T, H, top):
    """y = w2 (w1 x) of single values (times 1 where gated).  Bound, in units of 2^-23: one of the block's largest |x| for the terms of x, one of
    the largest |h| for those of h, and for the sums of eight terms each, which add up to 4/3 of
    the value, ten additions (sum_error)."""
    rng = np.random.default_rng(T + H)
    E, I = 4, H
    bits = {"bf16": 8, "f16": 11}[dtype]
    low = 24 - bits                                            # the last bit of the smallest is 2^-23 of the largest
    x = rng.uniform(1.0, 2.0, (T, H)) * np.exp2(-rng.integers(0, low, (T, H))) * rng.choice([-1.0, 1.0], (T, H))
    x[:, 0::32] = rng.uniform(1.9, 2.0, x[:, 0::32].shape)
    x *= np.exp2(rng.integers(-1, 4, (T, (H + 31) // 32))).repeat(32, axis=1)[:, :H]
    x = host64(tensor(x, dtype))
    L = {"x": x, "router": np.zeros((E, H)), "rb": np.array([0.0, 3.0, 1.0, 2.0]), "b1": None, "b2": None}
    w1, w2 = picking(rng, E, I, H), picking(rng, E, H, I)
    up = np.concatenate([w1, np.zeros_like(w1)], axis=1) if gated else w1
    mxfp4(L, "w1", up)
    mxfp4(L, "w2", w2)
    if gated:                                                  # the up half is a bias of 1
        L["b1"] = np.concatenate([np.zeros((E, I)), np.ones((E, I))], axis=1)
    y, experts, probs, _, _ = run(L, top, dtype, "mxfp4", "none", gated=gated)
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
    order = [1, 3, 2][:top]
    assert experts.tolist() == [order] * T
    p = host64(probs)                                          # their own error is no matter here
    largest = lambda v: np.abs(np.pad(v, ((0, 0), (0, -v.shape[1] % 32)))).reshape(T, -1, 32).max(axis=2).repeat(32, axis=1)[:, : v.shape[1]]  # noqa: E731
    u, want, bound = 2.0 ** -23, np.zeros((T, H)), np.zeros((T, H))
    for j, e in enumerate(order):
        h = x @ w1[e].T
        dh = u * (largest(x) @ np.abs(w1[e]).T) + ref.sum_error(8) * 4.0 / 3.0 * np.abs(h)
        o = h @ w2[e].T
        do = dh @ np.abs(w2[e]).T + u * (largest(np.abs(h) + dh) @ np.abs(w2[e]).T) + ref.sum_error(8) * 4.0 / 3.0 * np.abs(o)
        want += p[:, j: j + 1] * o
        bound += p[:, j: j + 1] * (do + (top + 2) * u * np.abs(o))
    got = host64(y)
    err, lim = np.abs(got - want), bound + ref.ulp(np.abs(want) + bound, dtype)
    assert np.all(err <= lim), float((err / lim).max())
    # six terms of x would leave several times the bound
    r = x.copy()
    for _ in range(6):
        r = r - rounded_once(r)
    assert T == 1 or np.any(np.abs(r) > 6 * u * largest(x))


def rounded_once(r):
    """The first term of r: each block of 32 to the 4-bit grid times the smallest power of two that holds it."""
    T, K = r.shape
    b = np.pad(r, ((0, 0), (0, -K % 32))).reshape(T, -1, 32)
    top = np.abs(b).max(axis=2, keepdims=True)
    X = np.exp2(np.ceil(np.log2(np.where(top > 0, top, 1.0) / 6.0)))
    return (np.sign(b) * ref.GRID[ref.round_e2m1(b / X)] * X).reshape(T, -1)[:, :K]
