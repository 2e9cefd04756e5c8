"""Plain 64-bit implementations of the MXFP4 operators and the mixture-of-experts
layer, written from their definitions in numpy, and the error bounds that the
tests hold the kernels to.  No code is shared with the library."""
from __future__ import annotations

import math

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def tiles_of(rows: int, K: int) -> tuple[int, int]:
    return -(-rows // 128), -(-K // 128)


def scale_place(r, b, ktiles):
    return ((r // 128) * ktiles + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4


def round_e2m1(v: np.ndarray) -> np.ndarray:
    """|v| -> code 0..7: nearest, ties to the even code, saturating."""
    d = np.abs(np.abs(v)[..., None] - GRID)
    best = d.min(axis=-1, keepdims=True)
    near = d == best
    first = near.argmax(axis=-1)
    tie = near.sum(axis=-1) > 1
    return np.where(tie & (first % 2 == 1), first + 1, first).astype(np.uint8)


def quantize(x: np.ndarray) -> tuple[np.ndarray, np.ndarray, np.ndarray]:
    """x [rows, K] float64 -> (codes bytes, scale bytes tiled, values float64)."""
    rows, K = x.shape
    kb = -(-K // 32)
    pad = np.zeros((rows, kb * 32))
    pad[:, :K] = x
    blk = pad.reshape(rows, kb, 32)
    with np.errstate(invalid="ignore"):
        amax = np.abs(blk).max(axis=2)
    bad = ~np.isfinite(amax)
    _, e = np.frexp(np.where(bad, 1.0, amax))          # amax = m 2^e, m in [0.5, 1)
    b = np.where(amax > 0, np.maximum(e - 1 - 2 + 127, 0), 0)
    X = np.exp2(b.astype(np.float64) - 127)
    safe = np.where(bad[:, :, None], 0.0, blk)
    q = round_e2m1(safe / X[:, :, None])
    code = (q | (np.signbit(safe).astype(np.uint8) << 3)).astype(np.uint8)
    code[bad] = 0
    b = np.where(bad, 255, b).astype(np.uint8)
    vals = np.where(np.signbit(safe), -1.0, 1.0) * GRID[q] * X[:, :, None]
    vals[bad] = np.nan
    flat = code.reshape(rows, -1)
    packed = (flat[:, 0::2] | (flat[:, 1::2] << 4)).astype(np.uint8)
    rt, kt = tiles_of(rows, K)
    tiled = np.zeros(rt * kt * 512, dtype=np.uint8)
    tiled[scale_place(np.arange(rows)[:, None], np.arange(kb)[None, :], kt)] = b
    return packed, tiled, vals.reshape(rows, -1)[:, :K]


def values(codes: np.ndarray, tiled: np.ndarray, rows: int, K: int) -> np.ndarray:
    kb = -(-K // 32)
    kt = tiles_of(rows, K)[1]
    out = np.zeros((rows, kb * 32))
    out[:, 0::2], out[:, 1::2] = codes & 15, codes >> 4
    c = out.astype(np.int64)
    v = GRID[c & 7] * np.where(c & 8, -1.0, 1.0)
    b = tiled[scale_place(np.arange(rows)[:, None], np.arange(kb)[None, :], kt)].astype(np.float64)
    return (v * np.where(b == 255, np.nan, np.exp2(b - 127)).repeat(32, axis=1))[:, :K]


def act(z: np.ndarray, name: str, alpha: float) -> np.ndarray:
    if name == "relu":
        return np.where(z > 0, z, 0.0 * z)
    if name == "leaky_relu":
        return np.where(z > 0, z, alpha * z)
    if name == "tanh":
        return np.tanh(z)
    if name == "sigmoid":
        return 1.0 / (1.0 + np.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + np.vectorize(math.erf, otypes=[float])(z / math.sqrt(2.0)))
    if name == "silu":
        return z / (1.0 + np.exp(-z))
    return z


# The activations as the kernels evaluate them: tanh and sigmoid by the hardware's
# tanh (relative error about 2^-11), GELU by a formula good to 5.4e-7 in erf, SiLU
# by an exponential and a fast divide (a few units of 2^-23 each, taken as 2^-19).
def act_error(z: np.ndarray, name: str) -> np.ndarray:
    a = np.abs(z)
    if name in ("tanh", "sigmoid"):
        return np.full_like(a, 2.0 ** -10.9)
    if name == "gelu":
        return 3e-7 * a + 2.0 ** -21 * a
    if name == "silu":
        return 2.0 ** -19 * a
    return 2.0 ** -22 * a


SLOPE = 1.2        # the largest slope of any of them (GELU and SiLU reach about 1.13 and 1.1)


def sum_error(n: int) -> float:
    """Relative to sum |a b|: n products added in fp32 in any order, each addition rounded or
    truncated (2^-23 of the running sum at most)."""
    return (n + 2) * 2.0 ** -23


def ulp(v: np.ndarray, dtype: str) -> np.ndarray:
    mant, low = {"f32": (23, -126), "f16": (10, -14), "bf16": (7, -126)}[dtype]
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.abs(np.where(v == 0, 2.0 ** low, v))))
    return np.exp2(np.maximum(e, low) - mant)


def gemm(a: np.ndarray, b: np.ndarray, bias, name: str, alpha: float) -> tuple[np.ndarray, np.ndarray]:
    """act(a b^T + bias) and the bound on the kernel's error before its output rounding."""
    z = a @ b.T
    err = sum_error(a.shape[1] + 1) * (np.abs(a) @ np.abs(b).T + (0 if bias is None else np.abs(bias)))
    if bias is not None:
        z = z + bias
    return act(z, name, alpha), SLOPE * err + act_error(z, name)


def moe(x, router, w1, w2, top, name, alpha, gated, normalize, rb=None, b1=None, b2=None):
    """(y, experts, probs, bound on y before its rounding), everything in 64 bits."""
    T, H = x.shape
    E, I = router.shape[0], w2.shape[2]
    logits = x @ router.T + (0 if rb is None else rb)
    experts = np.argsort(-logits, axis=1, kind="stable")[:, :top]
    peak = logits.max(axis=1, keepdims=True)
    ex = np.exp(logits - peak)
    chosen = np.take_along_axis(ex, experts, axis=1)
    probs = chosen / (chosen if normalize else ex).sum(axis=1, keepdims=True)
    # a logit is off by at most this, and so a probability relatively by twice that, plus the exponentials' and the sum's roundings
    dl = sum_error(H + 1) * (np.abs(x) @ np.abs(router).T + (0 if rb is None else np.abs(rb))).max(axis=1)
    dp = 2 * dl + (E + 8) * 2.0 ** -23
    y, bound = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(top):
            e = int(experts[t, j])
            z = w1[e] @ x[t] + (0 if b1 is None else b1[e])
            dz = sum_error(H + 1) * (np.abs(w1[e]) @ np.abs(x[t]) + (0 if b1 is None else np.abs(b1[e])))
            if gated:
                a, u = act(z[:I], name, alpha), z[I:]
                h = a * u
                da = SLOPE * dz[:I] + act_error(z[:I], name)
                dh = da * np.abs(u) + (np.abs(a) + da) * dz[I:] + 2.0 ** -23 * np.abs(h)
            else:
                h = act(z, name, alpha)
                dh = SLOPE * dz + act_error(z, name)
            dh = dh + 2.0 ** -16 * np.abs(h)            # h as two bf16 halves
            o = w2[e] @ h + (0 if b2 is None else b2[e])
            # 3 (I + 1) additions: up to three products for each element of h; 2^-16 again where fp16
            # weights' low halves do not meet h's
            mag = np.abs(w2[e]) @ np.abs(h) + (0 if b2 is None else np.abs(b2[e]))
            do = np.abs(w2[e]) @ dh + (sum_error(3 * (I + 1)) + 2.0 ** -16) * mag
            y[t] += probs[t, j] * o
            bound[t] += probs[t, j] * (do + (dp[t] + (top + 2) * 2.0 ** -23) * (np.abs(o) + do))
    return y, experts, probs, bound, dp
