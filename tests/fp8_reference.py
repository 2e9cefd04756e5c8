"""Plain 64-bit implementation of the 8-bit block-scaled form, written from its definition
in numpy.  No code is shared with the library.  (Products and their error bounds are
those of mx_reference.)"""
from __future__ import annotations

import numpy as np

from mx_reference import scale_place


def _grid(exponents: int, fraction: int, bias: int, last: int) -> np.ndarray:
    one = 1 << fraction
    out = []
    for code in range(last + 1):
        e, f = code >> fraction, code & (one - 1)
        out.append((f / one) * 2.0 ** (1 - bias) if e == 0 else (1 + f / one) * 2.0 ** (e - bias))
    return np.array(out)


GRID = {"e4m3": _grid(4, 3, 7, 0x7e), "e5m2": _grid(5, 2, 15, 0x7b)}      # by code, without infinities and NaN


def tiles_of(rows: int, K: int) -> tuple[int, int]:
    return -(-rows // 128), -(-K // 512)


def pitch(K: int) -> int:
    return -(-K // 16) * 16


def nearest(a: np.ndarray, kind: str) -> np.ndarray:
    """a >= 0 -> code: nearest, ties to the even code."""
    g = GRID[kind]
    hi = np.clip(np.searchsorted(g, a), 1, len(g) - 1)       # g[hi - 1] < a <= g[hi]
    lo = hi - 1
    up, down = g[hi] - a, a - g[lo]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def quantize(x: np.ndarray, kind: str = "e4m3", square: bool = False):
    """x [rows, K] float64 -> (codes [rows, pitch] bytes, scale bytes tiled, values float64)."""
    rows, K = x.shape
    kb, rb = -(-K // 128), -(-rows // 128)
    pad = np.zeros((rb * 128, kb * 128))
    pad[:rows, :K] = x
    with np.errstate(invalid="ignore"):
        amax = np.abs(pad.reshape(rb * 128, kb, 128)).max(axis=2)
        if square:
            amax = amax.reshape(rb, 128, kb).max(axis=1).repeat(128, axis=0)
    amax = amax[:rows]
    bad = ~np.isfinite(amax)
    safe = np.where(bad, 0.0, amax)
    b = np.zeros(amax.shape)
    for i, v in np.ndenumerate(safe):
        while v / 2.0 ** (b[i] - 127) > GRID[kind][-1]:
            b[i] += 1
    X = np.exp2(b - 127).repeat(128, axis=1)[:, :K]
    z = np.where(bad.repeat(128, axis=1)[:, :K], 0.0, x)
    code = nearest(np.abs(z) / X, kind)
    vals = np.where(np.signbit(z), -1.0, 1.0) * GRID[kind][code] * X
    vals[bad.repeat(128, axis=1)[:, :K]] = np.nan
    codes = np.zeros((rows, pitch(K)), dtype=np.uint8)
    codes[:, :K] = (code | (np.signbit(z).astype(np.int64) << 7)).astype(np.uint8)
    rt, kt = tiles_of(rows, K)
    tiled = np.zeros(rt * kt * 512, dtype=np.uint8)
    tiled[scale_place(np.arange(rows)[:, None], np.arange(kb)[None, :], kt)] = np.where(bad, 255, b).astype(np.uint8)
    return codes, tiled, vals


def values(codes: np.ndarray, tiled: np.ndarray, K: int, kind: str) -> np.ndarray:
    rows, kb = codes.shape[0], -(-K // 128)
    b = tiled[scale_place(np.arange(rows)[:, None], np.arange(kb)[None, :], tiles_of(rows, K)[1])].astype(np.float64)
    X = np.where(b == 255, np.nan, np.exp2(b - 127)).repeat(128, axis=1)[:, :K]
    c = codes[:, :K].astype(np.int64)
    return GRID[kind][c & 127] * np.where(c & 128, -1.0, 1.0) * X
