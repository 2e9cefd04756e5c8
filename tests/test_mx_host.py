"""MXFP4 and mixture-of-experts entry points on the host: sizes and refusals (no GPU:
every call returns before any CUDA work), and pins of the plain 64-bit implementation
that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

import mx_reference as ref
from conv_activation_epilogue_gb300 import build, mmact

E, U, OK = mmact.MMACT_ERR_INVALID_ARG, mmact.MMACT_ERR_UNSUPPORTED, mmact.MMACT_OK
P = 0x7f0000000000          # never dereferenced
MIS = P + 8


@pytest.fixture(scope="module")
def lib():
    build.build()
    return mmact.load()


def test_sizes(lib):
    assert mmact.mmact_mxfp4_size(0, 0) == (0, 0)
    assert mmact.mmact_mxfp4_size(1, 1) == (16, 512)
    assert mmact.mmact_mxfp4_size(128, 128) == (128 * 64, 512)
    assert mmact.mmact_mxfp4_size(129, 129) == (129 * 80, 4 * 512)
    assert mmact.mmact_mxfp4_size(8192, 8192) == (8192 * 4096, 64 * 64 * 512)
    assert mmact.mmact_linear_mxfp4_workspace_bytes(3, 33) == 512 + 512
    assert mmact.mmact_linear_mxfp4_workspace_bytes(64, 256) == 64 * 128 + 2 * 512
    for rows, K in ((-1, 4), (4, -1), (1 << 31, 4)):
        with pytest.raises(mmact.MmactError):
            mmact.mmact_mxfp4_size(rows, K)
    out = ctypes.c_int64(-3)
    assert lib.mmact_mxfp4_size(4, 4, None, ctypes.byref(out)) == E
    assert lib.mmact_linear_mxfp4_workspace_bytes(4, -4, ctypes.byref(out)) == E
    assert lib.mmact_moe_workspace_bytes(4, 64, 64, 8, 9, ctypes.byref(out)) == U
    assert lib.mmact_moe_workspace_bytes(4, 64, 64, 8, 2, None) == E
    assert out.value == -3
    assert mmact.mmact_moe_workspace_bytes(64, 4096, 2048, 128, 8) > 64 * 8 * (4096 * 4 + 2 * 2048 * 2)


def test_quantize_host_validation(lib):
    q = lambda x=P, c=P, s=P, r=4, k=64, d=1: lib.mmact_quantize_mxfp4(x, c, s, r, k, d, 0, None)  # noqa: E731
    d = lambda c=P, s=P, y=P, r=4, k=64, t=1: lib.mmact_dequantize_mxfp4(c, s, y, r, k, t, None)  # noqa: E731
    for f in (q, d):
        assert f(None) == E
        assert f(r=-1) == E
        assert f(k=1 << 31) == E
        assert f(MIS) == U
        assert f(None, r=0) == OK
        assert f(None, k=0) == OK
    assert q(c=None) == E and q(s=None) == E and q(c=MIS) == U and q(s=MIS) == U
    assert q(d=3) == E and q(d=4) == E and d(t=3) == E
    assert d(y=MIS) == U


def gemm(lib, ac=P, as_=P, bc=P, bs=P, bias=None, C=P, M=4, N=4, K=64, cd=1, act=0):
    return lib.mmact_gemm_mxfp4(ac, as_, bc, bs, bias, C, M, N, K, cd, act, ctypes.c_float(0), None)


def linear(lib, x=P, wc=P, ws=P, bias=None, C=P, M=4, N=4, K=64, xd=1, cd=1, act=0, work=P):
    return lib.mmact_linear_mxfp4(x, wc, ws, bias, C, M, N, K, xd, cd, act, ctypes.c_float(0), work, None)


def test_product_host_validation(lib):
    for name in ("ac", "as_", "bc", "bs", "C"):
        assert gemm(lib, **{name: None}) == E
        assert gemm(lib, **{name: MIS}) == U
    for name in ("x", "wc", "ws", "C", "work"):
        assert linear(lib, **{name: None}) == E
        assert linear(lib, **{name: MIS}) == U
    for f in (gemm, linear):
        assert f(lib, M=-1) == E
        assert f(lib, N=1 << 31) == E
        assert f(lib, cd=3) == E
        assert f(lib, act=7) == E
        assert f(lib, act=-1) == E
        assert f(lib, bias=P + 2) == E
        assert f(lib, M=0) == OK
        assert f(lib, N=0) == OK
    assert linear(lib, xd=3) == E
    # more output tiles than are counted in 32 bits
    assert gemm(lib, M=(1 << 31) - 1, N=(1 << 31) - 1) == U


def moe(lib, x=P, router=P, rb=None, w1=P, s1=None, b1=None, w2=P, s2=None, b2=None, y=P, ids=P, probs=P, T=2, H=64,
        I=32, n=8, top=2, xd=1, wd=1, act=6, work=P):
    return lib.mmact_moe(x, router, rb, w1, s1, b1, w2, s2, b2, y, ids, probs, T, H, I, n, top, xd, wd, act,
                         ctypes.c_float(0), 1, 1, work, None)


def test_moe_host_validation(lib):
    for name in ("x", "router", "w1", "w2", "y", "ids", "probs", "work"):
        assert moe(lib, **{name: None}) == E
    for name in ("x", "router", "w1", "w2", "y", "work"):
        assert moe(lib, **{name: MIS}) == U
    for name in ("rb", "b1", "b2", "ids", "probs"):
        assert moe(lib, **{name: P + 2}) == E
    assert moe(lib, wd=4) == E                               # MXFP4 weights need their scales
    assert moe(lib, wd=4, s1=P, s2=MIS) == U
    assert moe(lib, wd=0) == U                               # fp16 weights with bf16 x
    assert moe(lib, wd=2) == U
    assert moe(lib, xd=2) == E
    assert moe(lib, wd=5) == E
    assert moe(lib, act=7) == E
    assert moe(lib, T=-1) == E
    assert moe(lib, T=65) == U
    assert moe(lib, H=60) == U
    assert moe(lib, I=0) == U
    assert moe(lib, top=9) == U
    assert moe(lib, n=513) == U
    assert moe(lib, n=500, top=17) == U
    assert moe(lib, T=0, x=None, y=None) == OK


def test_kernel_mode_validation(lib):
    for bad in (-1, 3):
        assert lib.mmact_set_gemm_mxfp4_kernel(bad) == E
    for good in (1, 2, 0):
        assert lib.mmact_set_gemm_mxfp4_kernel(good) == OK


def test_silu_belongs_to_the_new_operators_only(lib):
    assert lib.mmact_gemm(P, P, None, P, 64, 64, 64, 1, 1, mmact.ACT["silu"], ctypes.c_float(0), None) == E


def test_reference_rounding_pins():
    # a block whose largest value is 6: X = 1, so the grid and its ties stand as they are
    x = np.zeros((1, 32))
    x[0, :12] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.2, -0.26, 7.9, 5.01]
    c, s, v = ref.quantize(x)
    assert v[0, :12].tolist() == [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 0.0, -0.5, 6.0, 6.0]
    assert s[0] == 127 and np.count_nonzero(s) == 1
    assert c[0, 0] == 0x07 and c[0, 4] == 0x98        # 6 and 0; -0 (low half) and -0.5
    # powers of two: largest 2^-3 -> X = 2^-5
    c, s, v = ref.quantize(np.full((1, 40), 2.0 ** -3))
    assert s[0] == s[1] == 122 and np.all(v == 2.0 ** -3) and c.shape == (1, 32) and not c[0, 20:].any()
    assert np.array_equal(ref.values(c, s, 1, 40), v)


def test_reference_scale_tiles():
    # row 130 (tile 1, lane 2), block 5 (tile 1, byte 1) of a [200, 200] matrix: tile [1][1]
    assert ref.scale_place(130, 5, 2) == (1 * 2 + 1) * 512 + 2 * 16 + 0 + 1
    assert ref.scale_place(65, 0, 1) == 1 * 16 + 2 * 4
    seen = {ref.scale_place(r, b, 2) for r in range(256) for b in range(8)}
    assert seen == set(range(4 * 512))


def test_reference_moe_pin():
    # two experts that scale by 2 and by -1 (identity-like weights), one token: logits 1 and 0
    H = I = 8
    x = np.zeros((1, H))
    x[0, 0] = 1.0
    router = np.zeros((2, H))
    router[1, 0] = 1.0
    w1 = np.stack([np.eye(I), np.eye(I)])
    w2 = np.stack([2 * np.eye(H), -np.eye(H)])
    y, ids, p, bound, _ = ref.moe(x, router, w1, w2, 2, "none", 0.0, False, True)
    e = np.exp(1.0)
    assert ids.tolist() == [[1, 0]]
    assert np.allclose(p, [[e / (1 + e), 1 / (1 + e)]])
    assert np.allclose(y[0, 0], (-e + 2) / (1 + e)) and not y[0, 1:].any()
    assert 0 < bound[0, 0] < 1e-3
