"""8-bit entry points on the host: sizes and refusals (no GPU: every call returns before
any CUDA work), and pins of the plain 64-bit implementation that the GPU tests use."""
import ctypes

import numpy as np
import pytest
import torch

import fp8_reference as ref
from conv_activation_epilogue_gb300 import build, mmact

E, U, OK = mmact.MMACT_ERR_INVALID_ARG, mmact.MMACT_ERR_UNSUPPORTED, mmact.MMACT_OK
P = 0x7f0000000000          # never dereferenced
MIS = P + 8
BIG = (1 << 31) - 1


@pytest.fixture(scope="module")
def lib():
    build.build()
    return mmact.load()


def test_sizes(lib):
    assert mmact.mmact_fp8_size(0, 0) == (0, 0)
    assert mmact.mmact_fp8_size(1, 1) == (16, 512)
    assert mmact.mmact_fp8_size(128, 512) == (128 * 512, 512)
    assert mmact.mmact_fp8_size(129, 513) == (129 * 528, 4 * 512)
    assert mmact.mmact_linear_fp8_workspace_bytes(3, 33) == 512 + 512
    out = ctypes.c_int64(-3)
    assert lib.mmact_fp8_size(-1, 4, ctypes.byref(out), ctypes.byref(out)) == E
    assert lib.mmact_fp8_size(4, 1 << 31, ctypes.byref(out), ctypes.byref(out)) == E
    assert lib.mmact_fp8_size(4, 4, None, ctypes.byref(out)) == E
    assert lib.mmact_linear_fp8_workspace_bytes(4, -4, ctypes.byref(out)) == E
    assert lib.mmact_linear_fp8_workspace_bytes(4, 4, None) == E
    assert lib.mmact_linear_fp8_backward_workspace_bytes(4, 4, -1, ctypes.byref(out)) == E
    assert lib.mmact_linear_fp8_backward_workspace_bytes(4, 4, 4, None) == E
    assert lib.mmact_linear_fp8_backward_workspace_bytes(BIG, BIG, 4, ctypes.byref(out)) == U
    assert out.value == -3
    assert mmact.mmact_linear_fp8_backward_workspace_bytes(333, 1000, 776) >= 333 * 1008 + 1000 * 336 + 776 * 336


def test_quantize_host_validation(lib):
    q = lambda x=P, c=P, s=P, r=4, k=64, t=1, f=5, b=1: lib.mmact_quantize_fp8(x, c, s, r, k, t, f, b, 0, None)  # noqa: E731
    d = lambda x=P, c=P, s=P, r=4, k=64, t=1, f=5: lib.mmact_dequantize_fp8(c, s, x, r, k, f, t, None)  # noqa: E731
    for f in (q, d):
        for name in ("x", "c", "s"):
            assert f(**{name: None}) == E
            assert f(**{name: MIS}) == U
            assert f(**{name: None}, r=0) == OK
            assert f(**{name: None}, k=0) == OK
        assert f(r=-1) == E and f(k=1 << 31) == E
        for bad in (3, 4, 5, 7, -1):
            assert f(t=bad) == E
        for bad in (0, 1, 2, 3, 4, 7):
            assert f(f=bad) == E
    for bad in (0, 2, 127, 129, -1):
        assert q(b=bad) == E


def gemm(lib, ac=P, as_=P, bc=P, bs=P, bias=None, C=P, M=4, N=4, K=64, ad=5, bd=6, cd=1, act=0):
    return lib.mmact_gemm_fp8(ac, as_, bc, bs, bias, C, M, N, K, ad, bd, cd, act, ctypes.c_float(0), None)


def linear(lib, x=P, wc=P, ws=P, bias=None, C=P, M=4, N=4, K=64, xd=1, wd=5, cd=1, act=0, work=P):
    return lib.mmact_linear_fp8(x, wc, ws, bias, C, M, N, K, xd, wd, cd, act, ctypes.c_float(0), work, None)


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
        assert f(lib, cd=3) == E and f(lib, cd=5) == E
        assert f(lib, act=7) == E and f(lib, act=-1) == E
        assert f(lib, bias=P + 2) == E
        assert f(lib, M=0) == OK
        assert f(lib, N=0) == OK
    for bad in (1, 2, 4, 7):
        assert gemm(lib, ad=bad) == E and gemm(lib, bd=bad) == E and linear(lib, wd=bad) == E
    assert linear(lib, xd=5) == E
    # more output tiles than are counted in 32 bits
    assert gemm(lib, M=BIG, N=BIG) == U


def backward(lib, dy=P, x=P, wc=P, ws=P, dx=P, dw=P, db=P, M=4, N=4, K=64, xd=1, wd=5, gd=6, dwd=2, work=P):
    return lib.mmact_linear_fp8_backward(dy, x, wc, ws, dx, dw, db, M, N, K, xd, wd, gd, dwd, work, None)


def test_backward_host_validation(lib):
    for name in ("dy", "x", "wc", "ws", "work"):
        assert backward(lib, **{name: None}) == E
    for name in ("dy", "x", "wc", "ws", "dx", "dw", "work"):
        assert backward(lib, **{name: MIS}) == U
    assert backward(lib, db=P + 2) == E
    for name in ("M", "N", "K"):
        assert backward(lib, **{name: -1}) == E
        assert backward(lib, **{name: 1 << 31}) == E
    assert backward(lib, xd=5) == E and backward(lib, wd=2) == E and backward(lib, gd=2) == E and backward(lib, dwd=5) == E
    assert backward(lib, M=BIG, N=BIG) == U
    assert backward(lib, dx=None, dw=None, db=None, M=0) == OK
    assert backward(lib, dx=None, dw=None, db=None) == OK     # nothing wanted
    assert backward(lib, M=0, N=0, K=0) == OK


def test_kernel_mode_validation(lib):
    for bad in (-1, 3):
        assert lib.mmact_set_gemm_fp8_kernel(bad) == E
    for good in (1, 2, 0):
        assert lib.mmact_set_gemm_fp8_kernel(good) == OK


def test_cpu_tensors_are_refused(lib):
    x = torch.zeros((4, 64))
    codes = torch.zeros((4, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    scales = torch.zeros(512, dtype=torch.uint8)
    for call in (lambda: mmact.mmact_quantize_fp8(x, codes, scales),
                 lambda: mmact.mmact_dequantize_fp8(codes, scales, x),
                 lambda: mmact.mmact_gemm_fp8(codes, scales, codes, scales, None, x, 64),
                 lambda: mmact.mmact_linear_fp8(x, codes, scales, None, x, scales),
                 lambda: mmact.mmact_linear_fp8_backward(x, x, codes, scales, x, x, None, scales)):
        with pytest.raises(TypeError):
            call()


def test_reference_rounding_pins():
    assert ref.GRID["e4m3"][-1] == 448 and ref.GRID["e5m2"][-1] == 57344
    assert ref.GRID["e4m3"][1] == 2.0 ** -9 and ref.GRID["e5m2"][1] == 2.0 ** -16
    # largest value 448: X = 1, so the grid and its ties stand as they are
    x = np.zeros((1, 128))
    x[0, :8] = [448.0, 17.0, 19.0, 18.0, 17.1, -0.0009765625, 0.0029296875, 1.0]
    c, s, v = ref.quantize(x)
    assert v[0, :8].tolist() == [448.0, 16.0, 20.0, 18.0, 18.0, 0.0, 2.0 ** -8, 1.0] and s[0] == 127
    assert c[0, 0] == 0x7e and c[0, 5] == 0x80
    # just past it: the next power of two; just below 448 / 2 and at it: the one before
    for top, b in ((448.001, 128), (224.0, 126), (224.1, 127)):
        assert ref.quantize(np.full((1, 5), top))[1][0] == b
    # torch's own 8-bit types hold the same grids
    for kind, t in (("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)):
        codes = torch.arange(len(ref.GRID[kind]), dtype=torch.uint8).view(t)
        assert np.array_equal(codes.float().numpy().astype(np.float64), ref.GRID[kind])
    c, s, v = ref.quantize(np.random.default_rng(0).normal(0, 1, (200, 700)), "e5m2", True)
    assert np.array_equal(ref.values(c, s, 700, "e5m2"), v) and not c[:, 700:].any()
    assert c.shape == (200, 704) and np.count_nonzero(s) == 200 * 6


def test_square_blocks_turned_round_have_the_same_values():
    x = np.random.default_rng(1).normal(0, 1, (256, 384))
    assert np.array_equal(ref.quantize(x, square=True)[2], ref.quantize(x.T, square=True)[2].T)
