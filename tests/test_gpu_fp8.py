"""The 8-bit block-scaled operators on the GPU against the plain 64-bit implementation:
quantisation and its inverse exactly, products within a bound derived from fp32 accumulation."""
import numpy as np
import pytest
import torch

import fp8_reference as ref
import mx_reference as mx
from conv_activation_epilogue_gb300 import build, mmact
from parity import TORCH

pytestmark = pytest.mark.gpu
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    mmact.load()


def tensor(x: np.ndarray, dtype: str) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(TORCH[dtype]).cuda()


def host64(t: torch.Tensor) -> np.ndarray:
    return t.detach().float().cpu().numpy().astype(np.float64)


def empty(rows, K, kind="e4m3"):
    nc, ns = mmact.mmact_fp8_size(rows, K)
    return (torch.full((rows, nc // max(rows, 1)), 0xAB, dtype=torch.uint8, device="cuda").view(F8[kind]),
            torch.full((ns,), 0xCD, dtype=torch.uint8, device="cuda"))


def quantized(x, kind="e4m3", square=False, transposed=False):
    codes, scales = empty(*(x.shape[::-1] if transposed else x.shape), kind)
    mmact.mmact_quantize_fp8(x, codes, scales, 128 if square else 1, transposed)
    return codes, scales


def raw(codes):
    return codes.view(torch.uint8).cpu().numpy()


def spread(rng, rows, K, dtype):
    """Rows over many binades, some zeros, ties of both grids, denormals of the type."""
    x = rng.normal(0, 1, (rows, K)) * np.exp2(rng.integers(-10, 11, (rows, 1)))
    tie = rng.random((rows, K)) < 0.2
    x = np.where(tie, rng.choice([1.0625, 1.125, 1.1875, 1.25, 1.375, 1.625, 1.75, 1.875], (rows, K))
                 * np.exp2(rng.integers(-12, 3, (rows, K))) * rng.choice([-1, 1], (rows, K)), x)
    x[rng.random((rows, K)) < 0.05] = 0.0
    if rows > 2:
        x[rows // 2] = 0.0                                  # a row of zeros
        x[rows - 1] *= 2.0 ** {"f16": -24, "bf16": -140, "f32": -150}[dtype]   # mostly denormals
    return x


SIZES = [(1, 1), (1, 128), (1, 2048), (2, 127), (3, 129), (127, 64), (128, 128), (129, 130), (5, 1000), (300, 257),
         (64, 511), (66, 512), (130, 513), (257, 640)]


@pytest.mark.parametrize("rows,K", SIZES)
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("square", [False, True])
@pytest.mark.parametrize("transposed", [False, True])
def test_quantize_is_exact(rows, K, dtype, kind, square, transposed):
    rng = np.random.default_rng(rows * 1009 + K)
    x = tensor(spread(rng, rows, K, dtype), dtype)
    codes, scales = quantized(x.t().contiguous() if transposed else x, kind, square, transposed)
    c, s, v = ref.quantize(host64(x), kind, square)
    assert np.array_equal(scales.cpu().numpy(), s)           # the bytes of rows and blocks that do not exist too
    assert np.array_equal(raw(codes), c)
    # values: exact in fp32 (a subnormal value of a subnormal scale included)
    for out in ("f32", dtype):
        y = torch.full((rows, K), 7.0, dtype=TORCH[out], device="cuda")
        mmact.mmact_dequantize_fp8(codes, scales, y)
        assert torch.equal(y.cpu(), torch.from_numpy(v.astype(np.float32)).to(TORCH[out]))
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK


@pytest.mark.parametrize("square", [False, True])
@pytest.mark.parametrize("transposed", [False, True])
def test_quantize_infinities_and_nan_mark_their_block_only(transposed, square):
    x = np.ones((200, 400))
    x[0, 5], x[1, 140], x[2, 270], x[150, 395] = np.inf, -np.inf, np.nan, np.inf
    t = tensor(x, "bf16")
    codes, scales = quantized(t.t().contiguous() if transposed else t, "e4m3", square, transposed)
    with np.errstate(invalid="ignore"):
        c, s, v = ref.quantize(x, "e4m3", square)
    assert np.array_equal(raw(codes), c) and np.array_equal(scales.cpu().numpy(), s)
    y = torch.empty((200, 400), dtype=torch.bfloat16, device="cuda")
    mmact.mmact_dequantize_fp8(codes, scales, y)
    got = host64(y)
    assert np.array_equal(np.isnan(got), np.isnan(v)) and np.all(got[~np.isnan(v)] == 1.0)
    assert np.isnan(got).sum() == (3 * 128 * 128 + 72 * 16 if square else 3 * 128 + 16)


def test_quantize_extremes_of_fp32():
    big = float(np.finfo(np.float32).max)
    x = np.zeros((3, 256))
    x[0, :3] = big, -big / 2, 1.0
    x[1, :3] = 2.0 ** -149, -2.0 ** -126, 2.0 ** -127
    x[2, :40] = 2.0 ** -126 * np.arange(40)
    t = torch.from_numpy(x.astype(np.float32)).cuda()
    for kind in F8:
        codes, scales = quantized(t, kind)
        c, s, v = ref.quantize(x.astype(np.float32).astype(np.float64), kind)
        assert np.array_equal(raw(codes), c) and np.array_equal(scales.cpu().numpy(), s)
        y = torch.empty((3, 256), dtype=torch.float32, device="cuda")
        mmact.mmact_dequantize_fp8(codes, scales, y)
        # fp32's largest value, 2^128 (1 - 2^-24), lies next to 2^128 on either 8-bit grid, and fp32 has no 2^128
        assert v[0, 0] == 2.0 ** 128
        with np.errstate(over="ignore"):
            assert np.array_equal(host64(y), v.astype(np.float32).astype(np.float64))


def random_f8(rng, rows, K, std=1.0, kind="e4m3", square=False):
    """An 8-bit matrix with its 64-bit values; scales differ from block to block."""
    x = rng.normal(0, std, (rows, K)) * np.exp2(rng.integers(-3, 4, (rows, -(-K // 128)))).repeat(128, axis=1)[:, :K]
    c, s, v = ref.quantize(x.astype(np.float32).astype(np.float64), kind, square)
    return torch.from_numpy(c).cuda().view(F8[kind]), torch.from_numpy(s).cuda(), v


def check(got: torch.Tensor, want: np.ndarray, bound: np.ndarray, dtype: str):
    g = host64(got)
    err = np.abs(g - want)
    lim = bound + ref_half_step(np.abs(want) + bound, dtype)
    assert np.all(np.isfinite(g))
    worst = np.unravel_index(np.argmax(err / lim), err.shape)
    assert np.all(err <= lim), (worst, g[worst], want[worst], err[worst], lim[worst])


def ref_half_step(v, dtype):
    return mx.ulp(v, dtype) / 2


@pytest.fixture(params=[0, 1, 2], ids=["chosen", "rows", "pair"])
def kernel(request):
    """Each kernel for every shape: the shape's own choice is only about speed."""
    mmact.mmact_set_gemm_fp8_kernel(request.param)
    yield request.param
    mmact.mmact_set_gemm_fp8_kernel(0)


GEMMS = [(1, 1, 1), (1, 128, 32), (1, 136, 64), (2, 8, 96), (7, 129, 100), (16, 256, 256), (17, 100, 288), (33, 260, 511),
         (64, 640, 512), (65, 72, 1000), (128, 128, 128), (129, 127, 130), (200, 512, 2048), (256, 264, 768), (300, 1000, 320),
         (513, 520, 544), (640, 384, 4096)]


@pytest.mark.parametrize("M,N,K", GEMMS)
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
def test_gemm(M, N, K, out, kernel):
    rng = np.random.default_rng(M * 7919 + N * 31 + K)
    (ac, as_, av), (bc, bs, bv) = random_f8(rng, M, K), random_f8(rng, N, K, K ** -0.5, "e4m3", True)
    bias = rng.normal(0, 1, N).astype(np.float32)
    C = torch.full((M, N), float("nan"), dtype=TORCH[out], device="cuda")
    mmact.mmact_gemm_fp8(ac, as_, bc, bs, torch.from_numpy(bias).cuda(), C, K)
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
    want, bound = mx.gemm(av, bv, bias.astype(np.float64), "none", 0.0)
    check(C, want, bound, out)


@pytest.mark.parametrize("a", ["e4m3", "e5m2"])
@pytest.mark.parametrize("b", ["e4m3", "e5m2"])
@pytest.mark.parametrize("M,N,K", [(3, 200, 160), (130, 192, 300), (400, 300, 1100)])
def test_gemm_formats(a, b, M, N, K, kernel):
    rng = np.random.default_rng(M + N + K)
    (ac, as_, av), (bc, bs, bv) = random_f8(rng, M, K, kind=a), random_f8(rng, N, K, K ** -0.5, b)
    C = torch.full((M, N), float("nan"), dtype=torch.float32, device="cuda")
    mmact.mmact_gemm_fp8(ac, as_, bc, bs, None, C, K)
    want, bound = mx.gemm(av, bv, None, "none", 0.0)
    check(C, want, bound, "f32")


@pytest.mark.parametrize("name", ["none", "relu", "leaky_relu", "tanh", "sigmoid", "gelu", "silu"])
@pytest.mark.parametrize("M,N,K", [(3, 200, 160), (130, 192, 300), (260, 300, 256)])
def test_gemm_activations(name, M, N, K, kernel):
    rng = np.random.default_rng(M + N + K)
    (ac, as_, av), (bc, bs, bv) = random_f8(rng, M, K), random_f8(rng, N, K, K ** -0.5)
    for out, bias in (("f32", None), ("bf16", rng.normal(0, 1, N).astype(np.float32))):
        C = torch.full((M, N), float("nan"), dtype=TORCH[out], device="cuda")
        mmact.mmact_gemm_fp8(ac, as_, bc, bs, None if bias is None else torch.from_numpy(bias).cuda(), C, K, name, 0.3)
        want, bound = mx.gemm(av, bv, None if bias is None else bias.astype(np.float64), name, 0.3)
        check(C, want, bound, out)


@pytest.mark.parametrize("M", [700, 40])
def test_gemm_against_its_own_scales(M, kernel):
    """A one-hot A picks single values of B through every block and row: each scale byte and code
    has to be the one of its own row, block and place (exact)."""
    rng = np.random.default_rng(5)
    N, K = 384, 700
    bc, bs, bv = random_f8(rng, N, K)
    a = np.zeros((M, K))
    a[np.arange(M), np.arange(M) * (K // M)] = np.exp2(np.arange(M) % 5)
    c, s, av = ref.quantize(a)
    C = torch.empty((M, N), dtype=torch.float32, device="cuda")
    mmact.mmact_gemm_fp8(torch.from_numpy(c).cuda().view(F8["e4m3"]), torch.from_numpy(s).cuda(), bc, bs, None, C, K)
    assert np.array_equal(host64(C), av @ bv.T)


@pytest.mark.parametrize("M", [2, 140, 300])
def test_gemm_nan_scales_reach_their_row_or_column_only(M, kernel):
    rng = np.random.default_rng(6)
    N, K = 200, 640
    (ac, as_, av), (bc, bs, bv) = random_f8(rng, M, K), random_f8(rng, N, K)
    bs[mx.scale_place(150, 3, ref.tiles_of(N, K)[1])] = 255
    as_[mx.scale_place(1, 4, ref.tiles_of(M, K)[1])] = 255
    C = torch.empty((M, N), dtype=torch.float32, device="cuda")
    mmact.mmact_gemm_fp8(ac, as_, bc, bs, None, C, K, "relu")
    want = np.zeros((M, N), dtype=bool)
    want[1, :] = want[:, 150] = True
    assert np.array_equal(np.isnan(host64(C)), want)


@pytest.mark.parametrize("M,N", [(1, 8), (5, 129), (128, 256)])
def test_empty_k_is_the_activation_of_the_bias(M, N):
    bias = torch.linspace(-3, 3, N, device="cuda")
    b = bias.double().cpu().numpy()
    e = torch.empty(0, dtype=torch.uint8, device="cuda")
    for which in ("gemm", "linear"):
        C = torch.empty((M, N), dtype=torch.float32, device="cuda")
        w = e.view(F8["e4m3"])
        if which == "gemm":
            mmact.mmact_gemm_fp8(w.view(M, 0), e, w.view(N, 0), e, bias, C, 0, "silu")
        else:
            mmact.mmact_linear_fp8(torch.empty((M, 0), device="cuda"), w.view(N, 0), e, bias, C, e, "silu")
        check(C, np.broadcast_to(mx.act(b, "silu", 0), (M, N)), np.broadcast_to(mx.act_error(b, "silu"), (M, N)), "f32")


LINEARS = [(1, 512, 1024), (1, 333, 100), (5, 72, 640), (8, 1000, 4096), (9, 264, 520), (16, 130, 33), (17, 260, 4100),
           (32, 128, 777), (33, 640, 512), (80, 1001, 2056), (150, 128, 64), (260, 640, 256)]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,N,K", LINEARS)
def test_linear_is_quantise_and_gemm(dtype, M, N, K, kernel):
    rng = np.random.default_rng(M + K)
    x = tensor(rng.normal(0, 1, (M, K)) * np.exp2(rng.integers(-4, 5, (M, 1))), dtype)
    wc, ws, wv = random_f8(rng, N, K, K ** -0.5, "e5m2" if N % 2 else "e4m3", True)
    bias = rng.normal(0, 1, N).astype(np.float32)
    work = torch.full((mmact.mmact_linear_fp8_workspace_bytes(M, K),), 0xFF, dtype=torch.uint8, device="cuda")
    outs = []
    for _ in range(2):                                        # a used workspace makes no difference
        C = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        mmact.mmact_linear_fp8(x, wc, ws, torch.from_numpy(bias).cuda(), C, work, "gelu")
        outs.append(C)
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
    assert torch.equal(outs[0], outs[1])
    want, bound = mx.gemm(ref.quantize(host64(x))[2], wv, bias.astype(np.float64), "gelu", 0.0)
    check(outs[0], want, bound, "bf16")


def test_linear_marks_infinities_and_nan_like_the_quantiser():
    rng = np.random.default_rng(9)
    M, N, K = 5, 130, 320
    x = rng.normal(0, 1, (M, K))
    clean = x.copy()
    x[1, 7], x[3, 300] = np.inf, np.nan
    wc, ws, wv = random_f8(rng, N, K, K ** -0.5)
    work = torch.empty(mmact.mmact_linear_fp8_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    out = [torch.empty((M, N), dtype=torch.float32, device="cuda") for _ in range(2)]
    mmact.mmact_linear_fp8(tensor(x, "bf16"), wc, ws, None, out[0], work)
    mmact.mmact_linear_fp8(tensor(clean, "bf16"), wc, ws, None, out[1], work)
    assert torch.isnan(out[0][[1, 3]]).all() and torch.equal(out[0][[0, 2, 4]], out[1][[0, 2, 4]])


def test_linear_on_a_side_stream_and_in_a_graph():
    rng = np.random.default_rng(8)
    M, N, K = 40, 512, 1024
    x = tensor(rng.normal(0, 1, (M, K)), "bf16")
    wc, ws, wv = random_f8(rng, N, K, K ** -0.5)
    work = torch.empty(mmact.mmact_linear_fp8_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    C = torch.empty((M, N), dtype=torch.float32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mmact.mmact_linear_fp8(x, wc, ws, None, C, work, stream=s)
    s.synchronize()
    want, bound = mx.gemm(ref.quantize(host64(x))[2], wv, None, "none", 0.0)
    check(C, want, bound, "f32")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mmact.mmact_linear_fp8(x, wc, ws, None, C, work)
    x.copy_(tensor(rng.normal(0, 1, (M, K)), "bf16"))
    C.zero_()
    g.replay()
    torch.cuda.synchronize()
    want, bound = mx.gemm(ref.quantize(host64(x))[2], wv, None, "none", 0.0)
    check(C, want, bound, "f32")
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK


def values64(codes, scales, rows, K):
    v = torch.empty((rows, K), dtype=torch.float32, device="cuda")      # exact (tested above)
    mmact.mmact_dequantize_fp8(codes, scales, v)
    return v.double()


@pytest.mark.parametrize("M,N,K", [(1, 520, 8192), (16, 136, 4100), (100, 400, 2500), (1536, 1280, 640), (2816, 2560, 96),
                                   (130, 8200, 1030), (5000, 40, 2048), (9, 8192, 8192), (3, 8192, 8192), (16, 2048, 8192)])
def test_gemm_many_k_blocks_and_many_tiles(M, N, K, kernel):
    """Rings that go round, deep ones, two CTAs to an SM, several tiles for each CTA pair."""
    g = torch.Generator(device="cuda").manual_seed(M + K)
    a, b = (torch.empty((r, K), device="cuda").normal_(0, 1, generator=g) for r in (M, N))
    (ac, as_), (bc, bs) = quantized(a), quantized(b, "e4m3", True)
    for out in (torch.float32, torch.bfloat16):
        C = torch.full((M, N), float("nan"), dtype=out, device="cuda")
        mmact.mmact_gemm_fp8(ac, as_, bc, bs, None, C, K)
        assert mmact.mmact_get_last_error() == mmact.MMACT_OK
        va, vb = values64(ac, as_, M, K), values64(bc, bs, N, K)
        want = va @ vb.t()
        err, bound = (C.double() - want).abs(), mx.sum_error(K) * (va.abs() @ vb.abs().t())
        if out is torch.bfloat16:
            bound = bound + (want.abs() + bound) * 2.0 ** -8 + 2.0 ** -134
        assert bool((err <= bound).all())


BACKWARDS = [(1, 1, 1), (1, 200, 130), (5, 64, 300), (130, 129, 127), (333, 1000, 776), (256, 384, 512), (1200, 260, 640)]


def backward(dy, x, wt, grad_type, dw_dtype=torch.float32, want=("dx", "dw", "db")):
    (M, N), K = dy.shape, x.shape[1]
    nan = float("nan")
    dx = torch.full((M, K), nan, dtype=x.dtype, device="cuda") if "dx" in want else None
    dw = torch.full((N, K), nan, dtype=dw_dtype, device="cuda") if "dw" in want else None
    db = torch.full((N,), nan, device="cuda") if "db" in want else None
    work = torch.full((mmact.mmact_linear_fp8_backward_workspace_bytes(M, N, K),), 0xFF, dtype=torch.uint8, device="cuda")
    mmact.mmact_linear_fp8_backward(dy, x, wt[0], wt[1], dx, dw, db, work, grad_type=grad_type)
    return dx, dw, db


@pytest.mark.parametrize("M,N,K", BACKWARDS)
@pytest.mark.parametrize("dtype,kind,dwt", [("bf16", "e5m2", "f32"), ("f16", "e4m3", "bf16"), ("f32", "e5m2", "f32")])
def test_backward(M, N, K, dtype, kind, dwt, kernel):
    rng = np.random.default_rng(M + 3 * N + K)
    dy = tensor(rng.normal(0, 1, (M, N)) * np.exp2(rng.integers(-4, 5, (M, 1))), dtype)
    x = tensor(rng.normal(0, 1, (M, K)), dtype)
    w = tensor(rng.normal(0, K ** -0.5, (N, K)), "bf16")
    wt = quantized(w, "e4m3", True, transposed=True)
    dx, dw, db = backward(dy, x, wt, F8[kind], TORCH[dwt])
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
    gy, gx, gw = host64(dy), host64(x), host64(w)
    want, bound = mx.gemm(ref.quantize(gy, kind)[2], ref.quantize(gw, "e4m3", True)[2].T, None, "none", 0.0)
    check(dx, want, bound, dtype)
    want, bound = mx.gemm(ref.quantize(gy.T, kind)[2], ref.quantize(gx.T, "e4m3")[2], None, "none", 0.0)
    check(dw, want, bound, dwt)
    check(db[None], gy.sum(axis=0)[None], mx.sum_error(M) * np.abs(gy).sum(axis=0)[None], "f32")


@pytest.mark.parametrize("M,N,K", [(2900, 1500, 2600), (700, 5000, 2300), (6000, 2400, 1030), (20000, 600, 300)])
@pytest.mark.parametrize("dwt", [torch.float32, torch.float16])
def test_backward_large(M, N, K, dwt):
    """Both products in one launch, several tiles for each CTA pair, either one the longer."""
    g = torch.Generator(device="cuda").manual_seed(M)
    dy, x, w = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((M, N), (M, K), (N, K)))
    wt = quantized(w, "e4m3", True, transposed=True)
    dx, dw, db = backward(dy, x, wt, F8["e4m3"], dwt)
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
    a, b = values64(*quantized(dy), M, N), values64(*wt, K, N)
    at, xt = values64(*quantized(dy, transposed=True), N, M), values64(*quantized(x, transposed=True), K, M)
    for got, l, r, half in ((dx, a, b, 2.0 ** -8), (dw, at, xt, 0.0 if dwt is torch.float32 else 2.0 ** -11)):
        want = l @ r.t()
        bound = mx.sum_error(l.shape[1]) * (l.abs() @ r.abs().t())
        assert bool(((got.double() - want).abs() <= bound + half * (want.abs() + bound)).all())
    want = dy.double().sum(dim=0)
    assert bool(((db - want).abs() <= mx.sum_error(M) * dy.double().abs().sum(dim=0)).all())


def test_backward_of_the_wanted_gradients_only():
    rng = np.random.default_rng(2)
    M, N, K = 140, 260, 300
    dy, x = tensor(rng.normal(0, 1, (M, N)), "bf16"), tensor(rng.normal(0, 1, (M, K)), "bf16")
    wt = quantized(tensor(rng.normal(0, 1, (N, K)), "bf16"), "e4m3", True, transposed=True)
    every = backward(dy, x, wt, F8["e5m2"])
    for i, name in enumerate(("dx", "dw", "db")):
        got = backward(dy, x, wt, F8["e5m2"], want=(name,))
        assert [g is None for g in got] == [j != i for j in range(3)]
        assert torch.equal(got[i], every[i])
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK


@pytest.mark.parametrize("M,N,K", [(0, 40, 24), (6, 0, 24), (6, 40, 0), (0, 0, 24)])
def test_backward_of_empty_dimensions_is_zero(M, N, K):
    dy, x = torch.ones((M, N), device="cuda"), torch.ones((M, K), device="cuda")
    c, s = mmact.mmact_fp8_size(K, N)
    wt = torch.zeros(c, dtype=torch.uint8, device="cuda").view(F8["e4m3"]), torch.zeros(s, dtype=torch.uint8, device="cuda")
    dx, dw, db = backward(dy, x, wt, F8["e5m2"])
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
    assert not dx.any() and not dw.any()
    assert torch.equal(db, dy.sum(dim=0))


def test_backward_against_differences():
    """The gradient of sum(dy * (x W^T)) along single entries, from values that 8 bits hold exactly (powers of
    two within a block's range), so that the products' own rounding is all that is left."""
    rng = np.random.default_rng(3)
    M, N, K = 40, 72, 56
    x, w, dy = (rng.choice([-2.0, -1.0, -0.5, 0.5, 1.0, 2.0], s) for s in ((M, K), (N, K), (M, N)))
    wt = quantized(tensor(w, "bf16"), "e4m3", True, transposed=True)
    dx, dw, db = backward(tensor(dy, "f32"), tensor(x, "f32"), wt, F8["e5m2"])

    def loss(x, w):
        return float((dy * (x @ w.T)).sum())

    for _ in range(20):
        i, j, n = rng.integers(M), rng.integers(K), rng.integers(N)
        step = np.zeros((M, K))
        step[i, j] = 0.25
        assert abs((loss(x + step, w) - loss(x - step, w)) / 0.5 - float(dx[i, j])) < 1e-9
        step = np.zeros((N, K))
        step[n, j] = 0.25
        assert abs((loss(x, w + step) - loss(x, w - step)) / 0.5 - float(dw[n, j])) < 1e-9
    assert np.array_equal(host64(db), dy.sum(axis=0))


def test_backward_in_a_graph_on_its_own_workspace():
    rng = np.random.default_rng(4)
    M, N, K = 300, 264, 520
    dy, x = tensor(rng.normal(0, 1, (M, N)), "bf16"), tensor(rng.normal(0, 1, (M, K)), "bf16")
    wt = quantized(tensor(rng.normal(0, 1, (N, K)), "bf16"), "e4m3", True, transposed=True)
    dx, dw, db = torch.empty_like(x), torch.empty((N, K), device="cuda"), torch.empty(N, device="cuda")
    work = torch.empty(mmact.mmact_linear_fp8_backward_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
    mmact.mmact_linear_fp8_backward(dy, x, *wt, dx, dw, db, work)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mmact.mmact_linear_fp8_backward(dy, x, *wt, dx, dw, db, work)
    dy.copy_(tensor(rng.normal(0, 1, (M, N)), "bf16"))
    work.fill_(0xFF)
    g.replay()
    torch.cuda.synchronize()
    for got, want in zip((dx, dw, db), backward(dy, x, wt, F8["e5m2"])):
        assert torch.equal(got, want)


@pytest.mark.parametrize("M,N,K", [(300, 520, 8192), (300, 520, 12345), (2000, 2600, 8192), (200, 8000, 20000)])
def test_fp32_sums_over_long_k(M, N, K, kernel):
    """Positive products, so that errors of one sign add up.  An accumulator takes at most 32 K blocks: 128 additions of
    32 products, each of which may cut off up to 2^-23 of the sum so far, which grows evenly: half of that on average,
    64 * 2^-23; then the partial sums' additions and the bias, rounded."""
    g = torch.Generator(device="cuda").manual_seed(M + K)
    a, b = (torch.rand((r, K), device="cuda", generator=g) for r in (M, N))
    (ac, as_), (bc, bs) = quantized(a), quantized(b)
    C = torch.full((M, N), float("nan"), device="cuda")
    bias = torch.rand(N, device="cuda", generator=g)
    mmact.mmact_gemm_fp8(ac, as_, bc, bs, bias, C, K, "leaky_relu", 0.5)
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
    want = values64(ac, as_, M, K) @ values64(bc, bs, N, K).t() + bias.double()
    chunks = -(-K // 2048)
    assert float(((C.double() - want).abs() / want).max()) <= (64 + chunks + 2) * 2.0 ** -23


def test_long_rows_pass_32_bit_offsets():
    """More than 2^31 values: a matrix whose last rows lie past 32-bit byte and element offsets."""
    rows, K = 70000, 32768
    x = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
    for r in (0, 65536, rows - 1):
        x[r] = torch.arange(K, device="cuda").remainder(13).to(torch.bfloat16) - 6
    for square in (False, True):
        codes, scales = quantized(x, "e4m3", square)
        y = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda")
        mmact.mmact_dequantize_fp8(codes, scales, y)
        for r in (0, 65536, rows - 1):
            assert torch.equal(y[r], x[r])
        assert int(torch.count_nonzero(y)) == sum(int(torch.count_nonzero(y[r])) for r in (0, 65536, rows - 1))
    # a product over such a matrix: its last rows
    a = torch.zeros((3, K), dtype=torch.bfloat16, device="cuda")
    a[0, 5], a[1, K - 1], a[2, 70] = 1.0, 2.0, 3.0
    ac, as_ = quantized(a)
    C = torch.full((3, rows), float("nan"), device="cuda")
    mmact.mmact_gemm_fp8(ac, as_, codes, scales, None, C, K)
    for i, (k, f) in enumerate(((5, 1.0), (K - 1, 2.0), (70, 3.0))):
        assert torch.equal(C[i], x[:, k].float() * f)


@pytest.mark.parametrize("M,N,K", [(1, 8192, 8192), (8, 8192, 8192), (5, 4100, 8195), (3, 520, 16000)])
@pytest.mark.parametrize("out", [torch.float32, torch.float16])
def test_linear_of_few_rows_over_long_k(M, N, K, out):
    """Rows quantised inside the product: deep rings that go round, rows that begin anywhere."""
    g = torch.Generator(device="cuda").manual_seed(N + K)
    x, w = torch.randn((M, K), generator=g, device="cuda").bfloat16(), torch.randn((N, K), generator=g, device="cuda").bfloat16()
    q = quantized(w, "e4m3", True)
    C = torch.full((M, N), float("nan"), dtype=out, device="cuda")
    work = torch.full((mmact.mmact_linear_fp8_workspace_bytes(M, K),), 0xFF, dtype=torch.uint8, device="cuda")
    mmact.mmact_linear_fp8(x, *q, None, C, work)
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
    a, b = values64(*quantized(x), M, K), values64(*q, N, K)
    want, bound = a @ b.t(), mx.sum_error(K) * (a.abs() @ b.abs().t())
    assert bool(((C.double() - want).abs() <= bound + (2.0 ** -24 if out is torch.float32 else 2.0 ** -11) * (want.abs() + bound)
                 + 2.0 ** -25).all())


def test_backward_passes_32_bit_offsets():
    """More than 2^31 values of dy: the last tokens' gradients and what they add to the weights' and the bias's."""
    M, N, K = 70000, 32768, 40
    g = torch.Generator(device="cuda").manual_seed(1)
    dy = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    dy[-200:] = torch.randn((200, N), generator=g, device="cuda").bfloat16()
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    wt = quantized(torch.randn((N, K), generator=g, device="cuda").bfloat16(), "e4m3", True, transposed=True)
    dx, dw, db = backward(dy, x, wt, F8["e4m3"])
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
    assert not dx[:-200].any()
    tail, a = dy[-200:], values64(*quantized(dy[-200:].contiguous()), 200, N)
    b = values64(*wt, K, N)
    want, bound = a @ b.t(), mx.sum_error(N) * (a.abs() @ b.abs().t())
    assert bool(((dx[-200:].double() - want).abs() <= bound + 2.0 ** -8 * (want.abs() + bound)).all())
    # the last 112 rows are a block of their own, the 88 before them lie in the block that ends at 69888
    first = M - 112 - 128
    a = values64(*quantized(dy[first:].t().contiguous()), N, 240)
    b = values64(*quantized(x[first:].t().contiguous()), K, 240)
    want, bound = a @ b.t(), mx.sum_error(M) * (a.abs() @ b.abs().t())
    assert bool(((dw.double() - want).abs() <= bound + 2.0 ** -24 * (want.abs() + bound)).all())
    want = tail.double().sum(dim=0)
    assert bool(((db - want).abs() <= mx.sum_error(M) * tail.double().abs().sum(dim=0)).all())


def test_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    codes = torch.zeros((4, 64), dtype=torch.uint8, device="cuda").view(F8["e4m3"])
    scales = torch.zeros(512, dtype=torch.uint8, device="cuda")
    C = torch.zeros((4, 4), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        mmact.mmact_quantize_fp8(x.int(), codes, scales)
    with pytest.raises(TypeError):
        mmact.mmact_quantize_fp8(x, codes.view(torch.uint8), scales)     # the codes' dtype is the format
    with pytest.raises(ValueError):
        mmact.mmact_quantize_fp8(x.t(), codes, scales)                   # not contiguous
    with pytest.raises(ValueError):
        mmact.mmact_quantize_fp8(x, codes[:3], scales)                   # too few codes
    with pytest.raises(ValueError):
        mmact.mmact_quantize_fp8(x, codes, scales[:256])
    with pytest.raises(ValueError):
        mmact.mmact_quantize_fp8(x, codes, scales, block_rows=64)
    with pytest.raises(ValueError):
        mmact.mmact_gemm_fp8(codes, scales, codes, scales, None, C, 128)  # codes are for K = 64
    with pytest.raises(ValueError):
        mmact.mmact_linear_fp8(x, codes, scales, None, C, torch.zeros(512, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        mmact.mmact_linear_fp8_backward(C, x, codes, scales, x[:3], None, None, scales)
    with pytest.raises(TypeError):
        mmact.mmact_linear_fp8_backward(C, x, codes, scales, None, None, None, scales, grad_type=torch.float16)
    off = torch.zeros(4 * 64 + 8, dtype=torch.uint8, device="cuda")[8:].view(4, 64).view(F8["e4m3"])
    with pytest.raises(mmact.MmactError) as ei:                          # codes not 16-byte aligned
        mmact.mmact_quantize_fp8(x, off, scales)
    assert ei.value.status == mmact.MMACT_ERR_UNSUPPORTED
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
