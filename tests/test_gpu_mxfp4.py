"""MXFP4 on the GPU against the plain 64-bit implementation: quantisation and its
inverse exactly, the product within a bound derived from fp32 accumulation."""
import numpy as np
import pytest
import torch

import mx_reference as ref
from conv_activation_epilogue_gb300 import build, mmact
from parity import TORCH

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    mmact.load()


def tensor(x: np.ndarray, dtype: str) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(TORCH[dtype]).cuda()


def host64(t: torch.Tensor) -> np.ndarray:
    return t.detach().float().cpu().numpy().astype(np.float64)


def quantized(x: torch.Tensor, transposed=False):
    rows, K = (x.shape[1], x.shape[0]) if transposed else x.shape
    nc, ns = mmact.mmact_mxfp4_size(rows, K)
    codes = torch.full((rows, nc // max(rows, 1)), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((ns,), 0xCD, dtype=torch.uint8, device="cuda")
    mmact.mmact_quantize_mxfp4(x, codes, scales, transposed=transposed)
    return codes, scales


def spread(rng, rows, K, dtype):
    """Rows over many binades, some zeros, ties of the 4-bit grid, denormals of the type."""
    x = rng.normal(0, 1, (rows, K)) * np.exp2(rng.integers(-10, 11, (rows, 1)))
    tie = rng.random((rows, K)) < 0.2
    x = np.where(tie, rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0], (rows, K)) * rng.choice([-1, 1], (rows, K)), x)
    x[rng.random((rows, K)) < 0.05] = 0.0
    if rows > 2:
        x[rows // 2] = 0.0                                  # a row of zeros
        x[rows - 1] *= 2.0 ** {"f16": -24, "bf16": -140, "f32": -150}[dtype]   # mostly denormals
    return x


SIZES = [(1, 1), (1, 32), (1, 2048), (2, 31), (3, 33), (127, 64), (128, 128), (129, 130), (5, 1000), (300, 257),
         (64, 255), (66, 512)]


@pytest.mark.parametrize("rows,K", SIZES)
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("transposed", [False, True])
def test_quantize_is_exact(rows, K, dtype, transposed):
    rng = np.random.default_rng(rows * 1009 + K)
    x = tensor(spread(rng, rows, K, dtype), dtype)
    codes, scales = quantized(x.t().contiguous() if transposed else x, transposed)
    c, s, v = ref.quantize(host64(x))
    assert np.array_equal(codes.cpu().numpy(), c)
    assert np.array_equal(scales.cpu().numpy(), s)           # the bytes of rows and blocks that do not exist too
    # values: exact in fp32 (a subnormal value of a subnormal scale included)
    y = torch.full((rows, K), 7.0, dtype=torch.float32, device="cuda")
    mmact.mmact_dequantize_mxfp4(codes, scales, y)
    assert np.array_equal(host64(y), v)
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK


@pytest.mark.parametrize("transposed", [False, True])
def test_quantize_infinities_and_nan_mark_their_block_only(transposed):
    x = np.ones((4, 96))
    x[0, 5], x[1, 40], x[2, 70], x[3, 95] = np.inf, -np.inf, np.nan, np.inf
    t = tensor(x, "bf16")
    codes, scales = quantized(t.t().contiguous() if transposed else t, transposed)
    with np.errstate(invalid="ignore"):
        c, s, v = ref.quantize(x)
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s)
    y = torch.empty((4, 96), dtype=torch.bfloat16, device="cuda")
    mmact.mmact_dequantize_mxfp4(codes, scales, y)
    got = host64(y)
    assert np.array_equal(np.isnan(got), np.isnan(v)) and np.isnan(got).sum() == 4 * 32
    assert np.all(got[~np.isnan(v)] == 1.0)


def test_quantize_extremes_of_fp32():
    big = float(np.finfo(np.float32).max)
    x = np.zeros((3, 64))
    x[0, :3] = big, -big / 2, 1.0
    x[1, :3] = 2.0 ** -149, -2.0 ** -126, 2.0 ** -127
    x[2, :40] = 2.0 ** -126 * np.arange(40)
    t = torch.from_numpy(x.astype(np.float32)).cuda()
    codes, scales = quantized(t)
    c, s, v = ref.quantize(x.astype(np.float32).astype(np.float64))
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s)
    y = torch.empty((3, 64), dtype=torch.float32, device="cuda")
    mmact.mmact_dequantize_mxfp4(codes, scales, y)
    assert np.array_equal(host64(y), v)


def random_mx(rng, rows, K, std=1.0):
    """A matrix in MXFP4 with its 64-bit values; scales differ from block to block."""
    x = rng.normal(0, std, (rows, K)) * np.exp2(rng.integers(-3, 4, (rows, -(-K // 32)))).repeat(32, axis=1)[:, :K]
    c, s, v = ref.quantize(x.astype(np.float32).astype(np.float64))
    return torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), v


def check(got: torch.Tensor, want: np.ndarray, bound: np.ndarray, dtype: str):
    g = host64(got)
    err = np.abs(g - want)
    lim = bound + ref.ulp(np.abs(want) + bound, dtype)
    assert np.all(np.isfinite(g))
    worst = np.unravel_index(np.argmax(err / lim), err.shape)
    assert np.all(err <= lim), (worst, g[worst], want[worst], err[worst], lim[worst])


GEMMS = [(1, 1, 1), (1, 128, 32), (1, 136, 64), (2, 8, 96), (7, 129, 100), (16, 256, 256), (17, 100, 288), (33, 260, 511),
         (64, 640, 512), (65, 72, 1000), (128, 128, 128), (129, 127, 130), (200, 512, 2048), (256, 264, 768), (300, 1000, 320),
         (513, 520, 544), (640, 384, 4096)]


@pytest.fixture(params=[0, 1, 2], ids=["chosen", "rows", "pair"])
def kernel(request):
    """Each kernel for every shape: the shape's own choice is only about speed."""
    mmact.mmact_set_gemm_mxfp4_kernel(request.param)
    yield request.param
    mmact.mmact_set_gemm_mxfp4_kernel(0)


@pytest.mark.parametrize("M,N,K", GEMMS)
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
def test_gemm(M, N, K, out, kernel):
    rng = np.random.default_rng(M * 7919 + N * 31 + K)
    (ac, as_, av), (bc, bs, bv) = random_mx(rng, M, K), random_mx(rng, N, K, K ** -0.5)
    bias = rng.normal(0, 1, N).astype(np.float32)
    C = torch.full((M, N), float("nan"), dtype=TORCH[out], device="cuda")
    mmact.mmact_gemm_mxfp4(ac, as_, bc, bs, torch.from_numpy(bias).cuda(), C, K)
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
    want, bound = ref.gemm(av, bv, bias.astype(np.float64), "none", 0.0)
    check(C, want, bound, out)


@pytest.mark.parametrize("name", ["none", "relu", "leaky_relu", "tanh", "sigmoid", "gelu", "silu"])
@pytest.mark.parametrize("M,N,K", [(3, 200, 160), (130, 192, 300), (260, 300, 256)])
def test_gemm_activations(name, M, N, K, kernel):
    rng = np.random.default_rng(M + N + K)
    (ac, as_, av), (bc, bs, bv) = random_mx(rng, M, K), random_mx(rng, N, K, K ** -0.5)
    for out, bias in (("f32", None), ("bf16", rng.normal(0, 1, N).astype(np.float32))):
        C = torch.full((M, N), float("nan"), dtype=TORCH[out], device="cuda")
        mmact.mmact_gemm_mxfp4(ac, as_, bc, bs, None if bias is None else torch.from_numpy(bias).cuda(), C, K, name, 0.3)
        want, bound = ref.gemm(av, bv, None if bias is None else bias.astype(np.float64), name, 0.3)
        check(C, want, bound, out)


def test_gemm_against_its_own_scales(kernel):
    """A one-hot A picks single values of B through every block and row: each scale byte and code
    has to be the one of its own row, block and place (exact)."""
    rng = np.random.default_rng(5)
    N, K = 384, 320
    bc, bs, bv = random_mx(rng, N, K)
    a = np.zeros((K, K))
    a[np.arange(K), np.arange(K)] = np.exp2(np.arange(K) % 5)
    c, s, av = ref.quantize(a)
    C = torch.empty((K, N), dtype=torch.float32, device="cuda")
    mmact.mmact_gemm_mxfp4(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), bc, bs, None, C, K)
    assert np.array_equal(host64(C), av @ bv.T)


@pytest.mark.parametrize("M", [2, 140, 300])
def test_gemm_nan_scales_reach_their_row_or_column_only(M, kernel):
    rng = np.random.default_rng(6)
    N, K = 200, 192
    (ac, as_, av), (bc, bs, bv) = random_mx(rng, M, K), random_mx(rng, N, K)
    kt = ref.tiles_of(N, K)[1]
    bs[ref.scale_place(150, 3, kt)] = 255
    as_[ref.scale_place(1, 5, ref.tiles_of(M, K)[1])] = 255
    C = torch.empty((M, N), dtype=torch.float32, device="cuda")
    mmact.mmact_gemm_mxfp4(ac, as_, bc, bs, None, C, K)
    bad = np.isnan(host64(C))
    want = np.zeros((M, N), dtype=bool)
    want[1, :] = want[:, 150] = True
    assert np.array_equal(bad, want)


@pytest.mark.parametrize("M,N", [(1, 8), (5, 129), (128, 256)])
def test_gemm_empty_k_is_the_activation_of_the_bias(M, N):
    bias = torch.linspace(-3, 3, N, device="cuda")
    C = torch.empty((M, N), dtype=torch.float32, device="cuda")
    e = torch.empty(0, dtype=torch.uint8, device="cuda")
    mmact.mmact_gemm_mxfp4(e.view(M, 0), e, e.view(N, 0), e, bias, C, 0, "silu")
    b = bias.double().cpu().numpy()
    check(C, np.broadcast_to(ref.act(b, "silu", 0), (M, N)), np.broadcast_to(ref.act_error(b, "silu"), (M, N)), "f32")


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 512, 1024), (1, 333, 100), (9, 264, 520), (16, 130, 33), (17, 260, 4100), (32, 128, 777),
                                   (33, 640, 512), (80, 1001, 2056), (150, 128, 64), (260, 640, 256)])
def test_linear_is_quantise_and_gemm(dtype, M, N, K, kernel):
    rng = np.random.default_rng(M + K)
    x = tensor(rng.normal(0, 1, (M, K)), dtype)
    wc, ws, wv = random_mx(rng, N, K, K ** -0.5)
    bias = rng.normal(0, 1, N).astype(np.float32)
    work = torch.full((mmact.mmact_linear_mxfp4_workspace_bytes(M, K),), 0xFF, dtype=torch.uint8, device="cuda")
    outs = []
    for _ in range(2):                                        # a used workspace makes no difference
        C = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        mmact.mmact_linear_mxfp4(x, wc, ws, torch.from_numpy(bias).cuda(), C, work, "gelu")
        outs.append(C)
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
    assert torch.equal(outs[0], outs[1])
    want, bound = ref.gemm(ref.quantize(host64(x))[2], wv, bias.astype(np.float64), "gelu", 0.0)
    check(outs[0], want, bound, "bf16")


def test_linear_marks_infinities_and_nan_like_the_quantiser():
    """Few rows, quantised inside the product: a block with an infinity or a NaN makes its row NaN."""
    rng = np.random.default_rng(9)
    M, N, K = 5, 130, 320
    x = rng.normal(0, 1, (M, K))
    clean = x.copy()
    x[1, 7], x[3, 300] = np.inf, np.nan
    wc, ws, wv = random_mx(rng, N, K, K ** -0.5)
    work = torch.empty(mmact.mmact_linear_mxfp4_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    out = [torch.empty((M, N), dtype=torch.float32, device="cuda") for _ in range(2)]
    mmact.mmact_linear_mxfp4(tensor(x, "bf16"), wc, ws, None, out[0], work)
    mmact.mmact_linear_mxfp4(tensor(clean, "bf16"), wc, ws, None, out[1], work)
    assert torch.isnan(out[0][[1, 3]]).all() and torch.equal(out[0][[0, 2, 4]], out[1][[0, 2, 4]])


def test_calls_on_a_side_stream_and_in_a_graph():
    rng = np.random.default_rng(8)
    M, N, K = 40, 512, 1024
    x = tensor(rng.normal(0, 1, (M, K)), "bf16")
    wc, ws, wv = random_mx(rng, N, K, K ** -0.5)
    work = torch.empty(mmact.mmact_linear_mxfp4_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    C = torch.empty((M, N), dtype=torch.float32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mmact.mmact_linear_mxfp4(x, wc, ws, None, C, work, stream=s)
    s.synchronize()
    want, bound = ref.gemm(ref.quantize(host64(x))[2], wv, None, "none", 0.0)
    check(C, want, bound, "f32")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mmact.mmact_linear_mxfp4(x, wc, ws, None, C, work)
    x2 = rng.normal(0, 1, (M, K))
    x.copy_(tensor(x2, "bf16"))
    C.zero_()
    g.replay()
    torch.cuda.synchronize()
    want, bound = ref.gemm(ref.quantize(host64(x))[2], wv, None, "none", 0.0)
    check(C, want, bound, "f32")
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK


@pytest.mark.parametrize("M,N,K", [(1, 520, 8192), (16, 136, 4100), (100, 400, 2500), (1536, 1280, 640), (2816, 2560, 96)])
def test_gemm_many_k_blocks_and_many_tiles(M, N, K, kernel):
    """K shared by clusters, rings that go round, several tiles for each CTA pair."""
    g = torch.Generator(device="cuda").manual_seed(M + K)
    a, b = (torch.empty((r, K), device="cuda").normal_(0, 1, generator=g) for r in (M, N))
    (ac, as_), (bc, bs) = quantized(a), quantized(b)
    C = torch.full((M, N), float("nan"), dtype=torch.float32, device="cuda")
    mmact.mmact_gemm_mxfp4(ac, as_, bc, bs, None, C, K)
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
    va, vb = torch.empty_like(a), torch.empty_like(b)          # exact (tested above)
    mmact.mmact_dequantize_mxfp4(ac, as_, va)
    mmact.mmact_dequantize_mxfp4(bc, bs, vb)
    va, vb = va.double(), vb.double()
    err, bound = (C.double() - va @ vb.t()).abs(), ref.sum_error(K) * (va.abs() @ vb.abs().t())
    assert bool((err <= bound).all())


def test_long_rows_pass_32_bit_offsets():
    """More than 2^31 values: a matrix whose last rows lie past 32-bit byte and element offsets."""
    rows, K = 70000, 32768
    x = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
    for r in (0, 65536, rows - 1):
        x[r] = torch.arange(K, device="cuda").remainder(13).to(torch.bfloat16) - 6
    codes, scales = quantized(x)
    y = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda")
    mmact.mmact_dequantize_mxfp4(codes, scales, y)
    for r in (0, 65536, rows - 1):
        v = ref.quantize(host64(x[r:r + 1]))[2]
        assert np.array_equal(host64(y[r:r + 1]), v)
    assert int(torch.count_nonzero(y)) == sum(int(torch.count_nonzero(y[r])) for r in (0, 65536, rows - 1))


def test_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    codes = torch.zeros((4, 32), dtype=torch.uint8, device="cuda")
    scales = torch.zeros(512, dtype=torch.uint8, device="cuda")
    C = torch.zeros((4, 4), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        mmact.mmact_quantize_mxfp4(x.cpu(), codes, scales)
    with pytest.raises(TypeError):
        mmact.mmact_quantize_mxfp4(x.int(), codes, scales)
    with pytest.raises(ValueError):
        mmact.mmact_quantize_mxfp4(x.t(), codes, scales)                 # not contiguous
    with pytest.raises(ValueError):
        mmact.mmact_quantize_mxfp4(x, codes[:3], scales)                 # too few codes
    with pytest.raises(ValueError):
        mmact.mmact_quantize_mxfp4(x, codes, scales[:256])
    with pytest.raises(ValueError):
        mmact.mmact_gemm_mxfp4(codes, scales, codes, scales, None, C, 128)   # codes are for K = 64
    with pytest.raises(ValueError):
        mmact.mmact_linear_mxfp4(x, codes, scales, None, C, torch.zeros(512, dtype=torch.uint8, device="cuda"))
    off = torch.zeros(4 * 32 + 8, dtype=torch.uint8, device="cuda")[8:].view(4, 32)
    with pytest.raises(mmact.MmactError) as ei:                          # codes not 16-byte aligned
        mmact.mmact_quantize_mxfp4(x, off, scales)
    assert ei.value.status == mmact.MMACT_ERR_UNSUPPORTED
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
