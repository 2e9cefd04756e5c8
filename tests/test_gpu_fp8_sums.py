"""Sums over long K into fp32 in 8 bits.  The tensor core cuts off what an addition to its accumulator has below the last
bit, always towards zero, so that the outputs of positive products all come out too small, the longer the accumulator's K the
more: an accumulator takes 16 K blocks at most (2048 values), whatever the kernel, the split of K over CTAs and the other product
of a launch.

Bounds, with the 32 products of an instruction counted as one addition.  An accumulator takes 64 of them.  Each cuts off
a part of 2^-23 of the sum so far, spread evenly: half of it on average; the sum so far grows evenly from nothing: half of the
whole on average.  So the outputs' mean error lies between -64 / 4 and 0 units of 2^-23 of their values; the accumulators' sums
and the bias are added rounded, either way alike: a unit more on both sides.  A single output: no more than 2^-23 at each
addition, half of the whole on average, 32 units; and at most one for each accumulator's sum, the bias and the output."""
import pytest
import torch

from conv_activation_epilogue_gb300 import build, mmact

pytestmark = pytest.mark.gpu
UNIT = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    mmact.load()


@pytest.fixture(params=[0, 1, 2], ids=["chosen", "rows", "pair"])
def kernel(request):
    mmact.mmact_set_gemm_fp8_kernel(request.param)
    yield request.param
    mmact.mmact_set_gemm_fp8_kernel(0)


def positive(seed, *shape):
    """Sizes over many binades, so that most products have bits below the sum's last one."""
    return torch.randn(shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).abs()


def quantized(x, kind=torch.float8_e4m3fn, square=False, transposed=False):
    rows, K = x.shape[::-1] if transposed else x.shape
    c, s = mmact.mmact_fp8_size(rows, K)
    q = (torch.empty((rows, c // rows), dtype=torch.uint8, device="cuda").view(kind), torch.empty(s, dtype=torch.uint8, device="cuda"))
    mmact.mmact_quantize_fp8(x, *q, 128 if square else 1, transposed)
    return q


def values(q, rows, K):
    v = torch.empty((rows, K), device="cuda")
    mmact.mmact_dequantize_fp8(*q, v)
    return v.double()


def check(got, want, K):
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
    rel = (got.double() - want) / want
    units = -(-K // 2048) + 8 + 2                             # accumulators (some are shorter: up to eight CTAs share K), bias, output
    assert float(rel.abs().max()) <= (32 + units) * UNIT
    # rounded additions, each off by half a unit at most, evenly (sigma 0.29): the mean over n outputs is within 4 sigma of 0, that is 1.16
    # (units / n)^0.5, less than 1 here
    assert units / rel.numel() <= 1 / 2
    assert -17 * UNIT <= float(rel.mean()) <= UNIT


@pytest.mark.parametrize("M,N,K", [(256, 384, 131072), (512, 512, 65536), (128, 300, 40000), (100, 130, 100001), (60, 200, 70000),
                                   (30, 264, 65536), (16, 640, 131072), (9, 1000, 33000), (300, 257, 36864)])
def test_products_of_long_k(M, N, K, kernel):
    a, b, bias = positive(M, M, K), positive(N, N, K), positive(K, N)
    qa, qb = quantized(a), quantized(b)
    C = torch.full((M, N), float("nan"), device="cuda")
    mmact.mmact_gemm_fp8(*qa, *qb, bias, C, K, "leaky_relu", 0.5)
    check(C, values(qa, M, K) @ values(qb, N, K).t() + bias.double(), K)


@pytest.mark.parametrize("M,N,K", [(256, 384, 65536), (128, 640, 8192), (300, 257, 36864), (40, 264, 32768), (12, 640, 16384)])
def test_long_k_is_no_worse_than_products_of_2048(M, N, K, kernel):
    """Closer than the bound above: the mean error is the mean over the accumulators, so no worse than that of products of 2048 K
    each in one accumulator, but for rounded additions (a unit)."""
    a, b = positive(M, M, K), positive(N, N, K)

    def mean(lo, hi):
        qa, qb = quantized(a[:, lo:hi].contiguous()), quantized(b[:, lo:hi].contiguous())
        C = torch.full((M, N), float("nan"), device="cuda")
        mmact.mmact_gemm_fp8(*qa, *qb, None, C, hi - lo)
        want = values(qa, M, hi - lo) @ values(qb, N, hi - lo).t()
        return float(((C.double() - want) / want).mean())

    whole = mean(0, K)
    mmact.mmact_set_gemm_fp8_kernel(2)                        # one accumulator for 2048 K
    parts = [mean(lo, lo + 2048) for lo in range(0, K, 2048)]
    assert whole >= sum(parts) / len(parts) - UNIT


@pytest.mark.parametrize("M,N,K", [(1, 1000, 131072), (3, 333, 70000), (8, 520, 65536), (8, 128, 40003)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_rows_quantised_inside_over_long_k(M, N, K, dtype):
    x, w = positive(M, M, K).to(dtype), positive(N, N, K)
    q = quantized(w)
    C = torch.full((M, N), float("nan"), device="cuda")
    work = torch.full((mmact.mmact_linear_fp8_workspace_bytes(M, K),), 0xFF, dtype=torch.uint8, device="cuda")
    mmact.mmact_linear_fp8(x, *q, None, C, work, "relu")
    check(C, values(quantized(x), M, K) @ values(q, N, K).t(), K)


# Few outputs over many tokens or many columns beside a product with one or two K blocks, either way round; one product alone.
BACKWARDS = [(8192, 100, 256), (18000, 64, 100), (64, 16384, 128), (64, 8192, 512), (8192, 512, 512), (40000, 200, 300), (100, 40000, 130),
             (131072, 100, 130), (3, 33000, 70)]


def gradients(dy, x, wt, want):
    (M, N), K = dy.shape, x.shape[1]
    nan = float("nan")
    dx = torch.full((M, K), nan, device="cuda") if "dx" in want else None
    dw = torch.full((N, K), nan, device="cuda") if "dw" in want else None
    db = torch.full((N,), nan, device="cuda")
    work = torch.full((mmact.mmact_linear_fp8_backward_workspace_bytes(M, N, K),), 0xFF, dtype=torch.uint8, device="cuda")
    mmact.mmact_linear_fp8_backward(dy, x, *wt, dx, dw, db, work, grad_type=torch.float8_e4m3fn)
    return dx, dw


@pytest.mark.parametrize("M,N,K", BACKWARDS)
@pytest.mark.parametrize("want", ["dx dw", "dx", "dw"])
def test_gradients_of_uneven_sizes(M, N, K, want, kernel):
    dy, x = positive(M, M, N), positive(K, M, K)
    wt = quantized(positive(N, K, N))
    dx, dw = gradients(dy, x, wt, want.split())
    if dx is not None:
        check(dx, values(quantized(dy), M, N) @ values(wt, K, N).t(), N)
    if dw is not None:
        check(dw, values(quantized(dy, transposed=True), N, M) @ values(quantized(x, transposed=True), K, M).t(), M)


def test_gradients_of_uneven_sizes_in_a_graph():
    M, N, K = 18000, 64, 100
    dy, x, wt = positive(1, M, N), positive(2, M, K), quantized(positive(3, K, N))
    dx, dw, db = torch.empty((M, K), device="cuda"), torch.empty((N, K), device="cuda"), torch.empty(N, device="cuda")
    work = torch.empty(mmact.mmact_linear_fp8_backward_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
    mmact.mmact_linear_fp8_backward(dy, x, *wt, dx, dw, db, work)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mmact.mmact_linear_fp8_backward(dy, x, *wt, dx, dw, db, work)
    dy.copy_(positive(4, M, N))
    work.fill_(0xFF)
    dw.zero_()
    g.replay()
    torch.cuda.synchronize()
    again = torch.empty_like(dw)
    mmact.mmact_linear_fp8_backward(dy, x, *wt, torch.empty_like(dx), again, db, work)
    assert torch.equal(dw, again) and mmact.mmact_get_last_error() == mmact.MMACT_OK
    e5 = torch.float8_e5m2
    check(dw, values(quantized(dy, e5, transposed=True), N, M) @ values(quantized(x, transposed=True), K, M).t(), M)
