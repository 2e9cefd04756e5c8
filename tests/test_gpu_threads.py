"""Calls from threads that have made no CUDA call before."""
import threading

import pytest
import torch

from conv_activation_epilogue_gb300 import build, mmact

pytestmark = pytest.mark.gpu
M, N, K = 256, 256, 512


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    mmact.load()


def fp8(x, **how):
    rows, k = x.shape[::-1] if how.get("transposed") else x.shape
    c, s = mmact.mmact_fp8_size(rows, k)
    q = torch.empty((rows, c // rows), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn), torch.empty(s, dtype=torch.uint8, device="cuda")
    mmact.mmact_quantize_fp8(x, *q, **how)
    return q


def mxfp4(x):
    c, s = mmact.mmact_mxfp4_size(*x.shape)
    q = torch.empty(c, dtype=torch.uint8, device="cuda"), torch.empty(s, dtype=torch.uint8, device="cuda")
    mmact.mmact_quantize_mxfp4(x, *q)
    return q


def operators():
    """name -> (call on a stream, its outputs)"""
    g = torch.Generator(device="cuda").manual_seed(0)
    x, w, dy = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((M, K), (N, K), (M, N)))
    wt = w.t().contiguous()
    out = {n: torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for n in ("gemm", "gemm_fp8", "linear_fp8", "gemm_mxfp4", "linear_mxfp4")}
    a8, b8, t8, a4, b4 = fp8(x), fp8(w), fp8(w, transposed=True), mxfp4(x), mxfp4(w)
    work = {n: torch.empty(1 << 22, dtype=torch.uint8, device="cuda") for n in ("linear_fp8", "linear_mxfp4", "backward", "route")}
    dx, dw, db = torch.empty_like(x), torch.empty((N, K), device="cuda"), torch.empty(N, device="cuda")
    z = torch.randn((M, 40), generator=g, device="cuda")
    experts, probs = torch.empty((M, 2), dtype=torch.int32, device="cuda"), torch.empty((M, 2), device="cuda")
    counts, loss = torch.empty(41, dtype=torch.int32, device="cuda"), torch.empty(1, device="cuda")
    return {
        "gemm": (lambda s: mmact.mmact_gemm(x, wt, None, out["gemm"], stream=s), [out["gemm"]]),
        "gemm_fp8": (lambda s: mmact.mmact_gemm_fp8(*a8, *b8, None, out["gemm_fp8"], K, stream=s), [out["gemm_fp8"]]),
        "linear_fp8": (lambda s: mmact.mmact_linear_fp8(x, *b8, None, out["linear_fp8"], work["linear_fp8"], stream=s), [out["linear_fp8"]]),
        "backward": (lambda s: mmact.mmact_linear_fp8_backward(dy, x, *t8, dx, dw, db, work["backward"], stream=s), [dx, dw, db]),
        "gemm_mxfp4": (lambda s: mmact.mmact_gemm_mxfp4(*a4, *b4, None, out["gemm_mxfp4"], K, stream=s), [out["gemm_mxfp4"]]),
        "linear_mxfp4": (lambda s: mmact.mmact_linear_mxfp4(x, *b4, None, out["linear_mxfp4"], work["linear_mxfp4"], stream=s),
                         [out["linear_mxfp4"]]),
        "route": (lambda s: mmact.mmact_moe_route(z, experts, probs, counts, loss, work["route"], stream=s), [experts, probs, counts, loss]),
    }


@pytest.mark.parametrize("name", ["gemm", "gemm_fp8", "linear_fp8", "backward", "gemm_mxfp4", "linear_mxfp4", "route"])
def test_a_threads_first_cuda_call(name):
    call, outputs = operators()[name]
    stream = torch.cuda.Stream()
    call(stream)
    stream.synchronize()
    want = [t.clone() for t in outputs]
    for t in outputs:
        t.zero_()
    torch.cuda.synchronize()
    errors = []

    def run():
        try:
            call(stream)
        except Exception as e:
            errors.append(e)

    for _ in range(2):
        thread = threading.Thread(target=run)
        thread.start()
        thread.join()
    assert not errors, errors
    stream.synchronize()
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
    for got, w in zip(outputs, want):
        assert torch.equal(got, w)


def test_threads_at_once():
    """Each its own operator, stream and workspace."""
    every = operators()
    streams = {n: torch.cuda.Stream() for n in every}
    torch.cuda.synchronize()
    for n, (call, _) in every.items():
        call(streams[n])
    torch.cuda.synchronize()
    want = {n: [t.clone() for t in outputs] for n, (_, outputs) in every.items()}
    torch.cuda.synchronize()
    errors = []

    def run(n):
        try:
            for _ in range(5):
                every[n][0](streams[n])
        except Exception as e:
            errors.append((n, e))

    threads = [threading.Thread(target=run, args=(n,)) for n in every]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for n, (_, outputs) in every.items():
        for got, w in zip(outputs, want[n]):
            assert torch.equal(got, w)
