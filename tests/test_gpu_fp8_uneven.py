"""Gradients of a linear layer in 8 bits whose two products differ much: one of few tiles over a long K, one of many
tiles over a short K.  Some share a launch, some have one each."""
import pytest
import torch

import mx_reference as mx
from conv_activation_epilogue_gb300 import build, mmact

pytestmark = pytest.mark.gpu
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    mmact.load()


def random(seed, *shape):
    return torch.randn(shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))


def quantized(x, kind=E4, square=False, transposed=False):
    rows, K = x.shape[::-1] if transposed else x.shape
    c, s = mmact.mmact_fp8_size(rows, K)
    q = (torch.empty((rows, c // rows), dtype=torch.uint8, device="cuda").view(kind), torch.empty(s, dtype=torch.uint8, device="cuda"))
    mmact.mmact_quantize_fp8(x, *q, 128 if square else 1, transposed)
    return q


def values(q, rows, K):
    v = torch.empty((rows, K), device="cuda")
    mmact.mmact_dequantize_fp8(*q, v)
    return v.double()


class Layer:
    def __init__(self, M, N, K, dtype=torch.bfloat16, dw=torch.float32):
        self.dims = M, N, K
        self.dy, self.x = random(M, M, N).to(dtype), random(K, M, K).to(dtype)
        self.wt = quantized(random(N, N, K).to(dtype), square=True, transposed=True)
        self.dx, self.dw = torch.empty_like(self.x), torch.empty((N, K), dtype=dw, device="cuda")
        self.db = torch.empty(N, device="cuda")
        self.work = torch.empty(mmact.mmact_linear_fp8_backward_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")

    def __call__(self, dx=True, dw=True, db=True):
        for t in (self.dx, self.dw, self.db):
            t.fill_(float("nan"))
        self.work.fill_(0xFF)
        mmact.mmact_linear_fp8_backward(self.dy, self.x, *self.wt, self.dx if dx else None, self.dw if dw else None,
                                        self.db if db else None, self.work)

    def check(self, dx=True, dw=True, db=True):
        M, N, K = self.dims
        half = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
        # fp16 has steps of 2^-24 below 2^-14: half of one beside the relative half step (the other types' are below 2^-133)
        step = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
        assert mmact.mmact_get_last_error() == mmact.MMACT_OK
        for wanted, got, a, b, n in (
                (dx, self.dx, lambda: values(quantized(self.dy, E5), M, N), lambda: values(self.wt, K, N), N),
                (dw, self.dw, lambda: values(quantized(self.dy, E5, transposed=True), N, M),
                 lambda: values(quantized(self.x, transposed=True), K, M), M)):
            if not wanted:
                assert torch.isnan(got).all()
                continue
            l, r = a(), b()
            want, bound = l @ r.t(), mx.sum_error(n) * (l.abs() @ r.abs().t())
            assert bool(((got.double() - want).abs() <= bound + half[got.dtype] * (want.abs() + bound) + step[got.dtype]).all())
        if db:
            d = self.dy.double()
            assert bool(((self.db - d.sum(dim=0)).abs() <= mx.sum_error(M) * d.abs().sum(dim=0)).all())


# both sides of each rule by which the two products share a launch or do not
SIZES = [(8192, 512, 512), (6144, 512, 512), (4096, 512, 512), (8192, 768, 768), (8192, 1024, 1024), (8192, 768, 2048), (18000, 64, 100),
         (5001, 99, 257), (4000, 99, 257), (256, 8192, 1024), (200, 8000, 300), (100, 6500, 2000), (64, 8192, 512), (128, 6144, 4096),
         (64, 16384, 128), (2048, 1024, 1024), (2048, 512, 512), (1024, 4096, 512), (1, 9000, 130), (20000, 1, 1000),
         (16384, 64, 4096), (12288, 128, 4096), (64, 16384, 4096)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype,dw", [(torch.bfloat16, torch.float32), (torch.float16, torch.bfloat16)])
def test_gradients(M, N, K, dtype, dw):
    s = Layer(M, N, K, dtype, dw)
    s()
    s.check()
    first = s.dx.clone(), s.dw.clone(), s.db.clone()
    s()
    for a, b in zip(first, (s.dx, s.dw, s.db)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("M,N,K", [(8192, 100, 256), (8192, 512, 512), (64, 16384, 128)])
@pytest.mark.parametrize("dx,dw,db", [(True, False, False), (False, True, False), (False, False, True), (False, True, True), (True, False, True)])
def test_wanted_gradients_only(M, N, K, dx, dw, db):
    s = Layer(M, N, K)
    s(dx, dw, db)
    s.check(dx, dw, db)


def test_calls_on_two_streams_and_in_a_graph():
    """One launch each on one stream, a shared launch on the other, at once; then a replayed one with other inputs."""
    a, b = Layer(8192, 512, 512), Layer(2048, 1024, 1024)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        for s, stream in zip((a, b), streams):
            with torch.cuda.stream(stream):
                s()
    torch.cuda.synchronize()
    a.check()
    b.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a()
        b()
    for s in (a, b):
        s.dy.copy_(torch.flip(s.dy, (0, 1)))
        s.x.mul_(0.5)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    a.check()
    b.check()
