"""Calls whose inputs the call before them has just written, back to back on a stream, against
the same calls with a synchronisation after each: bit for bit.  And the sources: no kernel of
these operators reads through the read-only path, which is for data that nobody writes while
the kernel is on the GPU, and theirs may still be written when they start."""
import os
import re

import numpy as np
import pytest
import torch

from conv_activation_epilogue_gb300 import build, mmact
from test_gpu_mxfp4 import host64, quantized, random_mx
import mx_reference as ref

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "conv_activation_epilogue_gb300", "csrc")
SOURCES = ["mxfp4.cu", "mxfp4.cuh", "gemm_mxfp4.cu", "gemm_mxfp4_rows.cu", "moe.cu", "moe.cuh", "moe_mxfp4.cu"]


@pytest.mark.parametrize("name", SOURCES)
def test_no_input_is_read_through_the_read_only_path(name):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert "__ldg" not in code and "global.nc" not in code
    assert not re.search(r"const\s+\w+\s*\*\s*__restrict__", code)     # the compiler's own licence for it


@pytest.fixture(scope="module")
def lib():
    build.build()
    mmact.load()


class Chain:
    """x -> linear -> mixture -> linear -> quantise -> product with itself -> values of the quantised form."""

    def __init__(self, seed, T, D, H, I, E, top, weights):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.K = T, D
        n = lambda *s: torch.randn(s, generator=g, device="cuda") * s[-1] ** -0.5  # noqa: E731
        self.p, self.o = quantized(n(H, D)), quantized(n(D, H))
        self.router, w1, w2 = n(E, H).bfloat16(), n(E * 2 * I, H), n(E * H, I)
        if weights == "mxfp4":
            (self.w1, self.s1), (self.w2, self.s2) = quantized(w1), quantized(w2)
        else:
            self.w1, self.w2, self.s1, self.s2 = w1.bfloat16().view(E, 2 * I, H), w2.bfloat16().view(E, H, I), None, None
        e = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        self.h, self.m, self.y = e(T, H), e(T, H), e(T, D)
        self.ids, self.probs = e(T, top, dtype=torch.int32), e(T, top, dtype=torch.float32)
        nc, ns = mmact.mmact_mxfp4_size(T, D)
        self.codes, self.scales = e(T, nc // T, dtype=torch.uint8), e(ns, dtype=torch.uint8)
        self.c, self.v = e(T, T, dtype=torch.float32), e(T, D)
        need = max(mmact.mmact_linear_mxfp4_workspace_bytes(T, max(D, H)), mmact.mmact_moe_workspace_bytes(T, H, I, E, top))
        self.work = e(need, dtype=torch.uint8)

    def __call__(self, x, after=lambda: None):
        mmact.mmact_linear_mxfp4(x, *self.p, None, self.h, self.work, "silu")
        after()
        mmact.mmact_moe(self.h, self.router, self.w1, self.w2, self.m, self.ids, self.probs, self.work,
                        w1_scales=self.s1, w2_scales=self.s2)
        after()
        mmact.mmact_linear_mxfp4(self.m, *self.o, None, self.y, self.work)
        after()
        mmact.mmact_quantize_mxfp4(self.y, self.codes, self.scales)
        after()
        mmact.mmact_gemm_mxfp4(self.codes, self.scales, self.codes, self.scales, None, self.c, self.K)
        after()
        mmact.mmact_dequantize_mxfp4(self.codes, self.scales, self.v)
        after()
        return [t.clone() for t in (self.h, self.m, self.y, self.c, self.v)]


@pytest.mark.gpu
@pytest.mark.parametrize("weights", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,D,H,I", [(1, 512, 1024, 256), (8, 1024, 512, 128), (40, 520, 1032, 200), (64, 4096, 2048, 64)])
def test_chains_back_to_back(lib, weights, T, D, H, I):
    chain = Chain(T, T, D, H, I, 8, 2, weights)
    g = torch.Generator(device="cuda").manual_seed(T + D)
    xs = [torch.randn((T, D), generator=g, device="cuda").bfloat16() for _ in range(30)]
    want = []
    for x in xs:
        want.append(chain(x, torch.cuda.synchronize))
    torch.cuda.synchronize()
    got = [chain(x) for x in xs]
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(got, want)):
        for name, u, v in zip("hmycv", a, b):
            assert torch.equal(u, v), (i, name)
    assert not torch.equal(want[0][2], want[1][2])
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK


@pytest.mark.gpu
def test_products_on_several_streams(lib):
    """Products whose CTAs share SMs, clusters among them, on four streams at once."""
    rng = np.random.default_rng(3)
    jobs = []
    for M, N, K in ((64, 1024, 4096), (16, 2048, 2048), (40, 640, 8192), (128, 512, 2048)):
        (ac, as_, av), (bc, bs, bv) = random_mx(rng, M, K), random_mx(rng, N, K, K ** -0.5)
        jobs.append((ac, as_, bc, bs, K, ref.gemm(av, bv, None, "none", 0.0), torch.cuda.Stream(),
                     [torch.empty((M, N), dtype=torch.float32, device="cuda") for _ in range(25)]))
    torch.cuda.synchronize()
    for i in range(25):
        for ac, as_, bc, bs, K, _, stream, out in jobs:
            mmact.mmact_gemm_mxfp4(ac, as_, bc, bs, None, out[i], K, stream=stream)
    torch.cuda.synchronize()
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
    for _, _, _, _, _, (want, bound), _, out in jobs:
        assert np.all(np.abs(host64(out[0]) - want) <= bound + ref.ulp(np.abs(want) + bound, "f32"))
        assert all(torch.equal(o, out[0]) for o in out)
