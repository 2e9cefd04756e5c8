"""The 8-bit products and the router together, as a training step of a feed-forward block uses them: router logits by
the library's product, choice and balance loss, a linear layer in 8 bits for each expert, its backward pass, and the
router's; against the same formulas in fp64 over the 8-bit values, eagerly and as a captured graph."""
import numpy as np
import pytest
import torch

import mx_reference as mx
import route_reference as ref
from conv_activation_epilogue_gb300 import build, mmact

pytestmark = pytest.mark.gpu
T, H, N, E, TOP, COEF = 192, 256, 320, 8, 2, 0.05


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    mmact.load()


def packed(rows, K, kind=torch.float8_e4m3fn):
    c, s = mmact.mmact_fp8_size(rows, K)
    return (torch.zeros((rows, c // rows), dtype=torch.uint8, device="cuda").view(kind),
            torch.zeros(s, dtype=torch.uint8, device="cuda"))


def quantized(x, transposed=False, square=False, kind=torch.float8_e4m3fn):
    q = packed(*(x.shape[::-1] if transposed else x.shape), kind)
    mmact.mmact_quantize_fp8(x, *q, block_rows=128 if square else 1, transposed=transposed)
    return q


def values(q, rows, K):
    y = torch.empty((rows, K), device="cuda")
    mmact.mmact_dequantize_fp8(*q, y)
    return y.double()


class Step:
    """One linear layer to an expert (z_e = q(x) W_e^T), outputs of the chosen experts weighted by their probabilities."""

    def __init__(self):
        g = torch.Generator(device="cuda").manual_seed(5)

        def w(*shape):
            return (torch.randn(shape, generator=g, device="cuda") * shape[-1] ** -0.5).bfloat16()

        self.x, self.dy = w(T, H) * 16, w(T, N)
        self.router = w(H, E)
        self.w = [w(N, H) for _ in range(E)]
        self.q = [quantized(v, square=True) for v in self.w]
        self.qt = [quantized(v, transposed=True, square=True) for v in self.w]     # W turned round, the same values
        self.logits = torch.empty((T, E), device="cuda")
        self.experts, self.probs = torch.empty((T, TOP), dtype=torch.int32, device="cuda"), torch.empty((T, TOP), device="cuda")
        self.counts, self.loss = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(1, device="cuda")
        self.z = torch.empty((E, T, N), dtype=torch.bfloat16, device="cuda")
        self.dz = torch.empty((E, T, N), dtype=torch.bfloat16, device="cuda")
        self.dx = torch.empty((E, T, H), dtype=torch.bfloat16, device="cuda")
        self.dw = torch.empty((E, N, H), device="cuda")
        self.db = torch.empty((E, N), device="cuda")
        self.dprobs, self.dlogits = torch.empty((T, TOP), device="cuda"), torch.empty((T, E), device="cuda")
        self.one = torch.ones(1, device="cuda")
        need = max(mmact.mmact_linear_fp8_workspace_bytes(T, H), mmact.mmact_linear_fp8_backward_workspace_bytes(T, N, H),
                   mmact.mmact_moe_route_workspace_bytes(T, E))
        self.work = torch.empty(need, dtype=torch.uint8, device="cuda")

    def __call__(self):
        mmact.mmact_gemm(self.x, self.router, None, self.logits)
        mmact.mmact_moe_route(self.logits, self.experts, self.probs, self.counts, self.loss, self.work, coef=COEF)
        rows = torch.arange(T, device="cuda").unsqueeze(1)
        for e in range(E):
            mmact.mmact_linear_fp8(self.x, *self.q[e], None, self.z[e], self.work)
        # d(sum dy . y) with y[t] = sum_j probs[t][j] z[experts[t][j]][t]
        chosen = self.z[self.experts.long(), rows].float()
        self.dprobs.copy_((chosen * self.dy.float().unsqueeze(1)).sum(dim=2))
        weight = torch.zeros((T, E), device="cuda").scatter_(1, self.experts.long(), self.probs)
        self.dz.copy_(weight.t().unsqueeze(2) * self.dy.float())
        for e in range(E):
            mmact.mmact_linear_fp8_backward(self.dz[e], self.x, *self.qt[e], self.dx[e], self.dw[e], self.db[e], self.work)
        mmact.mmact_moe_route_backward(self.logits, self.experts, self.counts, self.dprobs, self.one, self.dlogits, coef=COEF)


def check(s):
    z = s.logits.double().cpu().numpy()
    ids, p, n, loss, _ = ref.route(z, TOP, COEF, True)
    assert np.array_equal(s.experts.cpu().numpy(), ids) and np.array_equal(s.counts.cpu().numpy(), n)
    assert np.all(np.abs(s.probs.double().cpu().numpy() - p) <= ref.prob_error(z) * p + ref.TINY)
    assert abs(float(s.loss) - loss) <= (ref.prob_error(z) + (T + E) * 2.0 ** -23) * loss
    xq, xtq = values(quantized(s.x), T, H), values(quantized(s.x, transposed=True), H, T)
    e5 = torch.float8_e5m2
    for e in range(E):
        wq = values(s.q[e], N, H)
        assert torch.equal(wq, values(s.qt[e], H, N).t())
        dq = values(quantized(s.dz[e], kind=e5), T, N)
        dtq = values(quantized(s.dz[e], transposed=True, kind=e5), N, T)
        for got, a, b, half in ((s.z[e], xq, wq.t(), 2.0 ** -8), (s.dx[e], dq, wq, 2.0 ** -8), (s.dw[e], dtq, xtq.t(), 2.0 ** -24)):
            want, bound = a @ b, mx.sum_error(a.shape[1]) * (a.abs() @ b.abs())
            assert bool(((got.double() - want).abs() <= bound + half * (want.abs() + bound) + 2.0 ** -134).all())
        d = s.dz[e].double()
        assert bool(((s.db[e] - d.sum(dim=0)).abs() <= mx.sum_error(T) * d.abs().sum(dim=0)).all())
    want, bound = ref.backward(z, ids, n, s.dprobs.double().cpu().numpy(), 1.0, TOP, COEF, True)
    got = s.dlogits.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= bound + mx.ulp(np.abs(want) + bound, "f32") / 2)
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK


def test_a_training_step():
    s = Step()
    s()
    check(s)


def test_a_training_step_as_a_graph():
    s = Step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s()
    s.x.copy_(torch.flip(s.x, (0, 1)) * 0.75)
    for t in (s.z, s.dx, s.dw, s.db, s.dlogits, s.probs):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    check(s)


def test_two_streams_with_a_workspace_each():
    """The same calls at once on two streams, on different inputs."""
    a, b = Step(), Step()
    b.x.mul_(0.5)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for s, st in ((a, streams[0]), (b, streams[1])):
            with torch.cuda.stream(st):
                s()
    torch.cuda.synchronize()
    check(a)
    check(b)
