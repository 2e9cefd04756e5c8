"""A block of a language model's feed-forward path held in 4 bits: a projection, a mixture of experts
and an output projection.

    python examples/mixture_block.py [--tokens 1 16 200]

The weights are quantised to MXFP4 once (mmact_quantize_mxfp4); a call then is a linear layer that
quantises its input on the way (mmact_linear_mxfp4), the mixture layer for up to 64 tokens at a time
(mmact_moe) and another linear layer.  Every result is compared with the same formulas in fp64 over
the weights' 4-bit values, and one token is timed as a captured graph, the way a decoder would run it.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from conv_activation_epilogue_gb300 import mmact  # noqa: E402

MOE_TOKENS = 64


class Mxfp4:
    """A matrix [rows, K] in MXFP4."""

    def __init__(self, w: torch.Tensor):
        self.rows, self.K = w.shape
        codes, scales = mmact.mmact_mxfp4_size(self.rows, self.K)
        self.codes = torch.empty((self.rows, codes // self.rows), dtype=torch.uint8, device=w.device)
        self.scales = torch.empty(scales, dtype=torch.uint8, device=w.device)
        mmact.mmact_quantize_mxfp4(w, self.codes, self.scales)

    def values(self) -> torch.Tensor:
        y = torch.empty((self.rows, self.K), dtype=torch.float32, device=self.codes.device)
        mmact.mmact_dequantize_mxfp4(self.codes, self.scales, y)
        return y


class MixtureBlock:
    """y = out(moe(silu(proj(x)))): proj [H, D], router [E, H], w1 [E, 2 I, H], w2 [E, H, I], out [D, H]."""

    def __init__(self, proj, router, w1, w2, out, top: int, max_tokens: int):
        E, I2, H = w1.shape
        self.D, self.H, self.I, self.E, self.top = proj.shape[1], H, I2 // 2, E, top
        self.proj, self.out, self.router = Mxfp4(proj), Mxfp4(out), router
        self.w1, self.w2 = Mxfp4(w1.reshape(E * I2, H)), Mxfp4(w2.reshape(E * H, self.I))
        dev, n = proj.device, max_tokens
        self.h = torch.empty((n, H), dtype=torch.bfloat16, device=dev)          # between the layers
        self.m = torch.empty((n, H), dtype=torch.bfloat16, device=dev)
        self.experts = torch.empty((n, top), dtype=torch.int32, device=dev)
        self.probs = torch.empty((n, top), dtype=torch.float32, device=dev)
        need = max(mmact.mmact_linear_mxfp4_workspace_bytes(n, max(self.D, H)),
                   mmact.mmact_moe_workspace_bytes(min(n, MOE_TOKENS), H, self.I, E, top))
        self.workspace = torch.empty(need, dtype=torch.uint8, device=dev)

    def __call__(self, x: torch.Tensor, y: torch.Tensor) -> None:
        n = x.shape[0]
        h, m = self.h[:n], self.m[:n]
        mmact.mmact_linear_mxfp4(x, self.proj.codes, self.proj.scales, None, h, self.workspace, "silu")
        for t in range(0, n, MOE_TOKENS):
            s = slice(t, min(n, t + MOE_TOKENS))
            mmact.mmact_moe(h[s], self.router, self.w1.codes, self.w2.codes, m[s], self.experts[s], self.probs[s],
                            self.workspace, "silu", w1_scales=self.w1.scales, w2_scales=self.w2.scales)
        mmact.mmact_linear_mxfp4(m, self.out.codes, self.out.scales, None, y, self.workspace)

    def plain(self, x: torch.Tensor):
        """The same in fp64, each layer over what the layer before it gave here; (h, m, y)."""
        n = x.shape[0]
        h = torch.nn.functional.silu(Mxfp4(x).values().double() @ self.proj.values().double().T)
        m = torch.zeros((n, self.H), dtype=torch.float64, device=x.device)
        w1 = self.w1.values().view(self.E, 2 * self.I, self.H)
        w2 = self.w2.values().view(self.E, self.H, self.I)
        hx = self.h[:n].double()
        logits = hx @ self.router.double().T
        p, ids = torch.topk(logits, self.top, dim=1)
        p = torch.softmax(p, dim=1)
        for e in range(self.E):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            z = hx[t] @ w1[e].double().T
            o = (torch.nn.functional.silu(z[:, :self.I]) * z[:, self.I:]) @ w2[e].double().T
            m.index_add_(0, t, p[t, j, None] * o)
        y = Mxfp4(self.m[:n]).values().double() @ self.out.values().double().T
        return h, m, y


def build(D=1024, H=2048, I=768, E=16, top=4, max_tokens=256, seed=0) -> MixtureBlock:
    g = torch.Generator(device="cuda").manual_seed(seed)

    def w(*shape):
        return (torch.randn(shape, generator=g, device="cuda") * shape[-1] ** -0.5).bfloat16()

    return MixtureBlock(w(H, D), w(E, H), w(E, 2 * I, H), w(E, H, I), w(D, H), top, max_tokens)


def errors(block: MixtureBlock, tokens: int, seed: int = 1):
    """Largest error of each layer's output relative to its largest value."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((tokens, block.D), generator=g, device="cuda").bfloat16()
    y = torch.empty_like(x)
    block(x, y)
    got = (block.h[:tokens], block.m[:tokens], y)
    return [float((a.double() - b).abs().max() / b.abs().max()) for a, b in zip(got, block.plain(x))]


def time_graph(block: MixtureBlock, tokens: int, calls: int = 20) -> float:
    """Microseconds a call, `calls` of them in one graph."""
    x = torch.randn((tokens, block.D), device="cuda").bfloat16()
    y = torch.empty_like(x)
    block(x, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(calls):
            block(x, y)
    graph.replay()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    graph.replay()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) * 1e3 / calls


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, nargs="+", default=[1, 16, 200])
    tokens = ap.parse_args().tokens
    block = build(max_tokens=max(tokens))
    for n in tokens:
        print(f"{n} tokens: largest error of projection, mixture, output (of the largest value): "
              + ", ".join(f"{e:.1e}" for e in errors(block, n)))
    print(f"one token: {time_graph(block, 1):.1f} us a block")


if __name__ == "__main__":
    main()
