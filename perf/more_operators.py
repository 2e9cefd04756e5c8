"""Cases of the products in 8-bit floating point with a scale for each block of 128, and of a
mixture-of-experts router in training.

Each case is one pass through an operator as a program would call it:

  quantize    a tensor is quantised to 8 bits and read back (what a checkpoint or a check of the
              quantisation error does); the values come back
  linear      C = act(q(x) q(W)^T + bias): activations quantised on the way in, weights held in 8 bits
  backward    the gradients of that linear layer: dx = q(dy) q(W), dw = q(dy^T) q(x^T)^T, db = sum of dy
  route       a router's forward pass: choice of experts, their probabilities, how many slots each
              expert got, and the balance loss
  route_grad  its backward pass: the gradient of the logits from those of the probabilities and the loss

With `own` false everything is computed by elementary torch operations in 32 bits; with `own` true
by the library's entry points.

The 8-bit form: 128 consecutive values along K share a power-of-two scale (a byte b, value 2^(b - 127)),
the smallest with which the block's largest value does not pass the type's largest (e4m3 448, e5m2
57344; b is 0 at least); with square blocks, 128 rows share it too.  A row of codes takes K bytes, rounded up to 16
(zeros behind K).  Scales lie in tiles of 512 bytes for 128 rows x 4 blocks (tile [row / 128][block / 4]):
row r, block b at byte (r % 32) * 16 + (r % 128) / 32 * 4 + b % 4; bytes that stand for no row or block are 0.

A router's formulas: logits z [T, E]; a token's slots are the `top` experts of its largest logits, largest
first, the lower index first where they are equal; an expert with logit -inf is never chosen (slot -1,
probability 0), nor any by a token that the mask leaves out.  probs: softmax over the chosen logits, or over all
of them.  counts[e]: slots that chose e; counts[E]: the number n of tokens with a slot.
loss = coef * E * sum over e of counts[e] / (n * top) * (mean over those n tokens of softmax(z)[e]).
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2.0, "bf16": 2.0, "f32": 4.0}
# kind: (torch type, exponent of the largest binade, fraction bits, least exponent)
KINDS = {"e4m3": (torch.float8_e4m3fn, 8, 3, -6), "e5m2": (torch.float8_e5m2, 15, 2, -14)}
MAX_LOGITS = 131072 * 256


# ------------------------------------------------------------------ the cases --
def listed():
    return [
        # a short batch of gradients whose width ends inside a block
        {"name": "quant_ragged", "op": "quantize", "rows": 333, "k": 1000, "dtype": "f16", "kind": "e5m2", "block": 1,
         "trans": False},
        # a weight [K, N] as the 16-bit product takes it, quantised in square blocks when a model is loaded
        {"name": "quant_weight", "op": "quantize", "rows": 8192, "k": 8192, "dtype": "bf16", "kind": "e4m3", "block": 128,
         "trans": True},
        # one token through a wide layer: the weight's bytes are the work
        {"name": "linear_token", "op": "linear", "m": 1, "n": 8192, "k": 8192, "dtype": "bf16", "out": "bf16",
         "kind": "e4m3", "block": 128, "act": "gelu", "alpha": 0.0, "bias": True},
        # a decode batch with odd sizes everywhere
        {"name": "linear_ragged", "op": "linear", "m": 77, "n": 4001, "k": 2056, "dtype": "f16", "out": "f16",
         "kind": "e4m3", "block": 1, "act": "relu", "alpha": 0.0, "bias": False},
        # the library's own skinny product: a batch of sequences in decode, fp32 output
        {"name": "linear_skinny", "op": "linear", "m": 128, "n": 8192, "k": 8192, "dtype": "bf16", "out": "f32",
         "kind": "e4m3", "block": 128, "act": "leaky_relu", "alpha": 0.2, "bias": True},
        # a prompt: the library's largest product, bound by the tensor cores
        {"name": "linear_prompt", "op": "linear", "m": 8192, "n": 8192, "k": 8192, "dtype": "bf16", "out": "bf16",
         "kind": "e4m3", "block": 128, "act": "leaky_relu", "alpha": 0.2, "bias": True},
        # gradients of a small layer, sizes off the tiles
        {"name": "backward_ragged", "op": "backward", "m": 333, "n": 1000, "k": 776, "dtype": "f16", "grad": "f32",
         "kind": "e5m2", "block": 128},
        # a training step's batch of tokens through a wide layer
        {"name": "backward_batch", "op": "backward", "m": 8192, "n": 4096, "k": 4096, "dtype": "bf16", "grad": "f32",
         "kind": "e4m3", "block": 128},
        # the most tokens that the mixture layer takes at once: latency
        {"name": "route_few", "op": "route", "t": 64, "e": 64, "top": 8, "dtype": "bf16", "norm": True, "mask": False,
         "closed": False},
        # a training step's tokens over many experts, fp32 logits
        {"name": "route_batch", "op": "route", "t": 131072, "e": 256, "top": 8, "dtype": "f32", "norm": True,
         "mask": False, "closed": False},
        # a padded batch with an odd number of experts, some of them closed to some tokens
        {"name": "route_grad_ragged", "op": "route_grad", "t": 1237, "e": 21, "top": 2, "dtype": "f16", "norm": False,
         "mask": True, "closed": True},
        # the backward pass of the same training step
        {"name": "route_grad_batch", "op": "route_grad", "t": 131072, "e": 256, "top": 8, "dtype": "f32", "norm": True,
         "mask": False, "closed": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "backward", "route", "route_grad"])
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 8192), "k": _log(rng, 32, 8192), "dtype": rng.choice(["bf16", "f16", "f32"]),
                "kind": rng.choice(["e4m3", "e4m3", "e5m2"]), "block": rng.choice([1, 128]), "trans": rng.random() < 0.5}
    if op == "linear":
        m, n, k = _log(rng, 1, 8192), _log(rng, 64, 8192), _log(rng, 64, 8192)
        return {"op": op, "m": m, "n": n, "k": k, "dtype": rng.choice(["bf16", "f16", "f32"]),
                "out": rng.choice(["bf16", "bf16", "f16", "f32"]), "kind": rng.choice(["e4m3", "e4m3", "e5m2"]),
                "block": rng.choice([1, 128, 128]), "act": rng.choice(["none", "relu", "leaky_relu", "gelu", "silu"]),
                "alpha": 0.1, "bias": rng.random() < 0.7}
    if op == "backward":
        return {"op": op, "m": _log(rng, 1, 8192), "n": _log(rng, 64, 4096), "k": _log(rng, 64, 4096),
                "dtype": rng.choice(["bf16", "f16", "f32"]), "grad": rng.choice(["f32", "f32", "bf16"]),
                "kind": rng.choice(["e4m3", "e5m2"]), "block": rng.choice([1, 128, 128])}
    e = _log(rng, 4, 512)
    return {"op": op, "t": _log(rng, 1, min(131072, MAX_LOGITS // e)), "e": e, "top": rng.randint(1, min(16, e)),
            "dtype": rng.choice(["f32", "bf16", "f16"]), "norm": rng.random() < 0.6, "mask": rng.random() < 0.3,
            "closed": rng.random() < 0.3}


# ----------------------------------------------------- the 8-bit form, plain form --
def _power(n):
    """2^n in fp32 for whole n in -127..127, from its bits (2^-127 is subnormal)."""
    return torch.where(n <= -127, 0x400000, (n + 127) << 23).view(torch.float32)


def _quantize(x, kind, block):
    """x [rows, K] fp32 -> (value multiples [rows, K] fp32, scale exponents [rows, blocks])."""
    _, top, bits, low = KINDS[kind]
    rows, k = x.shape
    blocks = (k + 127) // 128
    a = torch.nn.functional.pad(x.abs(), (0, blocks * 128 - k)).view(rows, blocks, 128).amax(dim=2)
    if block == 128:
        full = torch.nn.functional.pad(a, (0, 0, 0, -rows % 128)).view(-1, 128, blocks)
        a = full.amax(dim=1).repeat_interleave(128, dim=0)[:rows]
    part, e = torch.frexp(a)                                  # a = part * 2^e, part in [0.5, 1)
    e = e - 1 - top + (part > 0.875).int()                    # 1.75 is the largest part of both types
    e = torch.where(a > 0, e, -127).clamp(min=-127)
    v = x * _power(-e).repeat_interleave(128, dim=1)[:, :k]   # exact
    step = _power((torch.frexp(v)[1] - 1).clamp(min=low) - bits)
    return (v / step).round() * step, e                       # round() is to nearest even


def _values(x, kind, block):
    """What x [rows, K] reads back as from 8 bits, in fp32."""
    q, e = _quantize(x.float(), kind, block)
    return q * _power(e).repeat_interleave(128, dim=1)[:, : q.shape[1]]


def _scale_place(rows, blocks, device):
    """Byte of each (row, block)'s scale in the tiled scales."""
    r = torch.arange(rows, device=device).unsqueeze(1)
    b = torch.arange(blocks, device=device).unsqueeze(0)
    tiles = (blocks + 3) // 4
    return ((r // 128) * tiles + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4


def _empty(rows, k, kind):
    """Room for a matrix [rows, K] in 8 bits: (codes, tiled scales)."""
    return (torch.zeros((rows, (k + 15) // 16 * 16), dtype=torch.uint8, device="cuda").view(KINDS[kind][0]),
            torch.zeros((rows + 127) // 128 * ((k + 511) // 512) * 512, dtype=torch.uint8, device="cuda"))


def _pack(x, kind, block):
    """x [rows, K] -> (codes, tiled scales) as a program holds them."""
    q, e = _quantize(x.float(), kind, block)
    codes, scales = _empty(*x.shape, kind)
    codes.view(torch.uint8)[:, : x.shape[1]] = q.to(KINDS[kind][0]).view(torch.uint8)
    scales[_scale_place(e.shape[0], e.shape[1], x.device).view(-1)] = (e + 127).to(torch.uint8).view(-1)
    return codes, scales


def _unpack(codes, scales, k):
    """Values [rows, k] in fp32 of the packed form."""
    rows, blocks = codes.shape[0], (k + 127) // 128
    e = scales[_scale_place(rows, blocks, codes.device)].int() - 127
    return codes.view(torch.uint8)[:, :k].view(codes.dtype).float() * _power(e).repeat_interleave(128, dim=1)[:, :k]


# ------------------------------------------------------------------ the inputs --
def _normal(gen, shape, dtype, std=1.0):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen).to(dtype)


def _spread(gen, x, dim):
    """Slices of x along `dim` over a few powers of two: tokens and rows of a model differ in size."""
    n = x.shape[dim]
    size = torch.exp2(torch.empty(n, device="cuda").uniform_(-6.0, 6.0, generator=gen))
    return (x.float() * (size if dim == 1 else size.unsqueeze(1))).to(x.dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case}
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "quantize":
        rows, k = case["rows"], case["k"]
        s["x"] = _spread(gen, _normal(gen, (k, rows) if case["trans"] else (rows, k), dt), 1 if case["trans"] else 0)
        s["codes"], s["scales"] = _empty(rows, k, case["kind"])
        s["y"] = torch.empty((rows, k), dtype=dt, device="cuda")
    elif op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        s["x"] = _normal(gen, (m, k), dt)
        s["codes"], s["scales"] = _pack(_normal(gen, (n, k), torch.bfloat16, k ** -0.5), case["kind"], case["block"])
        s["bias"] = _normal(gen, (n,), torch.float32, 0.5) if case["bias"] else None
        s["c"] = torch.empty((m, n), dtype=DTYPES[case["out"]], device="cuda")
    elif op == "backward":
        m, n, k = case["m"], case["n"], case["k"]
        s["x"] = _normal(gen, (m, k), dt)
        s["dy"] = _spread(gen, _normal(gen, (m, n), dt, m ** -0.5), 0)
        # W [N, K] as the forward pass has it, turned round once a step: [K, N], blocks along N
        s["codes"], s["scales"] = _pack(_normal(gen, (k, n), torch.bfloat16, k ** -0.5), case["kind"], case["block"])
        s["dx"] = torch.empty((m, k), dtype=dt, device="cuda")
        s["dw"] = torch.empty((n, k), dtype=DTYPES[case["grad"]], device="cuda")
        s["db"] = torch.empty(n, dtype=torch.float32, device="cuda")
    else:
        t, e, top = case["t"], case["e"], case["top"]
        # some experts are liked by all tokens
        z = _normal(gen, (t, e), torch.float32, 1.5) + _normal(gen, (e,), torch.float32, 0.7)
        if case["closed"]:
            z = torch.where(torch.rand((t, e), device="cuda", generator=gen) < 0.4, -math.inf, z)
        s["z"] = z.to(dt)
        s["mask"] = None
        if case["mask"]:
            s["mask"] = (torch.rand(t, device="cuda", generator=gen) < 0.8).to(torch.uint8)
        s["experts"] = torch.empty((t, top), dtype=torch.int32, device="cuda")
        s["probs"] = torch.empty((t, top), dtype=torch.float32, device="cuda")
        s["counts"] = torch.empty(e + 1, dtype=torch.int32, device="cuda")
        s["loss"] = torch.empty(1, dtype=torch.float32, device="cuda")
        if op == "route_grad":
            out = _plain_route(s)
            s["experts"], s["probs"], s["counts"] = out["experts"], out["probs"], out["counts"]
            s["dprobs"] = _normal(gen, (t, top), torch.float32, 0.1)
            s["dloss"] = torch.empty(1, device="cuda").uniform_(0.5, 2.0, generator=gen)
            s["dz"] = torch.empty_like(s["z"])
    return s


# ------------------------------------------------------------------- one pass --
COEF = 0.01


def _act(z, name, alpha):
    if name == "relu":
        return z.clamp(min=0.0)
    if name == "leaky_relu":
        return torch.where(z > 0, z, alpha * z)
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * 0.7071067811865476))
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _shares(s):
    """exp(z - largest) [T, E] and its sum [T, 1]; rows that choose nothing are all 0 with the sum 1."""
    z = s["z"].float()
    peak = z.amax(dim=1, keepdim=True)
    ok = peak > -math.inf
    if s["mask"] is not None:
        ok = ok & (s["mask"] != 0).unsqueeze(1)
    ex = torch.where(ok, torch.exp(z - torch.where(ok, peak, 0.0)), 0.0)
    return ex, torch.where(ok, ex.sum(dim=1, keepdim=True), 1.0), ok


def _plain_route(s):
    case, z = s["case"], s["z"].float()
    e, top = case["e"], case["top"]
    best, experts = torch.sort(z, dim=1, descending=True, stable=True)      # equal logits: the lowest index first
    best, experts = best[:, :top], experts[:, :top]
    ex, total, ok = _shares(s)
    chosen = ok & (best > -math.inf)
    mine = torch.where(chosen, ex.gather(1, experts), 0.0)
    over = torch.where(ok, mine.sum(dim=1, keepdim=True), 1.0) if case["norm"] else total
    experts = torch.where(chosen, experts, -1)
    counts = (experts.reshape(-1, 1) == torch.arange(e, device=z.device)).sum(dim=0) if z.numel() <= 1 << 22 else \
        torch.zeros(e + 1, dtype=torch.int64, device=z.device).index_add_(
            0, torch.where(chosen, experts, e).reshape(-1), torch.ones(experts.numel(), dtype=torch.int64, device=z.device))[:e]
    n = ok.sum()
    share = (ex / total).sum(dim=0, dtype=torch.float64)
    loss = COEF * e * (counts * share).sum() / (n * n * top).clamp(min=1)
    return {"experts": experts.int(), "probs": mine / over, "counts": torch.cat((counts, n.view(1))).int(),
            "loss": loss.float().view(1)}


def _plain_route_grad(s):
    case = s["case"]
    e, top = case["e"], case["top"]
    ex, total, ok = _shares(s)
    p = ex / total
    counts = s["counts"][:e].float()
    n = s["counts"][e].double()
    scale = (COEF * e / (n * n * top).clamp(min=1) * s["dloss"]).float()
    dz = scale * p * (counts - (p * counts).sum(dim=1, keepdim=True))
    chosen = s["experts"] >= 0
    at = s["experts"].clamp(min=0).long()
    g = torch.where(chosen, s["dprobs"], 0.0)
    mine = torch.where(chosen, ex.gather(1, at), 0.0)
    if case["norm"]:
        mine = mine / torch.where(ok, mine.sum(dim=1, keepdim=True), 1.0)
        dz.scatter_add_(1, at, mine * (g - (mine * g).sum(dim=1, keepdim=True)))
    else:
        mine = mine / total
        dz = dz - p * (mine * g).sum(dim=1, keepdim=True)
        dz.scatter_add_(1, at, mine * g)
    return dz.to(s["z"].dtype)


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        from conv_activation_epilogue_gb300 import mmact
        if op == "quantize":
            mmact.mmact_quantize_fp8(s["x"], s["codes"], s["scales"], block_rows=case["block"], transposed=case["trans"])
            mmact.mmact_dequantize_fp8(s["codes"], s["scales"], s["y"])
            return s["y"]
        if op == "linear":
            if "work" not in s:
                s["work"] = torch.empty(mmact.mmact_linear_fp8_workspace_bytes(case["m"], case["k"]), dtype=torch.uint8,
                                        device="cuda")
            mmact.mmact_linear_fp8(s["x"], s["codes"], s["scales"], s["bias"], s["c"], s["work"], case["act"], case["alpha"])
            return s["c"]
        if op == "backward":
            if "work" not in s:
                s["work"] = torch.empty(mmact.mmact_linear_fp8_backward_workspace_bytes(case["m"], case["n"], case["k"]),
                                        dtype=torch.uint8, device="cuda")
            mmact.mmact_linear_fp8_backward(s["dy"], s["x"], s["codes"], s["scales"], s["dx"], s["dw"], s["db"], s["work"],
                                            grad_type=KINDS[case["kind"]][0])
            return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}
        if op == "route":
            if "work" not in s:
                s["work"] = torch.empty(mmact.mmact_moe_route_workspace_bytes(case["t"], case["e"]), dtype=torch.uint8,
                                        device="cuda")
            mmact.mmact_moe_route(s["z"], s["experts"], s["probs"], s["counts"], s["loss"], s["work"], coef=COEF,
                                  normalize=case["norm"], mask=s["mask"])
            return {n: s[n] for n in ("experts", "probs", "counts", "loss")}
        mmact.mmact_moe_route_backward(s["z"], s["experts"], s["counts"], s["dprobs"], s["dloss"], s["dz"], coef=COEF,
                                       normalize=case["norm"], mask=s["mask"])
        return s["dz"]
    if op == "quantize":
        x = s["x"].float()
        return _values(x.t() if case["trans"] else x, case["kind"], case["block"]).to(s["x"].dtype)
    if op == "linear":
        z = _values(s["x"], "e4m3", 1) @ _unpack(s["codes"], s["scales"], case["k"]).t()
        if s["bias"] is not None:
            z = z + s["bias"]
        return _act(z, case["act"], case["alpha"]).to(s["c"].dtype)
    if op == "backward":
        dy, x = s["dy"].float(), s["x"].float()
        dx = _values(dy, case["kind"], 1) @ _unpack(s["codes"], s["scales"], case["n"]).t()
        dw = _values(dy.t(), case["kind"], 1) @ _values(x.t(), "e4m3", 1).t()
        return {"dx": dx.to(s["dx"].dtype), "dw": dw.to(s["dw"].dtype), "db": dy.sum(dim=0)}
    return _plain_route(s) if op == "route" else _plain_route_grad(s)


# ---------------------------------------------------------------------- work --
def work(case):
    op, b = case["op"], BYTES[case["dtype"]]
    code = 1.0 + (1.0 / 128.0)
    if op == "quantize":
        n = case["rows"] * case["k"]
        # read x, write the 8-bit form, read it, write the values
        return {"bytes": n * (2 * b + 2 * code), "flops": 4 * n}
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k * b + n * k * code + m * n * BYTES[case["out"]] + 4 * n * case["bias"], "flops": 2 * m * n * k}
    if op == "backward":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m * n + 2 * m * k) * b + n * k * (code + BYTES[case["grad"]]) + 4 * n, "flops": 4 * m * n * k + m * n}
    t, e, top = case["t"], case["e"], case["top"]
    if op == "route":
        return {"bytes": t * e * b + t * top * 8 + t * case["mask"] + 4 * e, "flops": t * e * 6}
    return {"bytes": 2 * t * e * b + t * top * 8 + t * case["mask"] + 4 * e, "flops": t * e * 8}


# ------------------------------------------------------- the definition, 64 bits --
GRIDS = {"e4m3": [0.0] + [(8 + f) * 2.0 ** (p - 10) if p else f * 2.0 ** -9 for p in range(16) for f in range(8)][1:127],
         "e5m2": [0.0] + [(4 + f) * 2.0 ** (p - 17) if p else f * 2.0 ** -16 for p in range(31) for f in range(4)][1:]}


def _rounded64(x, kind, block):
    """x [rows, K] -> its 8-bit values in 64 bits: blocks one after the other, by the grid's midpoints."""
    x = x.double()
    rows, k = x.shape
    grid = torch.tensor(GRIDS[kind], dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    out = torch.empty_like(x)
    for c in range(0, k, 128):
        part = x[:, c: c + 128]
        top = part.abs().max(dim=1, keepdim=True).values
        if block == 128:
            top = torch.cat([t.max().expand(t.shape[0], 1) for t in top.split(128)])
        # the smallest power of two with top / unit <= the grid's largest value, 2^-127 at least
        unit = torch.exp2(torch.ceil(torch.log2((top / grid[-1]).clamp(min=2.0 ** -140))).clamp(min=-127.0))
        unit = torch.where(top > unit * grid[-1], unit * 2, unit)
        unit = torch.where((top <= unit / 2 * grid[-1]) & (unit > 2.0 ** -127), unit / 2, unit)
        a = part.abs() / unit
        down = torch.searchsorted(mid, a.contiguous())        # mid[i - 1] < a <= mid[i]
        up = torch.searchsorted(mid, a.contiguous(), right=True)
        code = torch.where(down % 2 == 0, down, up)           # on a midpoint: the even code
        out[:, c: c + 128] = grid[code] * torch.sign(part) * unit
    return out


def _values64(codes, scales, k):
    """Values [rows, k] in 64 bits of the packed form, row blocks of 128 taken from their tiles."""
    rows, blocks = codes.shape[0], -(-k // 128)
    tiles = -(-blocks // 4)
    t = scales.view(-1, tiles, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, tiles * 4)[:rows, :blocks]
    c = codes.view(torch.uint8)[:, :k].long()
    kind = "e4m3" if codes.dtype == torch.float8_e4m3fn else "e5m2"
    grid = torch.tensor(GRIDS[kind] + [math.nan] * (128 - len(GRIDS[kind])), dtype=torch.float64, device=codes.device)
    unit = torch.tensor([2.0 ** (b - 127) for b in range(256)], dtype=torch.float64, device=codes.device)[t.long()]
    return grid[c % 128] * (1.0 - 2.0 * (c >= 128)) * unit.repeat_interleave(128, dim=1)[:, :k]


def _act64(z, name, alpha):
    if name == "relu":
        return torch.maximum(z, torch.zeros_like(z))
    if name == "leaky_relu":
        return torch.maximum(z, torch.zeros_like(z)) + alpha * torch.minimum(z, torch.zeros_like(z))
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def _route64(s):
    """(experts, their probabilities, softmax over all, chosen slots, tokens that count) in 64 bits."""
    case, z = s["case"], s["z"].double()
    on = torch.isfinite(z).any(dim=1)
    if s["mask"] is not None:
        on = on & s["mask"].bool()
    order = torch.argsort(-z, dim=1, stable=True)[:, : case["top"]]
    p = torch.softmax(torch.where(on.unsqueeze(1), z, torch.zeros_like(z)), dim=1) * on.unsqueeze(1)
    slot = on.unsqueeze(1) & torch.isfinite(z.gather(1, order))
    share = p.gather(1, order) * slot
    if case["norm"]:
        share = share / share.sum(dim=1, keepdim=True).clamp(min=1e-300)
    return torch.where(slot, order, torch.full_like(order, -1)), share, p, slot, on


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _rounded64(s["x"].t() if case["trans"] else s["x"], case["kind"], case["block"])
    if op == "linear":
        z = _rounded64(s["x"], "e4m3", 1) @ _values64(s["codes"], s["scales"], case["k"]).t()
        if s["bias"] is not None:
            z += s["bias"].double()
        return _act64(z, case["act"], case["alpha"])
    if op == "backward":
        dx = _rounded64(s["dy"], case["kind"], 1) @ _values64(s["codes"], s["scales"], case["n"]).t()
        dw = _rounded64(s["dy"].t(), case["kind"], 1) @ _rounded64(s["x"].t(), "e4m3", 1).t()
        return {"dx": dx, "dw": dw, "db": s["dy"].double().sum(dim=0)}
    e, top = case["e"], case["top"]
    experts, share, p, slot, on = _route64(s)
    counts = torch.bincount((experts + 1).flatten(), minlength=e + 1)[1:]
    n = max(int(on.sum()), 1)
    if op == "route":
        loss = COEF * e * (counts.double() / (n * top) * (p.sum(dim=0) / n)).sum()
        return {"experts": experts.int(), "probs": share, "counts": torch.cat((counts, on.sum().view(1))).int(),
                "loss": loss.view(1)}
    # d loss / d p is the same row for every token; d probs / d z by the softmax's own formula
    up = COEF * e / (n * n * top) * counts.double() * float(s["dloss"])
    dz = p * (up - p @ up.unsqueeze(1))
    g = s["dprobs"].double() * slot
    if case["norm"]:
        add = share * (g - (share * g).sum(dim=1, keepdim=True))
        return dz.scatter_add_(1, experts.clamp(min=0), add)
    full = torch.zeros_like(p).scatter_add_(1, experts.clamp(min=0), g)
    return dz + p * (full - (p * full).sum(dim=1, keepdim=True))
