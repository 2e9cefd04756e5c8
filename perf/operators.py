"""Cases of the 4-bit microscaled (MXFP4) operators and of the mixture-of-experts layer.

Each case is one pass through an operator as a program would call it:

  quantize  a tensor is quantised to MXFP4 and read back (what a cache, a checkpoint or a
            check of the quantisation error does); the values come back
  linear    C = act(q(x) q(W)^T + bias): activations quantised on the way in, weights held in
            MXFP4, the product with fp32 accumulation
  moe       a whole mixture-of-experts layer for a few tokens: router, choice of experts,
            (gated) up product, activation, down product, weighted sum

With `own` false everything is computed by elementary torch operations in 32 bits; with `own`
true by the library's entry points.

MXFP4 here: blocks of 32 values along K share one power-of-two scale (a byte, value 2^(b - 127),
255 = NaN); a value is one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign (codes 0..7, bit 3 the sign),
two to a byte, the even k in the low half.  A row of codes takes ceil(K / 32) * 16 bytes.  Scales
lie in tiles of 512 bytes for 128 rows x 4 blocks (tile [row / 128][block / 4]): row r, block b at
byte (r % 32) * 16 + (r % 128) / 32 * 4 + b % 4; bytes that stand for no row or block are 0.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2.0, "bf16": 2.0, "f32": 4.0, "mxfp4": 0.5 + 1.0 / 32.0}
MAX_MOE_WEIGHTS = 64 * 3 * 1792 * 4096


# ------------------------------------------------------------------ the cases --
def listed():
    return [
        # one token's activations before a product: the smallest call, latency
        {"name": "quant_token", "op": "quantize", "rows": 1, "k": 2048, "dtype": "bf16", "trans": False},
        # a short batch whose width ends inside a block
        {"name": "quant_ragged", "op": "quantize", "rows": 333, "k": 1000, "dtype": "f16", "trans": False},
        # a weight [K, N] as the 16-bit product takes it, quantised along K when a model is loaded
        {"name": "quant_weight", "op": "quantize", "rows": 8192, "k": 8192, "dtype": "bf16", "trans": True},
        # one token through a wide layer: the weight's bytes are the work
        {"name": "linear_token", "op": "linear", "m": 1, "n": 8192, "k": 8192, "dtype": "bf16", "out": "bf16",
         "act": "gelu", "alpha": 0.0, "bias": True},
        # a decode batch with odd sizes everywhere
        {"name": "linear_ragged", "op": "linear", "m": 77, "n": 4001, "k": 2056, "dtype": "f16", "out": "f16",
         "act": "relu", "alpha": 0.0, "bias": False},
        # the library's own sample product, fp32 output
        {"name": "linear_sample", "op": "linear", "m": 1024, "n": 640, "k": 256, "dtype": "f16", "out": "f32",
         "act": "leaky_relu", "alpha": 0.01, "bias": True},
        # the library's own skinny product: a batch of sequences in decode
        {"name": "linear_skinny", "op": "linear", "m": 128, "n": 8192, "k": 8192, "dtype": "bf16", "out": "bf16",
         "act": "leaky_relu", "alpha": 0.2, "bias": True},
        # a prompt: the library's largest product, bound by the tensor cores
        {"name": "linear_prompt", "op": "linear", "m": 8192, "n": 8192, "k": 8192, "dtype": "bf16", "out": "bf16",
         "act": "leaky_relu", "alpha": 0.2, "bias": True},
        # one token, a small layer of many thin experts: latency
        {"name": "moe_token", "op": "moe", "t": 1, "h": 2048, "i": 1024, "e": 64, "top": 8, "dtype": "bf16",
         "weights": "bf16", "act": "silu", "gated": True, "norm": True, "bias": False},
        # a few tokens, plain (ungated) experts with biases, sizes off the tiles
        {"name": "moe_ragged", "op": "moe", "t": 13, "h": 1032, "i": 776, "e": 21, "top": 2, "dtype": "f16",
         "weights": "f16", "act": "gelu", "gated": False, "norm": False, "bias": True},
        # a decode batch over experts held in 4 bits
        {"name": "moe_4bit", "op": "moe", "t": 16, "h": 4096, "i": 2048, "e": 128, "top": 4, "dtype": "bf16",
         "weights": "mxfp4", "act": "silu", "gated": True, "norm": True, "bias": True},
        # the most tokens of the form: every expert is read
        {"name": "moe_batch", "op": "moe", "t": 64, "h": 4096, "i": 1792, "e": 64, "top": 8, "dtype": "bf16",
         "weights": "bf16", "act": "silu", "gated": True, "norm": True, "bias": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "moe", "moe"])
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 8192), "k": _log(rng, 32, 8192),
                "dtype": rng.choice(["bf16", "f16", "f32"]), "trans": rng.random() < 0.5}
    if op == "linear":
        m, n, k = _log(rng, 1, 8192), _log(rng, 64, 8192), _log(rng, 64, 8192)
        return {"op": op, "m": m, "n": n, "k": k, "dtype": rng.choice(["bf16", "f16", "f32"]),
                "out": rng.choice(["bf16", "bf16", "f16", "f32"]),
                "act": rng.choice(["none", "relu", "leaky_relu", "gelu", "silu"]), "alpha": 0.1,
                "bias": rng.random() < 0.7}
    t = _log(rng, 1, 64)
    h, i = 8 * _log(rng, 32, 512), 8 * _log(rng, 32, 256)
    e = _log(rng, 4, 128)
    gated = rng.random() < 0.7
    e = max(4, min(e, MAX_MOE_WEIGHTS // (h * i * 3)))
    dtype = rng.choice(["bf16", "f16"])
    return {"op": op, "t": t, "h": h, "i": i, "e": e, "top": rng.randint(1, min(8, e)), "dtype": dtype,
            "weights": rng.choice([dtype, "mxfp4"]), "act": rng.choice(["silu", "gelu", "relu"]), "gated": gated,
            "norm": rng.random() < 0.7, "bias": rng.random() < 0.5}


# ------------------------------------------------------------- MXFP4, plain form --
def _quantize(x):
    """x [rows, K] fp32 -> (value multiples [rows, blocks, 32] fp32, scale bytes [rows, blocks])."""
    rows, k = x.shape
    blocks = (k + 31) // 32
    if blocks * 32 != k:
        x = torch.nn.functional.pad(x, (0, blocks * 32 - k))
    x = x.view(rows, blocks, 32)
    amax = x.abs().amax(dim=2)
    exponent = torch.frexp(amax)[1] - 3                      # floor(log2(amax)) - 2
    exponent = torch.where(amax > 0, exponent, -127).clamp(min=-127)
    v = x * ((127 - exponent) << 23).view(torch.float32).unsqueeze(2)     # x / 2^exponent, exactly
    a = v.abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    q = ((a / step).round() * step).clamp(max=6.0)           # round() is to nearest even
    return torch.copysign(q, v), (exponent + 127).to(torch.uint8)


def _powers(b):
    """Scale bytes -> fp32 powers of two 2^(b - 127), from their bits (2^-127 is subnormal)."""
    b = b.int()
    return torch.where(b == 0, 0x400000, b << 23).view(torch.float32)


def _codes(q):
    """Value multiples [rows, blocks, 32] -> packed codes [rows, blocks * 16]."""
    a = q.abs()
    c = torch.where(a < 2.0, a * 2.0, torch.where(a < 4.0, a + 2.0, a * 0.5 + 4.0)).to(torch.uint8)
    c = c | (torch.signbit(q).to(torch.uint8) << 3)
    c = c.view(q.shape[0], -1, 2)
    return c[:, :, 0] | (c[:, :, 1] << 4)


def _scale_place(rows, blocks, device):
    """Byte of each (row, block)'s scale in the tiled scales."""
    r = torch.arange(rows, device=device).unsqueeze(1)
    b = torch.arange(blocks, device=device).unsqueeze(0)
    tiles = (blocks + 3) // 4
    return ((r // 128) * tiles + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4


def _scale_bytes(rows, k):
    return (rows + 127) // 128 * ((k + 127) // 128) * 512


def _pack(x):
    """x [rows, K] -> (codes, tiled scales) as a program holds them."""
    q, s = _quantize(x.float())
    tiled = torch.zeros(_scale_bytes(*x.shape), dtype=torch.uint8, device=x.device)
    tiled[_scale_place(s.shape[0], s.shape[1], x.device).view(-1)] = s.view(-1)
    return _codes(q), tiled


def _unpack(codes, scale_bytes, k):
    """Packed codes [..., blocks * 16] and scale bytes [..., blocks] -> fp32 values [..., k]."""
    c = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                        device=codes.device)
    v = grid[c.int()]
    return (v.unflatten(-1, (-1, 32)) * _powers(scale_bytes).unsqueeze(-1)).flatten(-2)[..., :k]


# ------------------------------------------------------------------ the inputs --
def _normal(gen, shape, dtype, std=1.0):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen).to(dtype)


def _experts(gen, case, rows, k):
    """Weights of all experts [E, rows, K]: a tensor, or (codes, scales) of [E * rows, K]."""
    e, std = case["e"], k ** -0.5
    if case["weights"] != "mxfp4":
        w = torch.empty((e, rows, k), dtype=DTYPES[case["weights"]], device="cuda")
        return w.normal_(0.0, std, generator=gen), None
    return _pack(torch.empty((e * rows, k), dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=gen))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "quantize":
        rows, k, dt = case["rows"], case["k"], DTYPES[case["dtype"]]
        s["x"] = _normal(gen, (k, rows) if case["trans"] else (rows, k), dt)
        # rows of a model differ in size: spread them over a few powers of two
        size = torch.exp2(torch.empty(rows, device="cuda").uniform_(-6.0, 6.0, generator=gen))
        s["x"] = (s["x"].float() * (size if case["trans"] else size.unsqueeze(1))).to(dt)
        s["codes"] = torch.empty((rows, (k + 31) // 32 * 16), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(_scale_bytes(rows, k), dtype=torch.uint8, device="cuda")
        s["y"] = torch.empty((rows, k), dtype=dt, device="cuda")
    elif case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        s["x"] = _normal(gen, (m, k), DTYPES[case["dtype"]])
        s["codes"], s["scales"] = _pack(_normal(gen, (n, k), torch.bfloat16, k ** -0.5))
        s["bias"] = _normal(gen, (n,), torch.float32, 0.5) if case["bias"] else None
        s["c"] = torch.empty((m, n), dtype=DTYPES[case["out"]], device="cuda")
        s["work"] = torch.empty(m * ((k + 31) // 32 * 16) + 512 + _scale_bytes(m, k), dtype=torch.uint8, device="cuda")
    else:
        t, h, i, e, dt = case["t"], case["h"], case["i"], case["e"], DTYPES[case["dtype"]]
        up = 2 * i if case["gated"] else i
        s["x"] = _normal(gen, (t, h), dt)
        s["router"] = _normal(gen, (e, h), dt, h ** -0.5)
        s["w1"], s["s1"] = _experts(gen, case, up, h)
        s["w2"], s["s2"] = _experts(gen, case, h, i)
        s["rb"] = s["b1"] = s["b2"] = None
        if case["bias"]:
            s["rb"] = _normal(gen, (e,), torch.float32, 0.2)
            s["b1"] = _normal(gen, (e, up), torch.float32, 0.2)
            s["b2"] = _normal(gen, (e, h), torch.float32, 0.2)
        s["y"] = torch.empty((t, h), dtype=dt, device="cuda")
        s["experts"] = torch.empty((t, case["top"]), dtype=torch.int32, device="cuda")
        s["probs"] = torch.empty((t, case["top"]), dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------------- one pass --
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


def _expert_values(s, name, rows, k, chosen):
    """fp32 weights [n, rows, k] of the experts `chosen` (None: of all)."""
    w, sc = s["w" + name], s["s" + name]
    if sc is None:
        return (w if chosen is None else w[chosen]).float()
    e = s["case"]["e"]
    blocks = (k + 31) // 32
    w = w.view(e, rows, blocks * 16)
    sc = sc[_scale_place(e * rows, blocks, w.device)].view(e, rows, blocks)
    return _unpack(w, sc, k) if chosen is None else _unpack(w[chosen], sc[chosen], k)


def _plain_moe(s):
    case, x = s["case"], s["x"].float()
    t, h, i, e, top = case["t"], case["h"], case["i"], case["e"], case["top"]
    up = 2 * i if case["gated"] else i
    logits = x @ s["router"].float().t()
    if s["rb"] is not None:
        logits = logits + s["rb"]
    best, experts = torch.sort(logits, dim=1, descending=True, stable=True)   # ties: the lowest index first
    best, experts = best[:, :top], experts[:, :top]
    peak = logits.amax(dim=1, keepdim=True)
    over = best if case["norm"] else logits
    probs = torch.exp(best - peak) / torch.exp(over - peak).sum(dim=1, keepdim=True)
    # the chosen experts alone where they are few, every expert otherwise
    few = t * top <= e
    chosen = experts.reshape(-1) if few else None
    w1 = _expert_values(s, "1", up, h, chosen)
    xs = x.repeat_interleave(top, dim=0).unsqueeze(2) if few else x.t().expand(e, h, t)
    z = torch.bmm(w1, xs)                                     # [t * top, up, 1] or [e, up, t]
    del w1
    if s["b1"] is not None:
        z = z + (s["b1"] if chosen is None else s["b1"][chosen]).unsqueeze(2)
    z = _act(z[:, :i], case["act"], 0.0) * z[:, i:] if case["gated"] else _act(z, case["act"], 0.0)
    o = torch.bmm(_expert_values(s, "2", h, i, chosen), z)    # [t * top, h, 1] or [e, h, t]
    if s["b2"] is not None:
        o = o + (s["b2"] if chosen is None else s["b2"][chosen]).unsqueeze(2)
    if few:
        o = o.view(t, top, h)
    else:
        o = o[experts, :, torch.arange(t, device=x.device).unsqueeze(1)]       # [t, top, h]
    y = (probs.unsqueeze(2) * o).sum(dim=1)
    return {"y": y.to(s["x"].dtype), "experts": experts.int(), "probs": probs}


def run(state):
    s, case = state, state["case"]
    if own:
        from conv_activation_epilogue_gb300 import mmact
        if case["op"] == "quantize":
            mmact.mmact_quantize_mxfp4(s["x"], s["codes"], s["scales"], transposed=case["trans"])
            mmact.mmact_dequantize_mxfp4(s["codes"], s["scales"], s["y"])
            return s["y"]
        if case["op"] == "linear":
            mmact.mmact_linear_mxfp4(s["x"], s["codes"], s["scales"], s["bias"], s["c"], s["work"], case["act"],
                                     case["alpha"])
            return s["c"]
        if "work" not in s:
            s["work"] = torch.empty(mmact.mmact_moe_workspace_bytes(case["t"], case["h"], case["i"], case["e"], case["top"]),
                                    dtype=torch.uint8, device="cuda")
        mmact.mmact_moe(s["x"], s["router"], s["w1"], s["w2"], s["y"], s["experts"], s["probs"], s["work"], case["act"],
                        gated=case["gated"], normalize=case["norm"], router_bias=s["rb"], b1=s["b1"], b2=s["b2"],
                        w1_scales=s["s1"], w2_scales=s["s2"])
        return {"y": s["y"], "experts": s["experts"], "probs": s["probs"]}
    if case["op"] == "quantize":
        x = s["x"].float()
        q, b = _quantize(x.t() if case["trans"] else x)
        return (q * _powers(b).unsqueeze(2)).flatten(1)[:, : case["k"]].to(s["x"].dtype)
    if case["op"] == "linear":
        q, b = _quantize(s["x"].float())
        x = (q * _powers(b).unsqueeze(2)).flatten(1)[:, : case["k"]]
        blocks = (case["k"] + 31) // 32
        w = _unpack(s["codes"], s["scales"][_scale_place(case["n"], blocks, x.device)], case["k"])
        z = x @ w.t()
        if s["bias"] is not None:
            z = z + s["bias"]
        return _act(z, case["act"], case["alpha"]).to(s["c"].dtype)
    return _plain_moe(s)


# ---------------------------------------------------------------------- work --
def work(case):
    if case["op"] == "quantize":
        n = case["rows"] * case["k"]
        # read x, write the 4-bit form, read it, write the values
        return {"bytes": n * (2 * BYTES[case["dtype"]] + 2 * BYTES["mxfp4"]), "flops": 4 * n}
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k * BYTES[case["dtype"]] + n * k * BYTES["mxfp4"] + m * n * BYTES[case["out"]] + 4 * n * case["bias"],
                "flops": 2 * m * n * k}
    t, h, i, e, top = (case[n] for n in ("t", "h", "i", "e", "top"))
    each = (3 if case["gated"] else 2) * h * i
    read = e * (1.0 - (1.0 - top / e) ** t)                 # experts that some token chose, expected
    return {"bytes": read * each * BYTES[case["weights"]] + (e * h + 2 * t * h) * BYTES[case["dtype"]],
            "flops": 2 * t * (top * each + e * h)}


# ------------------------------------------------------- the definition, 64 bits --
def _two_to(n):
    """2^n in 64 bits for whole n in (-1023, 1024), exactly."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _nearest(v):
    """|v| to the grid of 4-bit values by its midpoints; a midpoint goes to the even code."""
    a, code = v.abs(), torch.zeros_like(v, dtype=torch.int64)
    for n, mid in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        code += (a > mid) if n % 2 == 0 else (a >= mid)
    return torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=v.device)[code] * torch.sign(v)


def _rounded64(x):
    """x [rows, K] -> its MXFP4 values in 64 bits."""
    x = x.double()
    rows, k = x.shape
    full = torch.zeros((rows, -(-k // 32) * 32), dtype=torch.float64, device=x.device)
    full[:, :k] = x
    full = full.view(rows, -1, 32)
    top = full.abs().max(dim=2, keepdim=True).values
    unit = _two_to(((top.view(torch.int64) >> 52) - 1023 - 2).clamp(min=-127))
    return (_nearest(full / unit) * unit).reshape(rows, -1)[:, :k]


def _values64(codes, scales, rows, k):
    """Values [rows, k] in 64 bits of the packed form, row blocks of 128 taken from their tiles."""
    blocks = -(-k // 32)
    tiles = -(-blocks // 4)
    t = scales.view(-1, tiles, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, tiles * 4)[:rows, :blocks]
    low, high = (codes % 16).double(), (codes // 16).double()
    c = torch.empty((rows, blocks * 32), dtype=torch.float64, device=codes.device)
    c[:, 0::2], c[:, 1::2] = low, high
    sign, c = 1.0 - 2.0 * (c >= 8), c % 8
    v = torch.where(c < 4, c / 2, torch.where(c < 6, c - 2, 2 * c - 8))
    return (sign * v * _two_to(t.long() - 127).repeat_interleave(32, dim=1))[:, :k]


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


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return _rounded64(s["x"].t() if case["trans"] else s["x"])
    if case["op"] == "linear":
        w = _values64(s["codes"], s["scales"], case["n"], case["k"])
        z = _rounded64(s["x"]) @ w.t()
        if s["bias"] is not None:
            z += s["bias"].double()
        return _act64(z, case["act"], case["alpha"])
    t, h, i, top = case["t"], case["h"], case["i"], case["top"]
    up = 2 * i if case["gated"] else i
    x = s["x"].double()
    logits = x @ s["router"].double().t() + (0.0 if s["rb"] is None else s["rb"].double())
    order = torch.argsort(-logits, dim=1, stable=True)[:, :top]
    share = torch.softmax(logits, dim=1).gather(1, order)
    if case["norm"]:
        share = share / share.sum(dim=1, keepdim=True)
    y = torch.zeros((t, h), dtype=torch.float64, device=x.device)
    for e in sorted(set(order.flatten().tolist())):
        if s["s1"] is None:
            w1, w2 = s["w1"][e].double(), s["w2"][e].double()
        else:
            w1 = _expert64(s["w1"], s["s1"], e, up, h)
            w2 = _expert64(s["w2"], s["s2"], e, h, i)
        token, place = (order == e).nonzero(as_tuple=True)
        z = x[token] @ w1.t() + (0.0 if s["b1"] is None else s["b1"][e].double())
        z = _act64(z[:, :i], case["act"], 0.0) * z[:, i:] if case["gated"] else _act64(z, case["act"], 0.0)
        o = z @ w2.t() + (0.0 if s["b2"] is None else s["b2"][e].double())
        y.index_add_(0, token, share[token, place].unsqueeze(1) * o)
    return {"y": y, "experts": order.int(), "probs": share}


def _expert64(codes, scales, e, rows, k):
    """Expert e's rows of the packed [E * rows, k]: whole groups of 128 rows around them, then cut."""
    first, last = e * rows // 128 * 128, min(-(-(e + 1) * rows // 128) * 128, codes.shape[0])
    tiles = -(-k // 128)
    v = _values64(codes[first:last], scales[first // 128 * tiles * 512: -(-last // 128) * tiles * 512], last - first, k)
    return v[e * rows - first: (e + 1) * rows - first]
