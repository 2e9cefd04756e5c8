"""The mixture-of-experts layer on the GPU against the plain 64-bit implementation.
x and the router hold small multiples of a power of two, so that the logits are exact
in fp32 and the choice of experts, ties included, has one right answer."""
import numpy as np
import pytest
import torch

import mx_reference as ref
from conv_activation_epilogue_gb300 import build, mmact
from parity import TORCH
from test_gpu_mxfp4 import host64, tensor

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    mmact.load()


def layer(seed, T, H, I, E, dtype, weights, gated=True, bias=False, w_std=None):
    rng = np.random.default_rng(seed)
    up = 2 * I if gated else I
    L = {"x": rng.integers(-16, 17, (T, H)) / 8.0, "router": rng.integers(-4, 5, (E, H)) / 64.0}
    for name, rows, k in (("w1", up, H), ("w2", H, I)):
        w = rng.normal(0, (w_std or k ** -0.5), (E * rows, k))
        if weights == "mxfp4":
            c, s, v = ref.quantize(w)
            L[name + "_codes"], L[name + "_scales"], L[name] = c, s, v.reshape(E, rows, k)
        else:
            L[name] = host64(tensor(w, dtype)).reshape(E, rows, k)
    for name, shape in (("rb", (E,)), ("b1", (E, up)), ("b2", (E, H))):
        L[name] = (rng.integers(-64, 65, shape) / 64.0) if bias else None
    return L


def run(L, top, dtype, weights, act="silu", alpha=0.0, gated=True, normalize=True, stream=None):
    T, H = L["x"].shape
    E, I = L["router"].shape[0], L["w2"].shape[2]
    dev = {}
    for k in ("x", "router"):
        dev[k] = tensor(L[k], dtype)
    if weights == "mxfp4":
        for k in ("w1", "w2"):
            dev[k] = torch.from_numpy(L[k + "_codes"]).cuda()
            dev[k + "_scales"] = torch.from_numpy(L[k + "_scales"]).cuda()
    else:
        for k in ("w1", "w2"):
            dev[k], dev[k + "_scales"] = tensor(L[k], dtype), None
    opt = {k: None if L[k] is None else tensor(L[k], "f32") for k in ("rb", "b1", "b2")}
    y = torch.full((T, H), float("nan"), dtype=TORCH[dtype], device="cuda")
    experts = torch.full((T, top), -1, dtype=torch.int32, device="cuda")
    probs = torch.full((T, top), float("nan"), dtype=torch.float32, device="cuda")
    work = torch.full((mmact.mmact_moe_workspace_bytes(T, H, I, E, top),), 0xFF, dtype=torch.uint8, device="cuda")
    call = lambda: mmact.mmact_moe(dev["x"], dev["router"], dev["w1"], dev["w2"], y, experts, probs, work, act, alpha,  # noqa: E731
                                   gated=gated, normalize=normalize, router_bias=opt["rb"], b1=opt["b1"], b2=opt["b2"],
                                   w1_scales=dev["w1_scales"], w2_scales=dev["w2_scales"], stream=stream)
    call()
    return y, experts, probs, call, dev


def check(L, out, top, dtype, act="silu", alpha=0.0, gated=True, normalize=True):
    y, experts, probs = out[:3]
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
    want, ids, p, bound, dp = ref.moe(L["x"], L["router"], L["w1"], L["w2"], top, act, alpha, gated, normalize, L["rb"],
                                      L["b1"], L["b2"])
    assert np.array_equal(experts.cpu().numpy(), ids)
    assert np.all(np.abs(host64(probs) - p) <= dp[:, None] * p)
    got = host64(y)
    lim = bound + ref.ulp(np.abs(want) + bound, dtype)
    assert np.all(np.isfinite(got))
    err = np.abs(got - want)
    assert np.all(err <= lim), (np.argmax(err / lim), float((err / lim).max()))


TYPES = [("bf16", "bf16"), ("f16", "f16"), ("bf16", "mxfp4"), ("f16", "mxfp4")]


@pytest.mark.parametrize("dtype,weights", TYPES)
@pytest.mark.parametrize("T,H,I,E,top", [(1, 8, 8, 1, 1), (1, 256, 64, 8, 2), (2, 40, 24, 5, 5), (3, 520, 136, 16, 3),
                                         (13, 264, 200, 21, 2), (17, 128, 96, 4, 1), (33, 96, 160, 7, 4),
                                         (64, 72, 40, 3, 2), (64, 136, 64, 40, 16), (5, 1032, 16, 512, 8), (1, 4096, 520, 6, 2),
                                         (9, 2304, 1048, 4, 2), (40, 520, 2600, 3, 1), (2, 48, 16, 3, 1),
                                         (5, 64, 32, 4, 2), (2, 96, 64, 60, 1), (30, 200, 64, 90, 8)])
def test_layer(dtype, weights, T, H, I, E, top):
    gated, bias = (T + E) % 3 != 0, T % 2 == 1
    L = layer(T * 131 + H + I + E, T, H, I, E, dtype, weights, gated, bias)
    out = run(L, top, dtype, weights, "silu" if gated else "gelu", gated=gated, normalize=T != 3)
    check(L, out, top, dtype, "silu" if gated else "gelu", gated=gated, normalize=T != 3)


@pytest.mark.parametrize("act", ["none", "relu", "leaky_relu", "tanh", "sigmoid", "gelu", "silu"])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("normalize", [True, False])
def test_activations_and_forms(act, gated, normalize):
    L = layer(3, 6, 160, 72, 9, "bf16", "bf16", gated, True)
    out = run(L, 3, "bf16", "bf16", act, 0.2, gated, normalize)
    check(L, out, 3, "bf16", act, 0.2, gated, normalize)


@pytest.mark.parametrize("dtype,weights", TYPES)
def test_all_tokens_choose_one_expert(dtype, weights):
    L = layer(4, 64, 128, 48, 6, dtype, weights, True, False)
    L["rb"] = np.array([0, 0, 0, 200.0, 0, 0])
    out = run(L, 1, dtype, weights)
    assert torch.all(out[1] == 3)
    check(L, out, 1, dtype)


def test_equal_logits_choose_the_lowest_indices():
    L = layer(5, 4, 64, 16, 10, "bf16", "bf16")
    L["x"][2] = 0.0                                     # every logit 0
    L["router"][7] = L["router"][1]                     # equal for every token
    out = run(L, 4, "bf16", "bf16")
    assert out[1][2].tolist() == [0, 1, 2, 3]
    check(L, out, 4, "bf16")
    # -0 and +0 are equal logits
    L["router"][:] = 0.0
    L["rb"] = np.array([-0.0, 0.0] * 5)
    out = run(L, 3, "bf16", "bf16")
    assert out[1].tolist() == [[0, 1, 2]] * 4


@pytest.mark.parametrize("dtype,weights", TYPES)
def test_nan_stays_in_its_token_or_expert(dtype, weights):
    L = layer(6, 5, 64, 32, 6, dtype, weights)
    clean = run(L, 2, dtype, weights)
    L["x"][3, 10] = np.nan
    y, experts, probs, _, _ = run(L, 2, dtype, weights)
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
    assert torch.isnan(y[3]).all() and torch.isnan(probs[3]).all()
    assert int(experts.min()) >= 0 and int(experts.max()) < 6
    keep = [0, 1, 2, 4]
    assert torch.equal(y[keep], clean[0][keep]) and torch.equal(experts[keep], clean[1][keep])


def test_an_infinite_router_bias_masks_or_forces_experts():
    L = layer(7, 4, 64, 16, 6, "bf16", "bf16", bias=True)
    L["rb"][1] = L["rb"][4] = -np.inf                   # never chosen while others are left
    out = run(L, 4, "bf16", "bf16")
    assert not np.isin(out[1].cpu().numpy(), [1, 4]).any()
    check(L, out, 4, "bf16")
    out = run(L, 6, "bf16", "bf16")                     # chosen last, with weight 0
    assert out[1][:, 4:].tolist() == [[1, 4]] * 4 and torch.all(out[2][:, 4:] == 0)


@pytest.mark.parametrize("weights", ["bf16", "mxfp4"])
def test_nan_expert_weights_reach_their_tokens_only(weights):
    L = layer(8, 12, 64, 32, 6, "bf16", weights)
    y, experts, _, call, dev = run(L, 2, "bf16", weights)
    clean = y.clone()
    e = int(experts[0, 0])
    hit = (experts == e).any(dim=1)
    if weights == "bf16":
        dev["w2"][e, 3, 5] = float("nan")
    else:
        dev["w2_scales"][ref.scale_place(e * 64 + 3, 0, 1)] = 255
    call()
    assert torch.isnan(y[hit, 3]).all()
    keep = torch.ones(64, dtype=torch.bool, device="cuda")
    keep[3] = False
    assert torch.equal(y[:, keep], clean[:, keep]) and torch.equal(y[~hit], clean[~hit])


def test_large_intermediates_keep_fp32_range():
    """h past fp16's largest value: 300 * 300 = 90000, halved again by the down product."""
    L = layer(9, 2, 64, 32, 4, "f16", "f16", True)
    L["x"][:] = 1.0
    L["w1"][:] = 300.0 / 64.0
    L["w2"][:] = 1.0 / 1024.0
    out = run(L, 2, "f16", "f16", "relu")
    check(L, out, 2, "f16", "relu")
    assert float(out[0].float().min()) > 2800


def test_scales_above_two_and_subnormal_scales():
    L = layer(10, 3, 64, 32, 4, "bf16", "mxfp4")
    for scale in (2.0 ** 40, 2.0 ** -60):
        for name, rows, k in (("w1", 64, 64), ("w2", 64, 32)):
            v = L[name].reshape(4 * rows, k) * (scale if name == "w1" else 1.0)
            L[name + "_codes"], L[name + "_scales"], q = ref.quantize(v)
            L[name] = q.reshape(4, rows, k)
        out = run(L, 2, "bf16", "mxfp4", "relu")
        check(L, out, 2, "bf16", "relu")


def test_results_repeat_and_graphs_replay():
    L = layer(11, 24, 256, 128, 12, "bf16", "bf16")
    y, experts, probs, call, dev = run(L, 4, "bf16", "bf16")
    first = y.clone()
    for _ in range(5):
        call()
        assert torch.equal(y, first)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    y.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = run(L, 4, "bf16", "bf16", stream=s)
    s.synchronize()
    check(L, out, 4, "bf16")


@pytest.mark.parametrize("dtype,weights", TYPES)
@pytest.mark.parametrize("T,H,I,gated", [(64, 64, 16, True), (64, 72, 200, False), (49, 40, 72, True), (16, 64, 16, False)])
def test_the_most_experts_and_choices(dtype, weights, T, H, I, gated):
    L = layer(T + I, T, H, I, 512, dtype, weights, gated, True)
    out = run(L, 16, dtype, weights, gated=gated)
    check(L, out, 16, dtype, gated=gated)


@pytest.mark.parametrize("dtype,weights", TYPES)
@pytest.mark.parametrize("T,H,I,E,top,gated", [(32, 4096, 1792, 16, 4, True), (64, 2048, 2056, 12, 3, False),
                                               (1, 2048, 1024, 64, 8, True)])
def test_large_layers_under_load(dtype, weights, T, H, I, E, top, gated):
    """Rings that turn over hundreds of times, calls back to back; the plain form in fp64 on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(T + H)
    x = torch.randint(-16, 17, (T, H), generator=g, device="cuda").double() / 8
    router = torch.randint(-4, 5, (E, H), generator=g, device="cuda").double() / 64
    up = 2 * I if gated else I
    t = TORCH[dtype]
    w, dev, scales = {}, {}, {}
    for name, rows, k in (("w1", up, H), ("w2", H, I)):
        v = torch.randn((E * rows, k), generator=g, device="cuda") * k ** -0.5
        if weights == "mxfp4":
            nc, ns = mmact.mmact_mxfp4_size(E * rows, k)
            dev[name] = torch.empty((E * rows, nc // (E * rows)), dtype=torch.uint8, device="cuda")
            scales[name] = torch.empty(ns, dtype=torch.uint8, device="cuda")
            mmact.mmact_quantize_mxfp4(v, dev[name], scales[name])
            mmact.mmact_dequantize_mxfp4(dev[name], scales[name], v)
        else:
            v = v.to(t)
            dev[name], scales[name] = v.view(E, rows, k), None
        w[name] = v.view(E, rows, k)
    y = torch.empty((T, H), dtype=t, device="cuda")
    experts = torch.empty((T, top), dtype=torch.int32, device="cuda")
    probs = torch.empty((T, top), dtype=torch.float32, device="cuda")
    work = torch.full((mmact.mmact_moe_workspace_bytes(T, H, I, E, top),), 0xFF, dtype=torch.uint8, device="cuda")
    xd, rd = x.to(t), router.to(t)
    results = []
    for _ in range(12):
        mmact.mmact_moe(xd, rd, dev["w1"], dev["w2"], y, experts, probs, work, "silu", gated=gated,
                        w1_scales=scales["w1"], w2_scales=scales["w2"])
        results.append(y.clone())
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
    assert all(torch.equal(r, results[0]) for r in results)

    logits = x @ router.T
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :top]
    assert torch.equal(experts.long(), ids)
    ex = torch.exp(logits - logits.max(dim=1, keepdim=True).values)
    chosen = torch.gather(ex, 1, ids)
    p = chosen / chosen.sum(dim=1, keepdim=True)
    dl = ref.sum_error(H + 1) * (x.abs() @ router.abs().T).max(dim=1).values
    dp = 2 * dl + (E + 8) * 2.0 ** -23
    assert bool(((probs.double() - p).abs() <= dp[:, None] * p).all())
    want, bound = torch.zeros_like(x), torch.zeros_like(x)
    for e in range(E):                                   # the bounds of mx_reference.moe
        at, j = torch.nonzero(ids == e, as_tuple=True)
        if at.numel() == 0:
            continue
        w1, w2 = w["w1"][e].double(), w["w2"][e].double()
        z = x[at] @ w1.T
        dz = ref.sum_error(H + 1) * (x[at].abs() @ w1.abs().T)
        a = torch.nn.functional.silu(z[:, :I])
        da = ref.SLOPE * dz[:, :I] + torch.from_numpy(np.asarray(ref.act_error(z[:, :I].cpu().numpy(), "silu"))).cuda()
        if gated:
            h, dh = a * z[:, I:], da * z[:, I:].abs() + (a.abs() + da) * dz[:, I:]
        else:
            h, dh = a, da
        dh = dh + (2.0 ** -23 + 2.0 ** -16) * h.abs()
        o, mag = h @ w2.T, h.abs() @ w2.abs().T
        do = dh @ w2.abs().T + (ref.sum_error(3 * (I + 1)) + 2.0 ** -16) * mag
        want[at] += p[at, j, None] * o
        bound[at] += p[at, j, None] * (do + (dp[at, None] + (top + 2) * 2.0 ** -23) * (o.abs() + do))
    want, bound = want.cpu().numpy(), bound.cpu().numpy()
    err = np.abs(host64(y) - want)
    lim = bound + ref.ulp(np.abs(want) + bound, dtype)
    assert np.all(err <= lim), float((err / lim).max())


def test_no_tokens_and_refusals():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    work = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    ids = lambda T, k: torch.zeros((T, k), dtype=torch.int32, device="cuda")  # noqa: E731
    pr = lambda T, k: torch.zeros((T, k), dtype=torch.float32, device="cuda")  # noqa: E731

    def call(T=2, H=16, I=8, E=4, k=2, x=None, w1=None, w2=None, router=None, ws=work, **kw):
        x = bf(T, H) if x is None else x
        mmact.mmact_moe(x, bf(E, H) if router is None else router, bf(E, 2 * I, H) if w1 is None else w1,
                        bf(E, H, I) if w2 is None else w2, torch.empty_like(x), ids(T, k), pr(T, k), ws, **kw)

    call()
    call(T=0)
    for kw in (dict(T=65), dict(H=12, I=8), dict(I=12), dict(k=5), dict(k=0), dict(E=520), dict(E=20, k=17)):
        with pytest.raises(mmact.MmactError) as ei:
            call(**kw)
        assert ei.value.status == mmact.MMACT_ERR_UNSUPPORTED, kw
    with pytest.raises(ValueError):
        call(ws=work[:64])
    with pytest.raises(ValueError):
        call(w1=bf(4, 8, 16))                            # gated needs 2 I rows
    with pytest.raises(TypeError):
        call(w1=bf(4, 16, 16).half())
    with pytest.raises(ValueError):
        call(router=bf(4, 16).half())
    with pytest.raises(ValueError):
        call(b1=pr(4, 8))
    with pytest.raises(KeyError):
        call(act="swish")
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
