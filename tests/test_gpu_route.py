"""The router in training on the GPU against the plain 64-bit implementation: choices and
counts exactly, probabilities, loss and gradients within derived bounds."""
import numpy as np
import pytest
import torch

import mx_reference as mx
import route_reference as ref
from conv_activation_epilogue_gb300 import build, mmact
from parity import TORCH

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    mmact.load()


def host64(t):
    return t.detach().double().cpu().numpy()


def forward(z, top, coef=1.0, normalize=True, mask=None, stream=None):
    T, E = z.shape
    experts = torch.full((T, top), -7, dtype=torch.int32, device="cuda")
    probs = torch.full((T, top), float("nan"), device="cuda")
    counts = torch.full((E + 1,), -7, dtype=torch.int32, device="cuda")
    loss = torch.full((1,), float("nan"), device="cuda")
    work = torch.full((mmact.mmact_moe_route_workspace_bytes(T, E),), 0xFF, dtype=torch.uint8, device="cuda")
    mmact.mmact_moe_route(z, experts, probs, counts, loss, work, coef=coef, normalize=normalize, mask=mask, stream=stream)
    return experts, probs, counts, loss


def logits(rng, T, E, dtype, closed=0.0, ties=False):
    z = rng.normal(0, 1.5, (T, E)) + rng.normal(0, 0.7, E)
    if ties:
        z = np.round(z * 2) / 2
    z[rng.random((T, E)) < closed] = -np.inf
    t = torch.from_numpy(z.astype(np.float32)).to(TORCH[dtype]).cuda()
    return t, host64(t)


def check_forward(t, z, top, coef, normalize, mask=None):
    dev_mask = None if mask is None else torch.tensor(mask, dtype=torch.uint8, device="cuda")
    experts, probs, counts, loss = forward(t, top, coef, normalize, dev_mask)
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
    ids, p, n, want, _ = ref.route(z, top, coef, normalize, mask)
    assert np.array_equal(experts.cpu().numpy(), ids)
    assert np.array_equal(counts.cpu().numpy(), n)
    assert np.all(np.abs(host64(probs) - p) <= ref.prob_error(z) * p + ref.TINY)
    # a sum of positive terms over tokens, warps and CTAs: T roundings at most in each partial sum, not one after the other
    assert abs(float(loss) - want) <= (ref.prob_error(z) + (min(len(z), 2048) + z.shape[1]) * 2.0 ** -23) * want
    return experts, probs, counts, loss


SHAPES = [(1, 1, 1), (1, 4, 2), (7, 5, 5), (64, 64, 8), (33, 21, 2), (100, 32, 16), (129, 33, 4), (50, 65, 3), (300, 128, 8),
          (40, 129, 6), (65, 256, 8), (20, 257, 9), (31, 511, 16), (16, 512, 16), (70, 72, 1), (9, 160, 10)]


@pytest.mark.parametrize("T,E,top", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("normalize", [False, True])
def test_forward(T, E, top, dtype, normalize):
    rng = np.random.default_rng(T * 1000 + E)
    t, z = logits(rng, T, E, dtype)
    check_forward(t, z, top, 0.01, normalize)


@pytest.mark.parametrize("T,E,top", [(40, 8, 3), (130, 64, 8), (60, 200, 16), (33, 512, 5)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("normalize", [False, True])
def test_forward_with_ties_closed_experts_and_a_mask(T, E, top, dtype, normalize):
    rng = np.random.default_rng(E)
    t, z = logits(rng, T, E, dtype, closed=0.5, ties=True)
    z[3], z[5], z[6] = -np.inf, 0.25, -0.0                     # nothing left; all equal; both zeros
    z[6, ::2] = 0.0
    z[7, 1:] = -np.inf                                         # fewer than `top`
    t.copy_(torch.from_numpy(z))
    mask = (rng.random(T) < 0.8).astype(np.uint8)
    mask[[3, 5, 6, 7]] = 1
    check_forward(t, z, top, 0.5, normalize, mask)
    check_forward(t, z, top, 0.5, normalize, np.zeros(T, dtype=np.uint8))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_logits_of_the_types_lowest_value(dtype):
    """A mask that writes the lowest finite number: such experts are chosen last, and with nothing else a
    token is shared out evenly."""
    z = torch.randn((6, 40), device="cuda").to(TORCH[dtype])
    z[:, 5:] = torch.finfo(TORCH[dtype]).min
    z[2] = torch.finfo(TORCH[dtype]).min
    z[4, :5] = torch.finfo(TORCH[dtype]).max
    check_forward(z, host64(z), 8, 1.0, True)
    check_forward(z, host64(z), 8, 1.0, False)


def test_nan_and_infinite_logits_stay_in_their_token():
    rng = np.random.default_rng(1)
    t, z = logits(rng, 40, 70, "f32")
    clean = forward(t, 4)
    t[3, 60], t[9, 5], t[9, 6] = float("nan"), float("inf"), float("inf")
    t[11, 2] = -float("nan")
    experts, probs, counts, loss = forward(t, 4)
    ids = ref.route(host64(t), 4, 1.0, True)[0]
    assert np.array_equal(experts.cpu().numpy(), ids) and ids[3, 0] == 60 and ids[9, :2].tolist() == [5, 6] and ids[11, 0] == 2
    bad = torch.isnan(probs).any(dim=1)
    assert bad.nonzero().flatten().tolist() == [3, 9, 11] and torch.isnan(loss).all()
    keep = ~bad
    assert torch.equal(experts[keep], clean[0][keep]) and torch.equal(probs[keep], clean[1][keep])
    dz = torch.empty_like(t)
    mmact.mmact_moe_route_backward(t, experts, counts, torch.ones_like(probs), loss.fill_(1.0), dz)
    assert torch.equal(torch.isnan(dz).any(dim=1), bad)


def test_choice_is_that_of_the_mixture_layer():
    """The same logits give mmact_moe's experts and probabilities: x picks rows of the router."""
    T, H, I, E, top = 16, 64, 32, 24, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.eye(T, H, device="cuda").bfloat16()
    router = torch.randn((E, H), generator=g, device="cuda").bfloat16()
    w1, w2 = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((E, 2 * I, H), (E, H, I)))
    y = torch.empty_like(x)
    ids, p = torch.empty((T, top), dtype=torch.int32, device="cuda"), torch.empty((T, top), device="cuda")
    work = torch.empty(mmact.mmact_moe_workspace_bytes(T, H, I, E, top), dtype=torch.uint8, device="cuda")
    for normalize in (False, True):
        mmact.mmact_moe(x, router, w1, w2, y, ids, p, work, normalize=normalize)
        experts, probs, _, _ = forward(router[:, :T].t().contiguous(), top, 1.0, normalize)
        assert torch.equal(experts, ids)
        assert float((probs - p).abs().max()) <= 2 * ref.prob_error(None)


@pytest.mark.parametrize("T,E,top", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("normalize", [False, True])
def test_backward(T, E, top, dtype, normalize):
    rng = np.random.default_rng(T * 77 + E)
    t, z = logits(rng, T, E, dtype, closed=0.2 if T % 2 else 0.0)
    mask = (rng.random(T) < 0.8).astype(np.uint8) if T > 30 else None
    dev_mask = None if mask is None else torch.tensor(mask, device="cuda").bool()
    experts, probs, counts, _ = forward(t, top, 0.7, normalize, dev_mask)
    dp = torch.from_numpy(rng.normal(0, 0.1, (T, top)).astype(np.float32)).cuda()
    dl = torch.tensor([1.5], device="cuda")
    for gp, gl in ((dp, dl), (dp, None), (None, dl), (None, None)):
        dz = torch.full_like(t, float("nan"))
        mmact.mmact_moe_route_backward(t, experts, counts, gp, gl, dz, coef=0.7, normalize=normalize, mask=dev_mask)
        want, bound = ref.backward(z, experts.cpu().numpy(), counts.cpu().numpy(),
                                   np.zeros((T, top)) if gp is None else host64(gp), 0.0 if gl is None else 1.5, top, 0.7,
                                   normalize, mask)
        got = host64(dz)
        half = np.maximum(mx.ulp(np.abs(want) + bound, dtype) / 2, {"f32": 0.0, "bf16": 0.0, "f16": 2.0 ** -25}[dtype])
        assert np.all(np.abs(got - want) <= bound + half)
        assert not got[(z == -np.inf)].any()
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK


def test_backward_of_slots_named_twice_or_outside():
    """Lists that no forward pass gives: equal entries add up, others than 0..E-1 count as none."""
    rng = np.random.default_rng(8)
    t, z = logits(rng, 5, 40, "f32")
    ids = np.array([[3, 3, 3, 7], [39, 0, 39, 0], [-1, 40, 1000, 5], [2, -1, 2, -5], [1, 2, 3, 4]])
    counts = torch.ones(41, dtype=torch.int32, device="cuda")
    dp = torch.from_numpy(rng.normal(0, 1, (5, 4)).astype(np.float32)).cuda()
    dz = torch.empty_like(t)
    mmact.mmact_moe_route_backward(t, torch.tensor(ids, dtype=torch.int32, device="cuda"), counts, dp, None, dz,
                                   normalize=False)
    want, bound = ref.backward(z, np.where((ids < 0) | (ids >= 40), -1, ids), np.ones(41), host64(dp), 0.0, 4, 1.0, False)
    err, lim = np.abs(host64(dz) - want), bound + mx.ulp(np.abs(want) + bound, "f32") / 2
    assert np.all(err <= lim), (np.argwhere(err > lim)[:5], err[err > lim][:5], lim[err > lim][:5])


@pytest.mark.parametrize("T,E,top,dtype", [(131072, 64, 8, "bf16"), (70001, 129, 4, "f32"), (200000, 512, 2, "f16")])
def test_many_tokens(T, E, top, dtype):
    """Against torch in fp64: several tokens for each warp, every SM."""
    g = torch.Generator(device="cuda").manual_seed(T)
    z = torch.randn((T, E), generator=g, device="cuda").to(TORCH[dtype])
    mask = torch.rand(T, generator=g, device="cuda") < 0.9
    experts, probs, counts, loss = forward(z, top, 0.01, True, mask)
    z64 = z.double()
    order = torch.sort(z64, dim=1, descending=True, stable=True)[1][:, :top]
    order[~mask] = -1
    assert torch.equal(experts.long(), order)
    n = int(mask.sum())
    want = torch.bincount(order[mask].flatten(), minlength=E)
    assert torch.equal(counts[:E].long(), want) and int(counts[E]) == n
    p = torch.softmax(z64, dim=1)
    q = p.gather(1, order.clamp(min=0)) * mask[:, None]
    q = q / q.sum(dim=1, keepdim=True).clamp(min=1e-30)
    assert bool(((probs - q).abs() <= ref.prob_error(None) * q).all())
    ref_loss = float(0.01 * E * (want / (n * top) * p[mask].sum(dim=0) / n).sum())
    assert abs(float(loss) - ref_loss) <= (ref.prob_error(None) + 4096 * 2.0 ** -23) * ref_loss
    again = forward(z, top, 0.01, True, mask)
    for a, b in zip((experts, probs, counts, loss), again):
        assert torch.equal(a, b)                               # bit for bit
    dz = torch.empty_like(z)
    dp = torch.randn((T, top), generator=g, device="cuda")
    mmact.mmact_moe_route_backward(z, experts, counts, dp, torch.ones(1, device="cuda"), dz, coef=0.01, mask=mask)
    up = 0.01 * E / (n * n * top) * want
    dwant = p * (up - (p * up).sum(dim=1, keepdim=True)) * mask[:, None]
    dwant.scatter_add_(1, order.clamp(min=0), q * (dp - (q * dp).sum(dim=1, keepdim=True)))
    half = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}[dtype]
    bound = torch.zeros_like(dwant).scatter_add_(1, order.clamp(min=0), 8 * ref.prob_error(None) * q * (dp.abs() + 4.0))
    assert bool(((dz.double() - dwant).abs() <= bound + half * dwant.abs() + 8 * ref.prob_error(None) * float(up.max()) * p
                 + (2.0 ** -25 if dtype == "f16" else 0.0)).all())


@pytest.mark.parametrize("T,E,top,dtype", [(5000, 64, 8, "bf16"), (3001, 257, 3, "f32"), (4000, 30, 2, "f16")])
def test_backward_in_place(T, E, top, dtype):
    t, _ = logits(np.random.default_rng(T), T, E, dtype)
    experts, probs, counts, loss = forward(t, top)
    dp, dz = torch.randn((T, top), device="cuda"), torch.empty_like(t)
    mmact.mmact_moe_route_backward(t, experts, counts, dp, loss, dz)
    mmact.mmact_moe_route_backward(t, experts, counts, dp, loss, t)
    assert torch.equal(t, dz)


def test_tokens_past_32_bit_offsets():
    """More than 2^31 logits: copies of a few tokens, so that every copy's choice and gradient are known."""
    E, top, base = 512, 4, 1000
    z = torch.randn((base, E), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").bfloat16()
    experts, probs, counts, loss = forward(z, top)
    copies = 4300
    many = z.repeat(copies, 1)
    e, p, c, l = forward(many, top)
    assert torch.equal(c.long(), counts.long() * copies) and torch.equal(e.view(copies, base, top), experts.expand(copies, base, top))
    assert torch.equal(p.view(copies, base, top), probs.expand(copies, base, top))
    # the same shares: the same loss, from sums over tokens in another order
    assert abs(float(l) - float(loss)) <= 2 * (ref.prob_error(None) + 8192 * 2.0 ** -23) * float(loss)
    dp = torch.randn((base, top), device="cuda")
    dz, dmany = torch.empty_like(z), torch.full_like(many, float("nan"))
    mmact.mmact_moe_route_backward(z, experts, counts, dp, None, dz)
    mmact.mmact_moe_route_backward(many, e, c, dp.repeat(copies, 1), None, dmany)
    assert torch.equal(dmany.view(copies, base, E)[[0, 1, 2100, 4200, 4299]], dz.expand(5, base, E))
    assert bool((dmany.view(copies, base, E) == dz).all())


def test_no_tokens():
    experts, probs, counts, loss = forward(torch.empty((0, 30), device="cuda"), 3)
    assert not counts.any() and float(loss) == 0.0
    mmact.mmact_moe_route_backward(torch.empty((0, 30), device="cuda"), experts, counts, probs, loss,
                                   torch.empty((0, 30), device="cuda"))
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK


def test_side_stream_and_graph():
    rng = np.random.default_rng(4)
    T, E, top = 500, 48, 4
    t, z = logits(rng, T, E, "bf16")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = forward(t, top)
    s.synchronize()
    for a, b in zip(out, forward(t, top)):
        assert torch.equal(a, b)
    experts, probs, counts, loss = out
    work = torch.empty(mmact.mmact_moe_route_workspace_bytes(T, E), dtype=torch.uint8, device="cuda")
    dz, dp, dl = torch.empty_like(t), torch.randn((T, top), device="cuda"), torch.ones(1, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mmact.mmact_moe_route(t, experts, probs, counts, loss, work)
        mmact.mmact_moe_route_backward(t, experts, counts, dp, dl, dz)
    t.copy_(logits(rng, T, E, "bf16")[0])
    work.fill_(0xEE)
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip((experts, probs, counts, loss), forward(t, top)):
        assert torch.equal(a, b)
    again = torch.empty_like(dz)
    mmact.mmact_moe_route_backward(t, experts, counts, dp, dl, again)
    assert torch.equal(dz, again)


def test_refusals():
    z = torch.zeros((4, 8), device="cuda")
    ids, p = torch.zeros((4, 2), dtype=torch.int32, device="cuda"), torch.zeros((4, 2), device="cuda")
    counts, loss = torch.zeros(9, dtype=torch.int32, device="cuda"), torch.zeros(1, device="cuda")
    work = torch.zeros(mmact.mmact_moe_route_workspace_bytes(4, 8), dtype=torch.uint8, device="cuda")
    mmact.mmact_moe_route(z, ids, p, counts, loss, work)
    for bad in (dict(logits=z.t()), dict(experts=ids[:3]), dict(probs=p[:, :1].contiguous()), dict(counts=counts[:8]),
                dict(loss=torch.zeros(2, device="cuda")), dict(workspace=work[:16]),
                dict(mask=torch.zeros(3, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            mmact.mmact_moe_route(**{**dict(logits=z, experts=ids, probs=p, counts=counts, loss=loss, workspace=work), **bad})
    for bad in (dict(logits=z.double()), dict(experts=ids.long()), dict(probs=p.half()), dict(mask=torch.zeros(4, device="cuda"))):
        with pytest.raises(TypeError):
            mmact.mmact_moe_route(**{**dict(logits=z, experts=ids, probs=p, counts=counts, loss=loss, workspace=work), **bad})
    with pytest.raises(ValueError):
        mmact.mmact_moe_route_backward(z, ids, counts, p[:3], loss, z.clone())
    with pytest.raises(TypeError):
        mmact.mmact_moe_route_backward(z, ids, counts, p, loss, z.half())
    nine = torch.zeros((4, 9), dtype=torch.int32, device="cuda")
    with pytest.raises(mmact.MmactError) as ei:                # more slots than experts
        mmact.mmact_moe_route(z, nine, nine.float(), counts, loss, work)
    assert ei.value.status == mmact.MMACT_ERR_UNSUPPORTED
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK


@pytest.mark.parametrize("T,E,top", [(70, 64, 8), (33, 256, 8), (20, 512, 16), (50, 30, 3)])
def test_equal_logits_everywhere(T, E, top):
    """A router whose weights are zeros: the first experts are chosen, by every token."""
    z = torch.zeros((T, E), device="cuda").bfloat16()
    z[1::2] = -0.0
    z[5] = 1.0
    z[7, E // 2:] = 1.0                                        # half of them
    check_forward(z, host64(z), top, 1.0, True)
    check_forward(z, host64(z), top, 1.0, False)


@pytest.mark.parametrize("normalize", [False, True])
def test_what_stands_in_left_out_tokens_and_empty_slots_is_not_looked_at(normalize):
    """Padded tokens hold anything, upstream gradients of slots that chose nobody too."""
    rng = np.random.default_rng(6)
    T, E, top = 60, 24, 4
    t, z = logits(rng, T, E, "f32")
    z[5, 2:] = -np.inf                                         # two slots of four
    z[9] = -np.inf
    t.copy_(torch.from_numpy(z))
    mask = np.ones(T, dtype=np.uint8)
    mask[[3, 20, 59]] = 0
    dev_mask = torch.tensor(mask, device="cuda")
    clean = forward(t, top, 0.3, normalize, dev_mask)
    dp = torch.randn((T, top), device="cuda")
    dl, dz, again = torch.ones(1, device="cuda"), torch.empty_like(t), torch.empty_like(t)
    mmact.mmact_moe_route_backward(t, clean[0], clean[2], dp, dl, dz, coef=0.3, normalize=normalize, mask=dev_mask)
    t[3], t[20, 7], t[59, 0] = float("nan"), float("inf"), -float("inf")
    dp[[3, 9, 20, 59]] = float("nan")
    dp[5, 2:] = float("inf")
    for a, b in zip(forward(t, top, 0.3, normalize, dev_mask), clean):
        assert torch.equal(a, b)
    listed = clean[0].clone()
    listed[3] = torch.arange(top)                              # a left-out token's list of its own
    mmact.mmact_moe_route_backward(t, listed, clean[2], dp, dl, again, coef=0.3, normalize=normalize, mask=dev_mask)
    assert torch.equal(dz, again) and not again[[3, 9, 20, 59]].any()
    want, bound = ref.backward(z, clean[0].cpu().numpy(), clean[2].cpu().numpy(), np.nan_to_num(host64(dp), posinf=0.0), 1.0, top,
                               0.3, normalize, mask)
    assert np.all(np.abs(host64(dz) - want) <= bound + mx.ulp(np.abs(want) + bound, "f32") / 2)
