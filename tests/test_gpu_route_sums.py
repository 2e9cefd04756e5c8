"""The router's balance loss to the precision of its sums: closely enough that one token left out of a column's sum
shows.

Bound.  A softmax probability is off by prob_error (relative), so a sum of them is too.  A column's sum is added up in fp32, each
addition off by 2^-24 of the sum so far at most: over the tokens of a group of lanes (a CTA of every SM has 8 such groups at
least), the groups of a CTA (96 at most), every 8th CTA (64 at most), and 8 partial sums; the loss adds at most 512 columns
in a tree (32 of them, then 16) and takes six more operations."""
import pytest
import torch

import route_reference as ref
from conv_activation_epilogue_gb300 import build, mmact

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    mmact.load()


def tolerance(T):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return ref.prob_error(None) + (-(-T // (sms * 8)) + 96 + 64 + 8 + 32 + 16 + 6) * 2.0 ** -24


def forward(z, top, mask=None, normalize=True):
    T, E = z.shape
    experts, probs = torch.empty((T, top), dtype=torch.int32, device="cuda"), torch.empty((T, top), device="cuda")
    counts, loss = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.full((1,), float("nan"), device="cuda")
    work = torch.full((mmact.mmact_moe_route_workspace_bytes(T, E),), 0xFF, dtype=torch.uint8, device="cuda")
    mmact.mmact_moe_route(z, experts, probs, counts, loss, work, coef=1.0, normalize=normalize, mask=mask)
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
    return counts, float(loss)


def reference(z, top, on):
    """(counts, a function of the tokens whose softmax counts that gives the loss) in 64 bits."""
    z64 = z.double()
    E, n = z.shape[1], int(on.sum())
    order = torch.sort(z64, dim=1, descending=True, stable=True)[1][:, :top]
    counts = torch.bincount(order[on].flatten(), minlength=E)
    p = torch.softmax(z64, dim=1)
    return counts, lambda keep: float(E * (counts.double() / (n * top) * p[keep].sum(dim=0) / n).sum())


# a round of all groups of lanes, and a few tokens more; every layout of a token over lanes
SIZES = [(E, top, T) for E, top in ((16, 2), (30, 1), (64, 4), (64, 8), (65, 3), (128, 8), (250, 8), (256, 9), (512, 16)) for T in (1, 33, 1217, 4865, 9731, 14593, 17011)]


@pytest.mark.parametrize("E,top,T", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_one_token_left_out_would_show(E, top, T, dtype):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    z = torch.randn((T, E), generator=g, device="cuda") + torch.linspace(0, 1, E, device="cuda")
    z[-1, E - 1] += 8.0                                       # the last token: nearly all of it on the expert chosen most
    z = z.to(dtype)
    on = torch.ones(T, dtype=torch.bool, device="cuda")
    counts, loss_of = reference(z, top, on)
    want, tol = loss_of(on), tolerance(T)
    got_counts, got = forward(z, top)
    assert torch.equal(got_counts[:E].long(), counts) and int(got_counts[E]) == T
    assert abs(got - want) <= tol * want
    assert 1 / T > 1.5 * tol                                  # a token's part, on average
    on[-1] = False
    assert abs(loss_of(on) - want) > 1.5 * tol * want


@pytest.mark.parametrize("T,E,top", [(131072, 64, 8), (131072, 256, 8), (70001, 129, 4), (200000, 512, 2), (300000, 16, 2)])
def test_many_tokens(T, E, top):
    g = torch.Generator(device="cuda").manual_seed(T)
    z = torch.randn((T, E), generator=g, device="cuda")
    mask = torch.rand(T, generator=g, device="cuda") < 0.9
    # late tokens that nearly all lie on one expert
    z[-40:, 3] += 20.0
    mask[-40:] = True
    counts, loss_of = reference(z, top, mask)
    got_counts, got = forward(z, top, mask)
    assert torch.equal(got_counts[:E].long(), counts) and int(got_counts[E]) == int(mask.sum())
    want, tol = loss_of(mask), tolerance(T)
    assert abs(got - want) <= tol * want
    fewer = mask.clone()
    fewer[-40:] = False
    assert abs(loss_of(fewer) - want) > 1.5 * tol * want


def test_uneven_shares():
    """Many tokens give an expert next to nothing that a few choose outright."""
    T, E = 100000, 32
    z = torch.zeros((T, E), device="cuda")
    z[:, 0] = 12.0
    z[::1000] = 0.0
    z[::1000, 7] = 30.0
    on = torch.ones(T, dtype=torch.bool, device="cuda")
    counts, loss_of = reference(z, 1, on)
    got_counts, got = forward(z, 1)
    assert torch.equal(got_counts[:E].long(), counts) and abs(got - loss_of(on)) <= tolerance(T) * loss_of(on)
