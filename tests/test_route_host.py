"""The router's entry points on the host: sizes and refusals (no GPU: every call returns
before any CUDA work), and pins of the plain 64-bit implementation."""
import ctypes

import numpy as np
import pytest
import torch

import route_reference as ref
from conv_activation_epilogue_gb300 import build, mmact

E, U, OK = mmact.MMACT_ERR_INVALID_ARG, mmact.MMACT_ERR_UNSUPPORTED, mmact.MMACT_OK
P = 0x7f0000000000          # never dereferenced
MIS = P + 8


@pytest.fixture(scope="module")
def lib():
    build.build()
    return mmact.load()


def route(lib, z=P, mask=None, ids=P, probs=P, counts=P, loss=P, T=4, n=8, top=2, zd=1, work=P):
    return lib.mmact_moe_route(z, mask, ids, probs, counts, loss, T, n, top, zd, 1, ctypes.c_float(1), work, None)


def grad(lib, z=P, mask=None, ids=P, counts=P, dp=P, dl=P, dz=P, T=4, n=8, top=2, zd=1):
    return lib.mmact_moe_route_backward(z, mask, ids, counts, dp, dl, dz, T, n, top, zd, 1, ctypes.c_float(1), None)


def test_host_validation(lib):
    for name in ("z", "ids", "probs", "counts", "loss", "work"):
        assert route(lib, **{name: None}) == E
    for name in ("z", "work"):
        assert route(lib, **{name: MIS}) == U
    for name in ("ids", "probs", "counts", "loss"):
        assert route(lib, **{name: P + 2}) == E
    for name in ("z", "ids", "counts", "dz"):
        assert grad(lib, **{name: None}) == E
    for name in ("z", "dz"):
        assert grad(lib, **{name: MIS}) == U
    for name in ("ids", "counts", "dp", "dl"):
        assert grad(lib, **{name: P + 2}) == E
    for f in (route, grad):
        for bad in (3, 4, 5, -1):
            assert f(lib, zd=bad) == E
        assert f(lib, T=-1) == E and f(lib, n=-1) == E and f(lib, top=-1) == E and f(lib, T=1 << 31) == E
        assert f(lib, n=0) == U and f(lib, n=513) == U and f(lib, top=0) == U and f(lib, top=9) == U
        assert f(lib, n=500, top=17) == U
        assert f(lib, T=(1 << 31) - 1, top=2) == U
    assert grad(lib, T=0) == OK


def test_workspace_sizes(lib):
    out = ctypes.c_int64(-3)
    assert lib.mmact_moe_route_workspace_bytes(4, 8, None) == E
    assert lib.mmact_moe_route_workspace_bytes(-1, 8, ctypes.byref(out)) == E
    assert lib.mmact_moe_route_workspace_bytes(4, 513, ctypes.byref(out)) == U
    assert out.value == -3
    assert mmact.mmact_moe_route_workspace_bytes(0, 8) >= 0
    last = 0
    for T in (1, 100, 10000, 1 << 20, 1 << 27):
        now = mmact.mmact_moe_route_workspace_bytes(T, 512)
        assert now >= last and now < 16 << 20
        last = now


def test_cpu_tensors_are_refused(lib):
    z, ids, p = torch.zeros((4, 8)), torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2))
    counts, loss, work = torch.zeros(9, dtype=torch.int32), torch.zeros(1), torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(TypeError):
        mmact.mmact_moe_route(z, ids, p, counts, loss, work)
    with pytest.raises(TypeError):
        mmact.mmact_moe_route_backward(z, ids, counts, p, loss, z)


def test_reference_pins():
    inf = np.inf
    z = np.array([[0.0, 1.0, 1.0, -inf], [-inf, -inf, -inf, -inf], [2.0, np.nan, 5.0, 1.0], [-inf, 3.0, -inf, -inf],
                  [0.0, 0.0, 0.0, 0.0]])
    ids, p, counts, _, full = ref.route(z, 2, 1.0, True)
    assert ids.tolist() == [[1, 2], [-1, -1], [1, 2], [1, -1], [0, 1]]
    assert counts.tolist() == [1, 4, 2, 0, 4]
    assert p[0].tolist() == [0.5, 0.5] and p[1].tolist() == [0, 0] and np.isnan(p[2]).all() and p[3].tolist() == [1, 0]
    # even shares: the loss is coef
    z = np.zeros((4, 4))
    z[np.arange(4), np.arange(4)] = 1.0
    assert abs(ref.route(z, 1, 0.25, True)[3] - 0.25) < 1e-15
    # everything to one expert: E times as much
    z = np.zeros((6, 4))
    z[:, 2] = 50.0
    assert abs(ref.route(z, 1, 1.0, True)[3] - 4.0) < 1e-12


@pytest.mark.parametrize("normalize", [False, True])
def test_reference_backward_against_differences(normalize):
    rng = np.random.default_rng(0)
    T, n, top = 5, 7, 3
    z = rng.normal(0, 1, (T, n))
    z[1, 2] = -np.inf
    mask = [1, 1, 0, 1, 1]
    ids, p, counts, loss, _ = ref.route(z, top, 0.3, normalize, mask)
    dp, dl = rng.normal(0, 1, (T, top)), 1.7
    dz, _ = ref.backward(z, ids, counts, dp, dl, top, 0.3, normalize, mask)
    assert not dz[2].any() and dz[1, 2] == 0.0
    for t in range(T):
        for e in range(n):
            if z[t, e] == -np.inf:
                continue
            step = np.zeros((T, n))
            step[t, e] = 1e-5
            d = [ref.objective(z + s * step, ids, counts, dp, dl, top, 0.3, normalize, mask) for s in (1, -1)]
            assert abs((d[0] - d[1]) / 2e-5 - dz[t, e]) < 1e-8
