"""The tensor-map cache under the MXFP4 product of large outputs, which takes five maps: a repeated
call encodes none, even where all five belong to one set of the cache."""
import struct

import numpy as np
import pytest
import torch

import mx_reference as ref
from conv_activation_epilogue_gb300 import build, mmact
from test_gpu_mxfp4 import host64, random_mx

pytestmark = pytest.mark.gpu
SETS = 64                                                      # a multiple of the cache's number of sets
BF16, F32 = 9, 7                                               # the driver's CUtensorMapDataType values


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    mmact.load()


def cache_set(ptr, kind, swizzle, dims, stride, box):
    """The set that a map's key hashes to (64-bit FNV-1a over its fields)."""
    key = struct.pack("<4iQ5Q4Q5I5I", kind, 2, swizzle, 0, ptr, *dims, 0, 0, 0, stride, 0, 0, 0, *box, 0, 0, 0, 1, 1, 0, 0, 0)
    h = 1469598103934665603
    for b in key:
        h = (h ^ b) * 1099511628211 & 0xFFFFFFFFFFFFFFFF
    return h % SETS


def test_five_maps_of_one_set():
    M = N = K = 256
    rng = np.random.default_rng(0)
    (ac, as_, av), (bc, bs, bv) = random_mx(rng, M, K), random_mx(rng, N, K)
    codes, scales = (64, M), (K // 128 * 128, 2)               # extents in 16- and 32-bit words
    keys = {"ac": (BF16, 1, codes, 128, (64, 128)), "as": (F32, 0, scales, 1024, (256, 1)),
            "bc": (BF16, 1, codes, 128, (64, 128)), "bs": (F32, 0, scales, 1024, (256, 2)),
            "c": (BF16, 1, (N, M), 2 * N, (64, 32))}
    room = torch.empty(5 << 18, dtype=torch.uint8, device="cuda")
    at = {}
    for i, (name, key) in enumerate(keys.items()):             # an address of each array whose map falls into set 7
        at[name] = next(o for o in range(i << 18, (i << 18) + (1 << 17), 16) if cache_set(room.data_ptr() + o, *key) == 7)
    view = lambda name, n: room[at[name]: at[name] + n]        # noqa: E731
    a, sa, b, sb = view("ac", ac.numel()).view(M, -1), view("as", as_.numel()), view("bc", bc.numel()).view(N, -1), view("bs", bs.numel())
    C = view("c", 2 * M * N).view(torch.bfloat16).view(M, N)
    for to, v in ((a, ac), (sa, as_), (b, bc), (sb, bs)):
        to.copy_(v)
    mmact.mmact_set_gemm_mxfp4_kernel(2)
    try:
        counts = []
        for _ in range(6):
            C.zero_()
            mmact.mmact_gemm_mxfp4(a, sa, b, sb, None, C, K)
            counts.append(mmact.mmact_tensor_map_cache_stats()[1])
    finally:
        mmact.mmact_set_gemm_mxfp4_kernel(0)
    assert mmact.mmact_get_last_error() == mmact.MMACT_OK
    want, bound = ref.gemm(av, bv, None, "none", 0.0)
    assert np.all(np.abs(host64(C) - want) <= bound + ref.ulp(np.abs(want) + bound, "bf16"))
    assert counts[2:] == counts[2:3] * 4, counts               # the second call may still encode what the first one's new maps replaced
