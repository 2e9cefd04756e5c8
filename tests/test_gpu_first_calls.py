"""The first calls of a process, from several threads at once: each sets up its operator's kernels or waits for the
thread that does, and all get the same result.  A child process each, as set-up happens once in one."""
import os
import subprocess
import sys

import pytest

from conv_activation_epilogue_gb300 import build

pytestmark = pytest.mark.gpu
ROOT = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..")

CHILD = """
import threading
import torch
from conv_activation_epilogue_gb300 import mmact

mmact.load()
THREADS, M, N, K = 8, 96, 256, 512
a, b = torch.ones((M, K), device="cuda"), torch.full((N, K), 0.5, device="cuda")
fp8 = {fp8}


def packed(rows):
    if fp8:
        c, s = mmact.mmact_fp8_size(rows, K)
        return (torch.full((rows, c // rows), 0x38, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),    # 1.0
                torch.full((s,), 127, dtype=torch.uint8, device="cuda"))
    c, s = mmact.mmact_mxfp4_size(rows, K)
    return torch.full((c,), 0x22, dtype=torch.uint8, device="cuda"), torch.full((s,), 127, dtype=torch.uint8, device="cuda")


A, B = packed(M), packed(N)
out = [torch.zeros((M, N), device="cuda") for _ in range(THREADS)]
streams = [torch.cuda.Stream() for _ in range(THREADS)]
torch.cuda.synchronize()
gate, errors = threading.Barrier(THREADS), []


def call(i):
    try:
        gate.wait()
        (mmact.mmact_gemm_fp8 if fp8 else mmact.mmact_gemm_mxfp4)(*A, *B, None, out[i], K, stream=streams[i])
    except Exception as e:
        errors.append(repr(e))


threads = [threading.Thread(target=call, args=(i,)) for i in range(THREADS)]
for t in threads:
    t.start()
for t in threads:
    t.join()
torch.cuda.synchronize()
assert not errors, errors
assert mmact.mmact_get_last_error() == mmact.MMACT_OK
for o in out:
    assert bool((o == float(K)).all())
"""


@pytest.mark.parametrize("fp8", [True, False], ids=["fp8", "mxfp4"])
def test_first_calls_from_several_threads(fp8):
    build.build()
    r = subprocess.run([sys.executable, "-c", CHILD.format(fp8=fp8)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
