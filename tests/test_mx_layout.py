"""Shared and tensor memory of the MXFP4 and mixture-of-experts kernels: the arithmetic of
csrc/mx_layout.h, compiled for the host and checked for every plan (no GPU)."""
import itertools
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "conv_activation_epilogue_gb300", "csrc")
SM_SMEM, RESERVED, COLS = 228 * 1024, 1024, 512      # of an SM; kept by it for each CTA; of its tensor memory


def compiled(tmp_path_factory, body):
    d = tmp_path_factory.mktemp("layout")
    (d / "m.cpp").write_text('#include <cstdio>\n#include "mx_layout.h"\nusing namespace mmact;\n' + body)
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(d / "m.cpp"), "-o", str(d / "m")], check=True)
    out = subprocess.run([str(d / "m")], check=True, capture_output=True, text=True).stdout
    return [tuple(map(int, line.split())) for line in out.splitlines()]


@pytest.fixture(scope="module")
def rows_kernels(tmp_path_factory):
    """(rows of a tile, ring stages, CTAs of a cluster, shared memory, columns of tensor memory)"""
    return compiled(tmp_path_factory, """
template <int BT> void all()
{
    for (int split = 1; split <= 8; split *= 2)
        for (int s = 1; s <= MxRowsCfg<BT>::MAX_STAGES; ++s)
            std::printf("%d %d %d %d %d\\n", BT, s, split, MxRowsCfg<BT>::smem_bytes(s, split), (int)MxRowsCfg<BT>::TMEM_COLS);
}
int main() { all<16>(); all<32>(); all<64>(); all<128>(); }
""")


def test_ctas_that_share_an_sm_all_have_their_columns(rows_kernels):
    """Products on several streams put CTAs of different kernels on one SM.  One that finds no columns
    waits for those that hold them, and these may wait for it, through their clusters: whatever fits an
    SM's shared memory has to fit its tensor memory."""
    smallest = {}
    for _, _, _, smem, cols in rows_kernels:
        smallest[cols] = min(smem, smallest.get(cols, smem))
        assert smem <= SM_SMEM - RESERVED
    assert set(smallest) <= {128, 256, 512}
    for n in range(1, 9):
        for mix in itertools.combinations_with_replacement(sorted(smallest), n):
            if sum(smallest[c] + RESERVED for c in mix) <= SM_SMEM:
                assert sum(mix) <= COLS, mix


def test_few_rows_leave_room_for_the_next_kernels_ctas(rows_kernels):
    """Two CTAs of up to 32 rows share an SM with full rings."""
    for bt, _, _, smem, _ in rows_kernels:
        if bt <= 32:
            assert 2 * (smem + RESERVED) <= SM_SMEM
