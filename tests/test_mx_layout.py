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


@pytest.fixture(scope="module")
def moe_layouts(tmp_path_factory):
    """(tokens, half a tile's rows, weight stages, bytes of one, token stages, bytes of one, their offset,
    MoeShared's offset, its size, bytes of a token's record)"""
    return compiled(tmp_path_factory, """
int main()
{
    for (int T = 1; T <= MOE_MAX_T; ++T)
        for (int half = 32; half <= 64; half += 8) {
            const MoeLayout l(T, half);
            std::printf("%d %d %d %d %d %d %d %d %d %d\\n", T, half, l.stages, l.stage_bytes, l.tstages, l.token_bytes, l.off_tokens,
                        l.off_shared, (int)sizeof(MoeShared), MOE_RECORD);
        }
}
""")


def test_a_token_stage_holds_every_record_that_is_read(moe_layouts):
    """An expert with n tokens is multiplied 8, 16 or 32 at a time, from as many records."""
    assert len(moe_layouts) == 64 * 5
    for T, _, _, _, _, token_bytes, _, _, _, record in moe_layouts:
        for n in range(1, min(T, 32) + 1):
            assert (8 if n <= 8 else 16 if n <= 16 else 32) * record <= token_bytes, (T, n)


def test_the_mixtures_rings_do_not_overlap(moe_layouts):
    for T, half, stages, stage_bytes, tstages, token_bytes, off_tokens, off_shared, shared, _ in moe_layouts:
        assert stages >= 2 and tstages >= 2 and stages * stage_bytes <= off_tokens
        assert stage_bytes == 2 * half * 256                 # 128 K of 2 * half rows
        assert off_tokens + tstages * token_bytes <= off_shared and off_shared % 16 == 0
        assert off_shared + shared <= SM_SMEM - RESERVED
        # all logits, and a bit for each expert and slot, before the rings start
        assert T * 512 * 4 + 512 * ((T * 16 + 31) // 32) * 4 <= off_shared
