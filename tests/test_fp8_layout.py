"""Shared and tensor memory of the 8-bit products of few rows: the arithmetic of csrc/mx_layout.h, compiled for the
host and checked for every plan (no GPU)."""
import itertools
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "conv_activation_epilogue_gb300", "csrc")
SM_SMEM, RESERVED, COLS = 228 * 1024, 1024, 512      # of an SM; kept by it for each CTA; of its tensor memory

PROGRAM = """
#include <cstdio>
#include "mx_layout.h"
using namespace mmact;
template <typename Cfg> void all(int kind, int bt)
{
    for (int split = 1; split <= 8; split *= 2)
        for (int s = 1; s <= Cfg::MAX_STAGES; ++s)
            std::printf("%d %d %d %d %d %d %d %d %d\\n", kind, bt, s, split, Cfg::smem_bytes(s, split), (int)Cfg::TMEM_COLS, Cfg::OFF_MISC,
                        Cfg::OFF_RING, Cfg::MAX_STAGES);
}
int main()
{
    all<F8RowsCfg<16>>(8, 16); all<F8RowsCfg<32>>(8, 32); all<F8RowsCfg<64>>(8, 64); all<F8RowsCfg<128>>(8, 128);
    all<F8RowsCfg<16, true>>(24, 16); all<F8RowsCfg<32, true>>(24, 32); all<F8RowsCfg<64, true>>(24, 64); all<F8RowsCfg<128, true>>(24, 128);
    all<MxRowsCfg<16>>(4, 16); all<MxRowsCfg<32>>(4, 32); all<MxRowsCfg<64>>(4, 64); all<MxRowsCfg<128>>(4, 128);
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """(operands' bits, times the accumulators, rows of a tile, ring stages, CTAs of a cluster, shared memory, columns, two offsets, most stages)"""
    d = tmp_path_factory.mktemp("layout")
    (d / "m.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(d / "m.cpp"), "-o", str(d / "m")], check=True)
    out = subprocess.run([str(d / "m")], check=True, capture_output=True, text=True).stdout
    return [tuple(map(int, line.split())) for line in out.splitlines()]


def test_ctas_that_share_an_sm_all_have_their_columns(plans):
    """Of 8-bit and 4-bit products alike: whatever fits an SM's shared memory has to fit its tensor memory."""
    smallest = {}
    for _, _, _, _, smem, cols, _, _, _ in plans:
        smallest[cols] = min(smem, smallest.get(cols, smem))
        assert smem <= SM_SMEM - RESERVED
    for n in range(1, 9):
        for mix in itertools.combinations_with_replacement(sorted(smallest), n):
            if sum(smallest[c] + RESERVED for c in mix) <= SM_SMEM:
                assert sum(mix) <= COLS, mix


def test_parts_do_not_overlap(plans):
    """Barriers (full and empty of each stage, even and odd chunk full, drained, sum taken over), two words, the ring or a partial tile."""
    for bits, bt, stages, split, smem, cols, misc, ring, most in plans:
        if bits == 4:
            continue
        assert (2 * most + 4) * 8 <= misc and misc % 8 == 0 and misc + 16 <= ring and ring % 1024 == 0
        assert ring + stages * (128 * 128 + bt * 128 + 1024) <= smem
        assert split == 1 or ring + bt * 512 <= smem
        assert bits // 8 * bt + 8 * most <= cols


def test_few_rows_leave_room_for_another_cta(plans):
    """Two CTAs of up to 32 rows share an SM with rings of five stages."""
    for bits, bt, stages, _, smem, _, _, _, _ in plans:
        if bits != 4 and bt <= 32 and stages <= 5:
            assert 2 * (smem + RESERVED) <= SM_SMEM
