// mx_layout.h -- shared and tensor memory of the MXFP4 and mixture-of-experts kernels:
// plain arithmetic, so that it can be checked on the host.
#pragma once

#include <cstdint>

namespace mmact {

constexpr int CTA_SMEM = 232448;               // shared memory that one CTA can ask for
constexpr int SM_SMEM = 233472, CTA_RESERVED = 1024;   // an SM's, and what it takes for each CTA beside what that asks for
constexpr int SM_TMEM_COLS = 512;

// Shared memory to ask for, at least, with `cols` columns of tensor memory, so that CTAs
// which fit an SM's shared memory fit its tensor memory too, whatever kernels and
// streams they are of: tensor memory is handed out in 128 columns, so CTAs that ask
// for more than all of it ask for 640 at least, and a fifth of the shared memory for
// every 128 keeps those apart.  A CTA that found no columns would wait for as long as
// another one holds them, and that one may wait in a cluster barrier for a CTA that
// waits for columns itself.
constexpr int tmem_min_smem(int cols) { return (SM_SMEM / 5 + 1) * (cols / 128) - CTA_RESERVED; }

// ------------------------------------------------ products of few rows or tiles --
constexpr int MX_ROWS_STAGES(int bt) { return bt <= 32 ? 5 : (bt == 64 ? 8 : 6); }   // at most

// Shared memory: barriers, then the ring: its stages of weights, of tokens, of scales
// (as many as the K blocks of a CTA ask for, so that small products leave room for
// the next kernel's CTAs, whose set-up then overlaps).
template <int BT>
struct MxRowsCfg {
    static constexpr int W_BYTES = 128 * 128, T_BYTES = BT * 128, S_BYTES = 2 * 1024;
    static constexpr int STAGE_BYTES = W_BYTES + T_BYTES + S_BYTES;
    // Up to 32 rows: two CTAs fit on an SM, for the same overlap; else as many as fit.
    static constexpr int MAX_STAGES = MX_ROWS_STAGES(BT);
    static constexpr uint32_t SCALE_COL = BT;                            // 16 columns for each stage
    static constexpr uint32_t TMEM_COLS = BT + 16 * MAX_STAGES <= 128 ? 128 : 256;
    static constexpr int OFF_BAR = 0, OFF_MISC = (2 * MAX_STAGES + 2) * 8, OFF_RING = 1024;
    static constexpr int PART_BYTES = BT * 512;                          // a partial tile, over the ring
    static constexpr int MIN_SMEM = tmem_min_smem((int)TMEM_COLS);
    static constexpr int smem_bytes(int stages, int split)
    {
        const int ring = OFF_RING + stages * STAGE_BYTES, part = split > 1 ? OFF_RING + PART_BYTES : 0;
        const int need = ring > part ? ring : part;
        return need > MIN_SMEM ? need : MIN_SMEM;
    }
    static_assert(OFF_MISC + 16 <= OFF_RING && OFF_RING + MAX_STAGES * STAGE_BYTES <= CTA_SMEM, "shared memory budget");
    static_assert(BT + 16 * MAX_STAGES <= TMEM_COLS, "tensor memory budget");
};

}  // namespace mmact
