// mx_layout.h -- shared and tensor memory of the MXFP4 and mixture-of-experts kernels:
// plain arithmetic, so that it can be checked on the host.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define MX_HOST_DEVICE __host__ __device__
#else
#define MX_HOST_DEVICE
#endif

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

// -------------------------------- products of few rows or tiles, 8-bit operands --
// (Separate rings, a deeper one for the weights: 128 rows' tokens then had four stages, and
// their latency from L2 was what a stage took, 128 x 8192 x 8192 24.0 us against 18.8.)
constexpr int F8_ROWS_STAGES(int bt) { return bt <= 32 ? 10 : (bt == 64 ? 8 : 6); }   // at most

// The same with ring stages of 128 K: the weights' and the tokens' scale tile are 512
// bytes each, 8 columns of tensor memory.  CHUNKS: three accumulators.
template <int BT, bool CHUNKS = false>
struct F8RowsCfg {
    static constexpr int W_BYTES = 128 * 128, T_BYTES = BT * 128, S_BYTES = 1024;
    static constexpr int STAGE_BYTES = W_BYTES + T_BYTES + S_BYTES;
    static constexpr int MAX_STAGES = F8_ROWS_STAGES(BT);
    static constexpr int ACCS = CHUNKS ? 3 : 1;
    static constexpr uint32_t SCALE_COL = ACCS * BT, COLS = SCALE_COL + 8 * MAX_STAGES;
    static constexpr uint32_t TMEM_COLS = COLS <= 128 ? 128 : (COLS <= 256 ? 256 : 512);
    static constexpr int OFF_BAR = 0, OFF_MISC = (2 * MAX_STAGES + 4) * 8, OFF_RING = 1024;
    static constexpr int PART_BYTES = BT * 512;                          // a partial tile, over the ring
    static constexpr int MIN_SMEM = tmem_min_smem((int)TMEM_COLS);
    static constexpr int smem_bytes(int stages, int split)
    {
        const int ring = OFF_RING + stages * STAGE_BYTES, part = split > 1 ? OFF_RING + PART_BYTES : 0;
        const int need = ring > part ? ring : part;
        return need > MIN_SMEM ? need : MIN_SMEM;
    }
    static_assert(OFF_MISC + 16 <= OFF_RING && OFF_RING + MAX_STAGES * STAGE_BYTES <= CTA_SMEM, "shared memory budget");
    static_assert(COLS <= TMEM_COLS && MIN_SMEM <= OFF_RING + MAX_STAGES * STAGE_BYTES, "tensor memory budget");
};

// ----------------------------------------------------------- mixture of experts --
constexpr int MOE_MAX_T = 64, MOE_MAX_K = 16, MOE_MAX_E = 512;
constexpr int MOE_MIN_GROUP = 16;                              // tokens of an expert that share a read of its weights, at least
constexpr int MOE_MAX_BARS = 40;

// Shared memory of an experts kernel beside its rings.
struct MoeShared {
    float probs[MOE_MAX_T * MOE_MAX_K];
    short choice[MOE_MAX_T * MOE_MAX_K];           // slot t * k + j -> expert
    short slot[MOE_MAX_T * MOE_MAX_K];             // slots by expert
    short count[MOE_MAX_E], start[MOE_MAX_E];      // slots of an expert, its first entry of slot[]
    short act[MOE_MAX_E + MOE_MAX_T * MOE_MAX_K / MOE_MIN_GROUP];       // groups of tokens of one expert, by expert:
    short first[MOE_MAX_E + MOE_MAX_T * MOE_MAX_K / MOE_MIN_GROUP + 1];                   // the expert and the first entry of slot[]
    int nact;
    int abort_flag, go;
    uint32_t tmem;
    uint64_t bar[MOE_MAX_BARS];
};

// ------------------------------------------------ mixture of experts, 16-bit weights --
constexpr int MOE_GROUP = 32;                                  // tokens of one expert that share a read of its weights

// Two rings.  A stage of weights is 128 K of a tile, two boxes of 64 K for each half:
// with 64 K a stage, what a warp does once a stage (waits, addresses, giving it back)
// took longer than the multiplication (one token, 2 of 8 experts of 4096 x 1792: 47.7 us,
// with 128 K 41.6; 64 tokens, 8 of 64 experts: 456 and 445).  A stage of tokens is the
// group's tokens, a record for each and a copy to a record: x over 256 K (two stages of
// weights, 512 bytes), or h over 128 K (its three parts, 768 bytes), because copies of
// 128 bytes were measured to keep one warp busy for longer than the weights take.  A
// record is 64 bytes longer than a multiple of 128, so that two tokens' 64-byte pieces
// lie on different banks.  The tokens' ring has room for as many as the call can send to
// one expert, and more stages of few: h comes from L2 when the grid barrier opens, and
// with 512 K of it in flight its latency was most of a small down product's time.  The
// rest is weights' stages, filled while the CTA waits for the barrier.
constexpr int MOE_STAGE_K = 128, MOE_BOXES = MOE_STAGE_K / 64, MOE_PARTS = 3, MOE_PART = MOE_STAGE_K * 2;
constexpr int MOE_RECORD = MOE_PARTS * MOE_PART + 64, MOE_MAX_STAGES = 9, MOE_MAX_TSTAGES = 8;
// Stages of weights to a stage of tokens, and what one copy of them is: of x, of h.
template <bool DOWN>
constexpr int MOE_SPAN = DOWN ? 1 : 2;
template <bool DOWN>
constexpr int MOE_TOKEN_K = MOE_SPAN<DOWN> * MOE_STAGE_K;
template <bool DOWN>
constexpr int MOE_TOKEN = MOE_TOKEN_K<DOWN> * 2 * (DOWN ? MOE_PARTS : 1);
static_assert(MOE_TOKEN<false> <= MOE_RECORD && MOE_TOKEN<true> <= MOE_RECORD, "records");
constexpr int MOE_RINGS = (CTA_SMEM - (int)sizeof(MoeShared)) & ~15;
static_assert(2 * MOE_MAX_STAGES + 2 * MOE_MAX_TSTAGES <= MOE_MAX_BARS, "barriers");

// Groups of eight tokens that a product warp multiplies for `tokens` of them, and so
// the records that it reads of a stage, whether there are tokens in them or not: what
// they hold reaches columns that are not stored.
MX_HOST_DEVICE constexpr int moe_eights(int tokens) { return tokens <= 8 ? 1 : (tokens <= 16 ? 2 : 4); }

// Shared memory of a call: the rings, then MoeShared.  Before the rings start, all
// logits and after them a bit for each expert and slot stand in their place.
struct MoeLayout {
    int stages, tstages, stage_bytes, token_bytes, off_tokens, off_shared;
    MX_HOST_DEVICE constexpr MoeLayout(int T, int half_rows)
        : stages(0), tstages(T <= 8 ? MOE_MAX_TSTAGES : (T <= 16 ? 6 : 3)), stage_bytes(MOE_BOXES * half_rows * 256),
          token_bytes(8 * moe_eights(T < MOE_GROUP ? T : MOE_GROUP) * MOE_RECORD), off_tokens(0), off_shared(0)
    {
        const int room = (MOE_RINGS - tstages * token_bytes) / stage_bytes;
        stages = room < MOE_MAX_STAGES ? room : MOE_MAX_STAGES;
        off_tokens = stages * stage_bytes;
        const int rings = off_tokens + tstages * token_bytes, plan = T * MOE_MAX_E * 4 + MOE_MAX_E * ((T * MOE_MAX_K + 31) / 32) * 4;
        off_shared = rings > plan ? rings : plan;
    }
};

// Every T and tile height has room, and two stages of weights at least.
constexpr bool layout_fits()
{
    for (int half = 32; half <= 64; half += 8)
        for (int T = 1; T <= MOE_MAX_T; ++T)
            if (MoeLayout(T, half).off_shared > MOE_RINGS || MoeLayout(T, half).stages < 2) return false;
    return true;
}
static_assert(layout_fits(), "rings, logits and bits");

}  // namespace mmact
