// moe.cu -- a whole mixture-of-experts layer for a few tokens (T <= 64) in two
// kernels.
//
//   router kernel    logits[t][e] = x[t] . router[e] + rb[e]
//   experts kernel   the k experts of each token (largest logits, ties to the
//                    lowest index) and their softmax weights; for every chosen
//                    expert, read once for up to 32 of its tokens:
//                    h = act(g) * u, g and u the two halves of w1[e] x + b1[e]
//                    (or h = act(w1[e] x + b1[e])); a grid barrier;
//                    o = w2[e] h + b2[e]; a grid barrier; y[t] = sum_j p[t][j] o[t, j]
//
// With few tokens every weight is used a handful of times: the time is that of
// reading the chosen experts' weights once, and everything is arranged so that
// the copies never stop.  The experts kernel is persistent, one CTA on each SM,
// taking the items in turn (a tile of weight rows x all of K of one expert; for a
// gated layer half of the rows are gate rows and half the up rows that go with
// them):
//
//   warp 0       producer: two TMA boxes (the tile's halves) of 128 bytes of K to a
//                ring stage.  It runs ahead over items and over the grid barrier:
//                weights of the down product are on their way while the last h is
//                being finished.
//   warp 9       tokens of the stage (x, or h once the grid barrier is passed), one
//                bulk copy for each token
//   warps 1..8   products: each has 8 + 8 rows of the tile on mma.sync.m16n8k16
//                as the 16-row operand (a gate row and its up row meet in one
//                thread) and eight tokens to its columns, over all of K, so no sums
//                cross warps; bias, activation and stores follow in registers.
//                Which K a lane holds does not matter to a sum over K as long as
//                both operands agree, so fragments are 16-byte loads in memory
//                order.
//
// The intermediate h is held as two bf16 halves hi = bf16(h), lo = bf16(h - hi),
// 16 bits of it, and multiplied as both, so no rounding to 16 bits stands between
// the two products.  fp16 down weights are split the same way (hi + lo is exact),
// which keeps h's fp32 range.  MXFP4 weights become bf16 in registers (exactly: a
// scale is a power of two).
#include "common.cuh"
#include "kernels_mx.h"
#include "mxfp4.cuh"

namespace mmact {

enum : int { W_F16 = 0, W_BF16 = 1, W_MX = 2 };

constexpr int MOE_MAX_T = 64, MOE_MAX_K = 16, MOE_MAX_E = 512;
constexpr int MOE_MMA_WARPS = 8;
constexpr int MOE_THREADS = 32 * (2 + MOE_MMA_WARPS);

// Tokens of one expert that share a read of its weights.
template <int W>
constexpr int MOE_GROUP = W == W_MX ? 16 : 32;
constexpr int MOE_MIN_GROUP = 16;

// Two rings.  A stage of weights is at most 128 rows x 128 bytes: 8 stages, about
// twice what has to be in flight on an SM.  A stage of tokens is the group's
// tokens over 256 K (four stages of 16-bit weights, one of MXFP4), hi and lo, a
// record for each: 512 bytes to a copy, because copies of 128 bytes were measured
// to keep one warp busy for twice the time of the weights' stage.  A record is 64
// bytes longer than a multiple of 128, so that two tokens' 64-byte pieces lie on
// different banks.
constexpr int MOE_STAGE_BYTES = 16384, MOE_STAGES = 8;
constexpr int MOE_TOKEN_K = 256, MOE_TOKEN = MOE_TOKEN_K * 2, MOE_RECORD = 2 * MOE_TOKEN + 64;
template <int W>
struct MoeRing {
    static constexpr int K = W == W_MX ? 256 : 64;             // K of a stage of weights
    static constexpr int SPAN = MOE_TOKEN_K / K;               // stages of weights to one of tokens
    static constexpr int TOKENS = MOE_GROUP<W> * MOE_RECORD;   // bytes of a stage of tokens
    static constexpr int TSTAGES = W == W_MX ? 4 : 2;
    static constexpr int OFF_TOKENS = MOE_STAGES * MOE_STAGE_BYTES;
    static constexpr int BYTES = OFF_TOKENS + TSTAGES * TOKENS;
};
constexpr int MOE_MAX_TSTAGES = 4;

// ------------------------------------------------------------------ helpers --
// A logit as a key whose unsigned order is the float order, NaN above all, and
// -0 equal to +0; never 0.
__device__ __forceinline__ uint32_t logit_key(float x)
{
    if (x != x) return 0xffffffffu;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

template <bool BF16>
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1)
{
    if constexpr (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Where element k of a token's row stands in the arrays that the products read.
// 16-bit weights: in place.  MXFP4: a lane holds a block of 32 codes, four words
// of eight, and a warp multiplies word w of the blocks t = 0..3 of 128 K at a
// time: so [w][t][8], and within the eight the order 0 4 1 5 2 6 3 7, because a
// word of eight codes yields its values as the pairs (i, i + 4).
template <int W>
__device__ __forceinline__ int token_at(int k)
{
    if constexpr (W != W_MX) return k;
    return (k & ~127) | ((k >> 3 & 3) << 5) | ((k >> 5 & 3) << 3) | ((k & 3) << 1) | (k >> 2 & 1);
}

// Eight codes times X as four bf16 pairs (i, i + 4).  A code moved to the top of
// its half-word has its sign in place; its three magnitude bits, moved to the
// lowest exponent bits and the highest fraction bit, read as the value times
// 2^-126 (0.5 as a subnormal).  One product with 2^126 X gives the bf16 value
// exactly; `m1` holds that factor, and `m2` the rest of it when X > 2.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ void mx_word_bf16(uint32_t w, uint32_t m1, uint32_t (&v)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t y = w << (12 - 4 * i);
        const uint32_t sign = y & 0x80008000u;
        const int s = 6 - (12 - 4 * i);                       // right shift (negative: left) of w
        const uint32_t em = s >= 0 ? w >> s : w << -s;
        v[i] = mul_bf16x2((em & 0x01c001c0u) | sign, m1);
    }
}

// Hi and lo bf16 halves of a pair of fp32 values.
__device__ __forceinline__ void split_pair(float a, float b, uint32_t &hi, uint32_t &lo)
{
    hi = pack2<OUT_BF16>(a, b);
    const float2 f = unpack2<OUT_BF16>(hi);
    lo = pack2<OUT_BF16>(a - f.x, b - f.y);
}

// Whole-warp forms of TMA instructions, issued by one elected lane (see mma_mxf4).
#define MMACT_ELECTED "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"

__device__ __forceinline__ void elected_expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile(MMACT_ELECTED "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void elected_load_2d(uint32_t dst, const CUtensorMap *m, uint32_t bar, int x, int y, uint64_t pol)
{
    asm volatile(MMACT_ELECTED
                 "@q cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
                 "[%0], [%1, {%3, %4}], [%2], %5;\n\t}" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "l"(pol)
                 : "memory");
}

#undef MMACT_ELECTED

// Copy of `bytes` (a multiple of 16) from global to shared memory, both 16-byte
// aligned, counted on an mbarrier; by each lane that calls it.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// Orders this thread's (and, through barriers, others') ordinary global accesses
// with bulk copies.
__device__ __forceinline__ void fence_proxy_async_all()
{
    asm volatile("fence.proxy.async;" ::: "memory");
}

// ------------------------------------------------------------------- router --
// One CTA for an expert and eight tokens: four warps share K.  The CTAs past
// those prepare what the experts kernel reads: its counters, x in
// the products' order (MXFP4: as bf16, hi and for fp16 x lo) with zeros up to a
// whole stage, and the same zeros of h.
constexpr int MOE_ROUTER_THREADS = 128;

template <int XT, int W>
__global__ void __launch_bounds__(MOE_ROUTER_THREADS) moe_router_kernel(const MoeArgs p, int token_groups)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    __shared__ float red[4][8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint16_t *xs = static_cast<const uint16_t *>(p.x);
    if ((int)blockIdx.x < p.E * token_groups) {
        const int e = blockIdx.x / token_groups, t0 = (blockIdx.x - e * token_groups) * 8, n = min(8, p.T - t0);
        const uint16_t *r = static_cast<const uint16_t *>(p.router) + (int64_t)e * p.H;
        float s[8] = {};
        for (int k = threadIdx.x * 8; k < p.H; k += MOE_ROUTER_THREADS * 8) {
            const uint4 b = __ldg(reinterpret_cast<const uint4 *>(r + k));
            const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
            uint4 a[8];                                        // tokens past the last one: the last one again
#pragma unroll
            for (int t = 0; t < 8; ++t) a[t] = __ldg(reinterpret_cast<const uint4 *>(xs + (int64_t)(t0 + min(t, n - 1)) * p.H + k));
            float2 g[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) g[j] = unpack2<XT>(bw[j]);
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const uint32_t aw[4] = {a[t].x, a[t].y, a[t].z, a[t].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = unpack2<XT>(aw[j]);
                    s[t] = fmaf(f.x, g[j].x, s[t]);
                    s[t] = fmaf(f.y, g[j].y, s[t]);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s[t] += __shfl_xor_sync(0xffffffffu, s[t], o);
            if (lane == 0) red[warp][t] = s[t];
        }
        __syncthreads();
        if (threadIdx.x < n)
            p.logits[(int64_t)(t0 + threadIdx.x) * p.E + e] =
                (red[0][threadIdx.x] + red[1][threadIdx.x]) + (red[2][threadIdx.x] + red[3][threadIdx.x]) +
                (p.router_bias != nullptr ? p.router_bias[e] : 0.0f);
        return;
    }
    // 1024 K of one token: 8 consecutive values, which stay together, to a thread
    const int chunks = (p.Hp + 1023) / 1024, at = (int)blockIdx.x - p.E * token_groups, t = at / chunks;
    const int k = (at - t * chunks) * 1024 + (int)threadIdx.x * 8;
    if (at == 0 && threadIdx.x < 2) p.counters[threadIdx.x] = 0;
    if (k < p.Hp) {
        const uint4 raw = k < p.H ? __ldg(reinterpret_cast<const uint4 *>(xs + (int64_t)t * p.H + k)) : make_uint4(0, 0, 0, 0);
        const int64_t to = (int64_t)t * p.Hp + token_at<W>(k);
        if constexpr (W != W_MX) {
            *reinterpret_cast<uint4 *>(p.x_hi + to) = raw;
        } else {
            // the pairs (i, i + 4) of the eight values
            const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
            uint32_t v[4], l[4] = {};
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __byte_perm(w[i >> 1], w[2 + (i >> 1)], i & 1 ? 0x7632 : 0x5410);
            if constexpr (XT == OUT_F16) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = unpack2<OUT_F16>(v[i]);
                    split_pair(f.x, f.y, v[i], l[i]);
                }
                *reinterpret_cast<uint4 *>(p.x_lo + to) = make_uint4(l[0], l[1], l[2], l[3]);
            }
            *reinterpret_cast<uint4 *>(p.x_hi + to) = make_uint4(v[0], v[1], v[2], v[3]);
        }
    }
    if (at != t * chunks) return;
    const int pad = (p.Ip - p.I) / 8;                          // eights of zeros past h's rows
    for (int i = threadIdx.x; i < pad * p.top; i += MOE_ROUTER_THREADS) {
        const int64_t to = ((int64_t)t * p.top + i / pad) * p.Ip + token_at<W>(p.I + i % pad * 8);
        *reinterpret_cast<uint4 *>(p.h_hi + to) = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4 *>(p.h_lo + to) = make_uint4(0, 0, 0, 0);
    }
}

// ------------------------------------------------------------ choice of experts --
// Shared memory of the experts kernel beside the ring.
struct MoeShared {
    float probs[MOE_MAX_T * MOE_MAX_K];
    short choice[MOE_MAX_T * MOE_MAX_K];           // slot t * k + j -> expert
    short slot[MOE_MAX_T * MOE_MAX_K];             // slots by expert
    short count[MOE_MAX_E], start[MOE_MAX_E];      // slots of an expert, its first entry of slot[]
    short act[MOE_MAX_E + MOE_MAX_T * MOE_MAX_K / MOE_MIN_GROUP];       // groups of tokens of one expert, by expert:
    short first[MOE_MAX_E + MOE_MAX_T * MOE_MAX_K / MOE_MIN_GROUP + 1];                   // the expert and the first entry of slot[]
    int nact;
    int abort_flag, go;
    uint64_t bar[2 * MOE_STAGES + 2 * MOE_MAX_TSTAGES];
};

// Top k of N tokens t, t + stride, ... by one warp: each round the largest key of
// those left, then the lowest index that has it; then the softmax weights, one to
// a lane.  A round is a chain of dependent steps: several tokens go through it
// side by side.
template <int N>
__device__ __forceinline__ void choose_experts(const MoeArgs &p, MoeShared &S, const float *logits, int t, int stride, int lane,
                                               bool write)
{
    static_assert(MOE_MAX_E <= 32 * 32, "one bit for each of a lane's logits");
    uint32_t taken[N] = {};                                    // bit i: this lane's logit i * 32 + lane is chosen
    int mine[N] = {}, first[N] = {};
    for (int j = 0; j < p.top; ++j) {
        uint32_t key[N] = {}, at[N] = {};
        for (int e = lane, i = 0; e < p.E; e += 32, ++i)
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const uint32_t k = (taken[n] >> i) & 1u ? 0u : logit_key(logits[(t + n * stride) * p.E + e]);
                if (k > key[n]) key[n] = k, at[n] = (uint32_t)e;
            }
        __syncwarp();
        uint32_t best[N];
#pragma unroll
        for (int n = 0; n < N; ++n) best[n] = __reduce_max_sync(0xffffffffu, key[n]);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int e = (int)__reduce_min_sync(0xffffffffu, key[n] == best[n] ? at[n] : 0xffffu);
            if ((e & 31) == lane) taken[n] |= 1u << (e >> 5);
            if (j == 0) first[n] = e;
            if (j == lane) mine[n] = e;
        }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const float *row = logits + (t + n * stride) * p.E;
        const float peak = row[first[n]];
        const float w = lane < p.top ? expf(row[mine[n]] - peak) : 0.0f;
        float total = w;
        if (!p.normalize) {
            total = 0.0f;
            for (int e = lane; e < p.E; e += 32) total += expf(row[e] - peak);
            __syncwarp();
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        if (lane < p.top) {
            const int at = (t + n * stride) * p.top + lane;
            S.choice[at] = (short)mine[n];
            S.probs[at] = w / total;
            if (write) {
                p.experts[at] = mine[n];
                p.probs[at] = w / total;
            }
        }
    }
}

// The slots of each expert, in groups, built by every CTA.  `mask`: for each
// expert one bit for each slot (in shared memory that is free until the rings
// start), from which counts and places follow by counting bits.
template <int GROUP>
__device__ __forceinline__ void build_lists(const MoeArgs &p, MoeShared &S, uint32_t *mask)
{
    const int tid = threadIdx.x, n_slots = p.T * p.top, words = (n_slots + 31) / 32;
    for (int i = tid; i < p.E * words; i += MOE_THREADS) mask[i] = 0;
    ptx::cta_sync();
    for (int s = tid; s < n_slots; s += MOE_THREADS) atomicOr(&mask[S.choice[s] * words + (s >> 5)], 1u << (s & 31));
    ptx::cta_sync();
    for (int e = tid; e < p.E; e += MOE_THREADS) {
        int c = 0;
        for (int w = 0; w < words; ++w) c += __popc(mask[e * words + w]);
        S.count[e] = (short)c;
    }
    ptx::cta_sync();
    if (tid < 32) {                                            // 32 experts at a time: running sums over the warp
        int n = 0, at = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + tid, c = e < p.E ? S.count[e] : 0, groups = (c + GROUP - 1) / GROUP;
            int sum = c, gsum = groups;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, sum, o), gup = __shfl_up_sync(0xffffffffu, gsum, o);
                if (tid >= o) sum += up, gsum += gup;
            }
            if (e < p.E) S.start[e] = (short)(at + sum - c);
            for (int g = 0; g < groups; ++g) {
                S.act[n + gsum - groups + g] = (short)e;
                S.first[n + gsum - groups + g] = (short)(at + sum - c + g * GROUP);
            }
            n += __shfl_sync(0xffffffffu, gsum, 31);
            at += __shfl_sync(0xffffffffu, sum, 31);
        }
        if (tid == 0) {
            S.first[n] = (short)at;
            S.nact = n;
        }
    }
    ptx::cta_sync();
    for (int s = tid; s < n_slots; s += MOE_THREADS) {
        const int e = S.choice[s];
        int at = S.start[e] + __popc(mask[e * words + (s >> 5)] & ((1u << (s & 31)) - 1u));
        for (int w = 0; w < s >> 5; ++w) at += __popc(mask[e * words + w]);
        S.slot[at] = (short)s;
    }
    ptx::cta_sync();
}

// ----------------------------------------------------------------- products --
// One product of the layer as the roles see it.  A tile is 2 * half_rows weight
// rows: r0 .. r0 + half_rows and the same number from `half` rows further on.
struct MoeProduct {
    int K, stages, tstages;          // ring stages of one item: weights, tokens
    int tiles;                       // items of one group of tokens
    int rows;                        // rows of one expert's matrix
    int half;                        // row distance between a tile's halves: I (gate, up), or half_rows
    int step;                        // rows from one tile to the next
    int limit;                       // rows the tiles count over: I or H
    const uint8_t *scales;           // MXFP4
    int64_t all_rows;                // rows of all experts
    int scale_tiles;                 // tiles of 128 K
    bool pairs;                      // the halves go together (gate, up)
};

__device__ __forceinline__ uint32_t word_of(const uint4 &u, int i)
{
    return i == 0 ? u.x : (i == 1 ? u.y : (i == 2 ? u.z : u.w));
}

// Factor 2^126 X of a scale byte as a bf16 pair; `rest` the part of X past 2.
__device__ __forceinline__ uint32_t mx_factor(uint32_t b, uint32_t &rest)
{
    const uint32_t e = min(b, 128u) + 126u;
    uint32_t m = b == 255u ? 0x7fc0u : e << 7;
    rest = b == 255u || b <= 128u ? 0x3f80u : (b - 128u + 127u) << 7;
    rest |= rest << 16;
    return m | (m << 16);
}


// A warp's view of an item.
struct MoeItem {
    uint32_t row;                    // shared address of this lane's row in the lower half, from a stage's start
    uint32_t upper;                  // from there to its row in the upper half
    int64_t ra, rb;                  // the two rows in the matrix of all experts
};

// Tokens of one piece of K (16 bytes of each row): this lane's 8 values of one
// token of each eight, hi and lo.
template <int NT, bool LO>
struct MoeTokens {
    uint4 h[NT], l[LO ? NT : 1];
};

template <int NT, bool LO>
__device__ __forceinline__ void load_tokens(MoeTokens<NT, LO> &x, uint32_t at)
{
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        x.h[n] = ptx::ld_shared_v4(at + n * 8 * MOE_RECORD);
        if constexpr (LO) x.l[n] = ptx::ld_shared_v4(at + n * 8 * MOE_RECORD + MOE_TOKEN);
    }
}

// acc += 16 rows x tokens over one piece: a, b the two rows' four pairs of values.
// The lo halves have sums of their own, so that half as many instructions wait
// for one another.
template <bool BF, int NT, bool LO>
__device__ __forceinline__ void piece_mma(float (&acc)[NT][4], float (&low)[LO ? NT : 1][4], const uint32_t (&a)[4],
                                          const uint32_t (&b)[4], const MoeTokens<NT, LO> &x)
{
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        mma_16816<BF>(acc[n], a[0], b[0], a[1], b[1], x.h[n].x, x.h[n].y);
        if constexpr (LO) mma_16816<BF>(low[n], a[0], b[0], a[1], b[1], x.l[n].x, x.l[n].y);
        mma_16816<BF>(acc[n], a[2], b[2], a[3], b[3], x.h[n].z, x.h[n].w);
        if constexpr (LO) mma_16816<BF>(low[n], a[2], b[2], a[3], b[3], x.l[n].z, x.l[n].w);
    }
}

// The rings of one CTA.
struct MoePipe {
    Pipe pp;                         // weights: full0, empty0
    uint32_t tfull0, tempty0;        // tokens
    uint32_t ring, tokens;           // shared addresses
};

// Stages used so far by a role.
struct MoeUse {
    uint32_t w, t;
};

// One warp's rows of an item over all of K: the two units of 64 bytes of each stage.
template <int W, int NT, bool LO, bool SPLITW>
__device__ __forceinline__ bool item_mma(float (&acc)[NT][4], const MoePipe &m, const MoeProduct &pr, const MoeItem &it,
                                         MoeUse use)
{
    using R = MoeRing<W>;
    const int lane = threadIdx.x & 31;
    const uint32_t sw = (uint32_t)(lane >> 2), t4 = (uint32_t)(lane & 3);   // the 128-byte swizzle: chunk ^ (row & 7)
    const uint32_t c0 = (t4 ^ sw) << 4, c1 = ((4u + t4) ^ sw) << 4;
    float low[LO || SPLITW ? NT : 1][4] = {};
    // MXFP4: the scale words of the two rows, loaded a stage ahead
    int64_t sa_at = 0, sb_at = 0;
    bool has_a = false, has_b = false;
    uint32_t wa[2] = {}, wb[2] = {};
    auto scales = [&](int u, uint32_t &a, uint32_t &b) {
        a = has_a && u < pr.scale_tiles ? __ldg(reinterpret_cast<const uint32_t *>(pr.scales + sa_at + (int64_t)u * 512)) : 0u;
        b = has_b && u < pr.scale_tiles ? __ldg(reinterpret_cast<const uint32_t *>(pr.scales + sb_at + (int64_t)u * 512)) : 0u;
    };
    if constexpr (W == W_MX) {
        sa_at = mx_scale_at(it.ra, 0, pr.scale_tiles);
        sb_at = mx_scale_at(it.rb, 0, pr.scale_tiles);
        has_a = it.ra < pr.all_rows;
        has_b = it.rb < pr.all_rows;
        scales(0, wa[0], wb[0]);
        scales(1, wa[1], wb[1]);
    }
#pragma unroll 1
    for (int s = 0; s < pr.stages; ++s, ++use.w) {
        const uint32_t slot = use.w % MOE_STAGES, row = m.ring + slot * MOE_STAGE_BYTES + it.row;
        const uint32_t part = (uint32_t)s % R::SPAN, tslot = use.t % R::TSTAGES;
        const uint32_t tok = m.tokens + tslot * R::TOKENS + sw * MOE_RECORD + part * (R::K * 2u) + t4 * 16u;
        if (part == 0 && !mx_warp_wait(m.pp, m.tfull0 + 8 * tslot, (use.t / R::TSTAGES) & 1u)) return false;
        if (!mx_warp_wait(m.pp, m.pp.full0 + 8 * slot, (use.w / MOE_STAGES) & 1u)) return false;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint4 fa = ptx::ld_shared_v4(row + (u ? c1 : c0)), fb = ptx::ld_shared_v4(row + it.upper + (u ? c1 : c0));
            if constexpr (W == W_MX) {
                // 128 K: a block of 32 codes to a lane, four words of eight
                const uint32_t sa = (wa[u] >> (8 * t4)) & 255u, sb = (wb[u] >> (8 * t4)) & 255u;
                scales(2 * s + 2 + u, wa[u], wb[u]);
                uint32_t ra, rb;
                const uint32_t ma = mx_factor(sa, ra), mb = mx_factor(sb, rb);
                const bool big = __any_sync(0xffffffffu, sa > 128u || sb > 128u);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    MoeTokens<NT, LO> x;
                    load_tokens<NT, LO>(x, tok + u * 256u + w * 64u);
                    uint32_t va[4], vb[4];
                    mx_word_bf16(word_of(fa, w), ma, va);
                    mx_word_bf16(word_of(fb, w), mb, vb);
                    if (big) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            va[i] = mul_bf16x2(va[i], ra);
                            vb[i] = mul_bf16x2(vb[i], rb);
                        }
                    }
                    piece_mma<true, NT, LO>(acc, low, va, vb, x);
                }
            } else {
                // 32 K: 8 values to a lane
                MoeTokens<NT, LO> x;
                load_tokens<NT, LO>(x, tok + u * 64u);
                uint32_t a[4] = {fa.x, fa.y, fa.z, fa.w}, b[4] = {fb.x, fb.y, fb.z, fb.w};
                if constexpr (SPLITW) {
                    // fp16 weights as two bf16 halves; the lo halves meet the tokens' hi halves only
                    uint32_t al[4], bl[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 va = unpack2<OUT_F16>(a[i]), vb = unpack2<OUT_F16>(b[i]);
                        split_pair(va.x, va.y, a[i], al[i]);
                        split_pair(vb.x, vb.y, b[i], bl[i]);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma_16816<true>(low[n], al[0], bl[0], al[1], bl[1], x.h[n].x, x.h[n].y);
                        mma_16816<true>(low[n], al[2], bl[2], al[3], bl[3], x.h[n].z, x.h[n].w);
                    }
                }
                piece_mma<W == W_BF16 || SPLITW, NT, LO>(acc, low, a, b, x);
            }
        }
        const bool last = part == R::SPAN - 1 || s == pr.stages - 1;   // of its stage of tokens
        __syncwarp();
        if (lane == 0) {
            ptx::mbar_arrive(m.pp.empty0 + 8 * slot);
            if (last) ptx::mbar_arrive(m.tempty0 + 8 * tslot);
        }
        use.t += last ? 1u : 0u;
    }
    if constexpr (LO || SPLITW)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[n][j] += low[n][j];
    return true;
}

// One item of the up (DOWN = false) or down product by one warp, stores included.
template <int XT, int W, bool DOWN, int NT>
__device__ __forceinline__ bool run_item(const MoeArgs &p, const MoeShared &S, const MoePipe &m, const MoeProduct &pr,
                                         const MoeUse &use, int ai, int tile)
{
    constexpr bool LO = DOWN || (W == W_MX && XT == OUT_F16);
    const int w = (int)(threadIdx.x >> 5) - 1, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int e = S.act[ai], first = S.first[ai], cnt = S.first[ai + 1] - first;
    const int r = tile * pr.step + 8 * w + g;                  // this lane's row in the lower half, within the expert
    MoeItem it;
    it.row = (uint32_t)(8 * w + g) * 128u;
    it.upper = (uint32_t)p.half_rows * 128u;
    it.ra = (int64_t)e * pr.rows + r;
    it.rb = it.ra + pr.half;
    float acc[NT][4] = {};
    if (!item_mma<W, NT, LO, DOWN && W == W_F16>(acc, m, pr, it, use)) return false;

    // acc[n][0..1]: the lower row, tokens n * 8 + 2 t4 and the next; acc[n][2..3]: the upper row
    const bool gated = pr.pairs;
    const int r2 = gated ? r : r + pr.half;
    const bool in1 = r < pr.limit, in2 = !gated && r2 < pr.limit;
    const float *bias = DOWN ? p.b2 : p.b1;
    const float bias1 = bias != nullptr && in1 ? bias[it.ra] : 0.0f;
    const float bias2 = bias != nullptr && (gated ? in1 : in2) ? bias[it.rb] : 0.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = n * 8 + 2 * t4 + j;
            if (c >= cnt) continue;
            const int64_t s = S.slot[first + c];
            float v1 = acc[n][j] + bias1, v2 = acc[n][2 + j] + bias2;
            if constexpr (DOWN) {
                if (in1) p.part[s * p.H + r] = v1;
                if (in2) p.part[s * p.H + r2] = v2;
            } else {
                auto put = [&](int row, float v) {
                    const int64_t at = s * p.Ip + token_at<W>(row);
                    const __nv_bfloat16 hi = __float2bfloat16_rn(v);
                    p.h_hi[at] = __bfloat16_as_ushort(hi);
                    p.h_lo[at] = __bfloat16_as_ushort(__float2bfloat16_rn(v - __bfloat162float(hi)));
                };
                v1 = act_mx(p.act, v1, p.alpha);
                if (gated) {
                    if (in1) put(r, v1 * v2);
                } else {
                    if (in1) put(r, v1);
                    if (in2) put(r2, act_mx(p.act, v2, p.alpha));
                }
            }
        }
    return true;
}

template <int XT, int W, bool DOWN>
__device__ __forceinline__ bool mma_phase(const MoeArgs &p, const MoeShared &S, const MoePipe &m, const MoeProduct &pr,
                                          MoeUse &use)
{
    const int n = S.nact * pr.tiles;
    for (int i = blockIdx.x; i < n; i += gridDim.x, use.w += (uint32_t)pr.stages, use.t += (uint32_t)pr.tstages) {
        const int ai = i / pr.tiles, tile = i - ai * pr.tiles, cnt = S.first[ai + 1] - S.first[ai];
        bool ok;
        if (cnt <= 8) ok = run_item<XT, W, DOWN, 1>(p, S, m, pr, use, ai, tile);
        else if (cnt <= 16 || MOE_GROUP<W> == 16) ok = run_item<XT, W, DOWN, 2>(p, S, m, pr, use, ai, tile);
        else ok = run_item<XT, W, DOWN, MOE_GROUP<W> / 8>(p, S, m, pr, use, ai, tile);
        if (!ok) return false;
    }
    return true;
}

// ------------------------------------------------------------- grid barriers --
// One thread: everything this CTA wrote before (its other threads ordered by a
// barrier) is visible to the CTAs that see the count.
__device__ __forceinline__ void grid_arrive(unsigned int *counter)
{
    __threadfence();
    atomicAdd(counter, 1u);
}

// One thread: waits for all CTAs of the grid, bounded.
__device__ __forceinline__ bool grid_wait(const Pipe &pp, unsigned int *counter)
{
    const uint64_t t0 = ptx::globaltimer();
    for (uint32_t it = 1;; ++it) {
        unsigned int c;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(c) : "l"(counter) : "memory");
        if (c >= gridDim.x) return true;
        if ((it & 31u) == 0 && (*pp.abort != 0u || ptx::globaltimer() - t0 > pp.wait_ns)) return false;
        if (it >= (1u << 30)) return false;
    }
}

// ------------------------------------------------------------------- kernel --
template <int W>
__device__ __forceinline__ bool produce(const CUtensorMap *map, const MoeArgs &p, const MoeShared &S, const MoePipe &m,
                                        const MoeProduct &pr, uint32_t &use, uint64_t pol)
{
    const int n = S.nact * pr.tiles;
    const uint32_t box = (uint32_t)p.half_rows * 128u;
    for (int i = blockIdx.x; i < n; i += gridDim.x) {
        const int ai = i / pr.tiles, tile = i - ai * pr.tiles, row = S.act[ai] * pr.rows + tile * pr.step;
        // the upper half of the last tile may have no rows (its products are not stored either)
        const bool both = pr.pairs || tile * pr.step + p.half_rows < pr.limit;
        for (int s = 0; s < pr.stages; ++s, ++use) {
            const uint32_t slot = use % MOE_STAGES, full = m.pp.full0 + 8 * slot, to = m.ring + slot * MOE_STAGE_BYTES;
            if (!mx_warp_wait(m.pp, m.pp.empty0 + 8 * slot, ((use / MOE_STAGES) & 1u) ^ 1u)) return false;
            elected_expect_tx(full, both ? 2u * box : box);
            elected_load_2d(to, map, full, s * 64, row, pol);
            if (both) elected_load_2d(to + box, map, full, s * 64, row + pr.half, pol);
        }
    }
    return true;
}

// The tokens of every item, in the weights' order: lane c copies token c's pieces.
template <int XT, int W, bool DOWN>
__device__ __forceinline__ bool produce_tokens(const MoeArgs &p, const MoeShared &S, const MoePipe &m, const MoeProduct &pr,
                                               uint32_t &use)
{
    using R = MoeRing<W>;
    constexpr bool LO = DOWN || (W == W_MX && XT == OUT_F16);
    const int lane = threadIdx.x & 31, n = S.nact * pr.tiles;
    for (int i = blockIdx.x; i < n; i += gridDim.x) {
        const int ai = i / pr.tiles, first = S.first[ai], cnt = S.first[ai + 1] - first;
        const int64_t slot_of = lane < cnt ? S.slot[first + lane] : 0;
        const int64_t from = DOWN ? slot_of * p.Ip : slot_of / p.top * p.Hp;
        const uint16_t *hi = (DOWN ? p.h_hi : p.x_hi) + from, *lo = (DOWN ? p.h_lo : p.x_lo) + from;
        for (int s = 0; s < pr.tstages; ++s, ++use) {
            const uint32_t slot = use % R::TSTAGES, full = m.tfull0 + 8 * slot;
            const uint32_t to = m.tokens + slot * R::TOKENS + (uint32_t)lane * MOE_RECORD;
            if (!mx_warp_wait(m.pp, m.tempty0 + 8 * slot, ((use / R::TSTAGES) & 1u) ^ 1u)) return false;
            elected_expect_tx(full, (uint32_t)cnt * MOE_TOKEN * (LO ? 2u : 1u));
            __syncwarp();
            if (lane < cnt) {
                bulk_load(to, hi + s * MOE_TOKEN_K, MOE_TOKEN, full);
                if constexpr (LO) bulk_load(to + MOE_TOKEN, lo + s * MOE_TOKEN_K, MOE_TOKEN, full);
            }
            __syncwarp();
        }
    }
    return true;
}

template <int XT, int W>
__global__ void __launch_bounds__(MOE_THREADS, 1)
    moe_experts_kernel(const __grid_constant__ CUtensorMap tm1, const __grid_constant__ CUtensorMap tm2, const MoeArgs p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    using R = MoeRing<W>;
    MoeShared &S = *reinterpret_cast<MoeShared *>(smem + R::BYTES);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    ptx::griddep_launch_dependents();
    const int active = p.half_rows / 8;                        // product warps that have rows
    MoePipe m;
    m.ring = ptx::smem_addr(smem);
    m.tokens = m.ring + R::OFF_TOKENS;
    m.pp.full0 = ptx::smem_addr(S.bar);
    m.pp.empty0 = m.pp.full0 + 8 * MOE_STAGES;
    m.tfull0 = m.pp.empty0 + 8 * MOE_STAGES;
    m.tempty0 = m.tfull0 + 8 * R::TSTAGES;
    m.pp.abort = reinterpret_cast<volatile uint32_t *>(&S.abort_flag);
    m.pp.status = p.status;
    m.pp.wait_ns = p.wait_ns;
    const bool aligned = (m.ring & 1023u) == 0;                // the swizzle counts rows from multiples of 1024 bytes
    if (threadIdx.x == 0) {
        if (!aligned) atomicOr(p.status, ST_SMEM_ALIGN);
        ptx::prefetch_tensormap(&tm1);
        ptx::prefetch_tensormap(&tm2);
        for (int s = 0; s < MOE_STAGES; ++s) {
            ptx::mbar_init(m.pp.full0 + 8 * s, 1);
            ptx::mbar_init(m.pp.empty0 + 8 * s, (uint32_t)active);
        }
        for (int s = 0; s < R::TSTAGES; ++s) {
            ptx::mbar_init(m.tfull0 + 8 * s, 1);
            ptx::mbar_init(m.tempty0 + 8 * s, (uint32_t)active);
        }
        S.abort_flag = aligned ? 0 : 1;
        ptx::fence_mbar_init();
    }
    ptx::griddep_wait();                                       // the router's logits
    // All logits where the weights will stand, the lists' masks where the tokens will.
    static_assert(MOE_MAX_T * MOE_MAX_E * 4 <= R::OFF_TOKENS, "all logits");
    static_assert(MOE_MAX_E * MOE_MAX_T * MOE_MAX_K / 8 <= R::TSTAGES * R::TOKENS, "a bit for each expert and slot");
    float *logits = reinterpret_cast<float *>(smem);
#pragma unroll 8
    for (int i = threadIdx.x; i < p.T * p.E; i += MOE_THREADS) logits[i] = __ldcg(p.logits + i);
    ptx::cta_sync();
    constexpr int WARPS = MOE_THREADS / 32;
    for (int t = warp; t < p.T; t += 4 * WARPS) {
        const int left = (p.T - t + WARPS - 1) / WARPS;        // tokens of this warp from t on
        const bool write = blockIdx.x == 0;
        if (left == 1) choose_experts<1>(p, S, logits, t, WARPS, lane, write);
        else if (left == 2) choose_experts<2>(p, S, logits, t, WARPS, lane, write);
        else if (left == 3) choose_experts<3>(p, S, logits, t, WARPS, lane, write);
        else choose_experts<4>(p, S, logits, t, WARPS, lane, write);
    }
    ptx::cta_sync();
    build_lists<MOE_GROUP<W>>(p, S, reinterpret_cast<uint32_t *>(smem + R::OFF_TOKENS));
    ptx::fence_proxy_async_smem();                             // before the copies that overwrite both
    ptx::cta_sync();

    const int hr = p.half_rows, ks = R::K, kt = MOE_TOKEN_K;
    const int step1 = p.gated ? hr : 2 * hr, step2 = 2 * hr;
    const MoeProduct up = {p.H, (p.H + ks - 1) / ks, (p.H + kt - 1) / kt, (p.I + step1 - 1) / step1, p.R1, p.gated ? p.I : hr, step1, p.I,
                           static_cast<const uint8_t *>(p.s1), (int64_t)p.E * p.R1, (p.H + 127) / 128, p.gated != 0};
    const MoeProduct down = {p.I, (p.I + ks - 1) / ks, (p.I + kt - 1) / kt, (p.H + step2 - 1) / step2, p.H, hr, step2, p.H,
                             static_cast<const uint8_t *>(p.s2), (int64_t)p.E * p.H, (p.I + 127) / 128, false};
    bool ok = aligned;
    if (warp == 0) {
        uint32_t use = 0;
        const uint64_t pol = ptx::createpolicy_evict_first();  // weights are read once
        ok = ok && produce<W>(&tm1, p, S, m, up, use, pol) && produce<W>(&tm2, p, S, m, down, use, pol);
        if (!ok && lane == 0) pipe_fail(m.pp);
        // every copy has landed before the CTA exits
        for (uint32_t u = use > (uint32_t)MOE_STAGES ? use - MOE_STAGES : 0; u < use; ++u)
            ptx::mbar_wait_bounded(m.pp.full0 + 8 * (u % MOE_STAGES), (u / MOE_STAGES) & 1u, DRAIN_NS, nullptr);
    } else if (warp == 1 + MOE_MMA_WARPS) {
        uint32_t use = 0;
        ok = ok && produce_tokens<XT, W, false>(p, S, m, up, use);
        // every h is written before any is read
        if (ok) ok = __all_sync(0xffffffffu, lane != 0 || grid_wait(m.pp, p.counters)) != 0;
        fence_proxy_async_all();
        ok = ok && produce_tokens<XT, W, true>(p, S, m, down, use);
        if (!ok && lane == 0) pipe_fail(m.pp);
        for (uint32_t u = use > (uint32_t)R::TSTAGES ? use - R::TSTAGES : 0; u < use; ++u)
            ptx::mbar_wait_bounded(m.tfull0 + 8 * (u % R::TSTAGES), (u / R::TSTAGES) & 1u, DRAIN_NS, nullptr);
    } else {
        MoeUse use = {0, 0};
        if (ok && warp <= active) ok = mma_phase<XT, W, false>(p, S, m, up, use);
        // this CTA's part of h is written
        fence_proxy_async_all();
        __syncwarp();
        asm volatile("barrier.sync 1, %0;" ::"n"(32 * MOE_MMA_WARPS) : "memory");
        if (ok && threadIdx.x == 32) grid_arrive(p.counters);
        __syncwarp();
        if (ok && warp <= active) ok = mma_phase<XT, W, true>(p, S, m, down, use);
        if (!ok && lane == 0) pipe_fail(m.pp);
    }
    __syncwarp();
    // every o is written before y is summed
    ptx::cta_sync();
    if (threadIdx.x == 0) {
        S.go = 0;
        if (*m.pp.abort == 0u) {
            grid_arrive(p.counters + 1);
            S.go = grid_wait(m.pp, p.counters + 1) ? 1 : 0;
            if (S.go == 0) pipe_fail(m.pp);
        }
    }
    ptx::cta_sync();
    if (S.go == 0) return;
    for (int64_t i = (int64_t)blockIdx.x * MOE_THREADS + threadIdx.x; i < (int64_t)p.T * p.H;
         i += (int64_t)gridDim.x * MOE_THREADS) {
        const int t = (int)(i / p.H), r = (int)(i - (int64_t)t * p.H);
        float y = 0.0f;
        for (int j = 0; j < p.top; ++j)
            y = fmaf(S.probs[t * p.top + j], __ldcg(p.part + (int64_t)(t * p.top + j) * p.H + r), y);
        if constexpr (XT == OUT_BF16) static_cast<__nv_bfloat16 *>(p.y)[i] = __float2bfloat16_rn(y);
        else static_cast<__half *>(p.y)[i] = __float2half_rn(y);
    }
}

template <int W>
constexpr int MOE_SMEM = MoeRing<W>::BYTES + (int)sizeof(MoeShared);
static_assert(MOE_SMEM<W_BF16> <= 232448 && MOE_SMEM<W_MX> <= 232448, "shared memory budget");

template <int XT, int W>
static cudaError_t launch_experts(const MoeLaunch &L, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)L.grid);
    cfg.blockDim = dim3(MOE_THREADS);
    cfg.dynamicSmemBytes = MOE_SMEM<W>;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;               // the CTAs wait for one another
    attr[0].val.cooperative = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, moe_experts_kernel<XT, W>, L.tm1, L.tm2, L.args);
}

template <int XT, int W>
static cudaError_t setup_experts()
{
    return cudaFuncSetAttribute(moe_experts_kernel<XT, W>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                MOE_SMEM<W>);
}

cudaError_t setup_moe_kernels()
{
    cudaError_t e = setup_experts<OUT_BF16, W_BF16>();
    if (e == cudaSuccess) e = setup_experts<OUT_F16, W_F16>();
    if (e == cudaSuccess) e = setup_experts<OUT_BF16, W_MX>();
    if (e == cudaSuccess) e = setup_experts<OUT_F16, W_MX>();
    return e;
}

cudaError_t launch_moe(const MoeLaunch &L, cudaStream_t stream)
{
    const MoeArgs &a = L.args;
    const int groups = (a.T + 7) / 8;
    const dim3 grid((unsigned)(a.E * groups + a.T * ((a.Hp + 1023) / 1024))), block(MOE_ROUTER_THREADS);
    auto router = a.w_type == W_MX ? (L.x_out == OUT_BF16 ? moe_router_kernel<OUT_BF16, W_MX> : moe_router_kernel<OUT_F16, W_MX>)
                                   : (L.x_out == OUT_BF16 ? moe_router_kernel<OUT_BF16, W_BF16>
                                                          : moe_router_kernel<OUT_F16, W_F16>);
    const cudaError_t e = launch_k(router, grid, block, 0, stream, a, groups);
    if (e != cudaSuccess) return e;
    if (a.w_type == W_MX)
        return L.x_out == OUT_BF16 ? launch_experts<OUT_BF16, W_MX>(L, stream) : launch_experts<OUT_F16, W_MX>(L, stream);
    return L.x_out == OUT_BF16 ? launch_experts<OUT_BF16, W_BF16>(L, stream) : launch_experts<OUT_F16, W_F16>(L, stream);
}

}  // namespace mmact
