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
// with a contiguous share of the items (16 weight rows x all of K of one expert;
// for a gated layer 8 gate rows and the 8 up rows that go with them):
//
//   warp 0       producer: TMA boxes of 8 rows x 512 bytes (MXFP4: 256 bytes and
//                the scales that belong to them) into a ring of stages.  It runs
//                ahead over items and over the grid barrier: weights of the down
//                product are on their way while the last h is being finished.
//   warps 1..8   products: the stages go round the eight warps; on
//                mma.sync.m16n8k16 with the weights as the 16-row operand and
//                eight tokens to its columns; which K a lane holds does not
//                matter to a sum over K as long as both operands agree, so the
//                fragments are 16-byte loads in memory order
//   warps 9..11  sums over the eight warps, bias, activation, stores
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
constexpr int MOE_MMA_WARPS = 8, MOE_EPI_WARPS = 3;
constexpr int MOE_THREADS = 32 * (1 + MOE_MMA_WARPS + MOE_EPI_WARPS);
constexpr int MOE_EPI_THREADS = 32 * MOE_EPI_WARPS;
constexpr int MOE_GROUP = 32;                                  // tokens of one expert that share a read of its weights

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

// Where element k of a token's row stands in the bf16 arrays that MXFP4 weights
// multiply: within each group of eight the order 0 4 1 5 2 6 3 7, because a
// 32-bit word of eight codes yields its values as the pairs (i, i + 4).
__device__ __forceinline__ int mx_order(int k)
{
    return (k & ~7) | ((k & 3) << 1) | ((k >> 2) & 1);
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

__device__ __forceinline__ void elected_load_3d(uint32_t dst, const CUtensorMap *m, uint32_t bar, int x, int y, int z)
{
    asm volatile(MMACT_ELECTED
                 "@q cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

#undef MMACT_ELECTED

// ------------------------------------------------------------------- router --
// One CTA for an expert and eight tokens: four warps share K.  The CTAs past
// those prepare what the experts kernel needs: its counters, and for MXFP4
// weights x in bf16 in the codes' order and the zeros past I of h.
constexpr int MOE_ROUTER_THREADS = 128;

template <int XT>
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
            float2 g[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) g[j] = unpack2<XT>(bw[j]);
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                if (t >= n) break;
                const uint4 a = __ldg(reinterpret_cast<const uint4 *>(xs + (int64_t)(t0 + t) * p.H + k));
                const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
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
            if (t >= n) break;
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
    const int t = blockIdx.x - p.E * token_groups;
    if (t == 0 && threadIdx.x < 2) p.counters[threadIdx.x] = 0;
    if (p.w_type == W_MX) {
        const uint16_t *x = xs + (int64_t)t * p.H;
        for (int k = threadIdx.x; k < p.Hp; k += MOE_ROUTER_THREADS) {
            float v = 0.0f;
            if (k < p.H) {
                if constexpr (XT == OUT_BF16) v = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(x)[k]);
                else v = __half2float(reinterpret_cast<const __half *>(x)[k]);
            }
            const __nv_bfloat16 hi = __float2bfloat16_rn(v);
            const int64_t at = (int64_t)t * p.Hp + mx_order(k);
            p.x_hi[at] = hi;
            if constexpr (XT == OUT_F16) p.x_lo[at] = __float2bfloat16_rn(v - __bfloat162float(hi));
        }
        const int pad = p.Ip - p.I;
        for (int i = threadIdx.x; i < pad * p.top; i += MOE_ROUTER_THREADS) {
            const int64_t at = ((int64_t)t * p.top + i / pad) * p.Ip + p.I + i % pad;
            p.h_hi[at] = p.h_lo[at] = __float2bfloat16_rn(0.0f);
        }
    }
}

// ------------------------------------------------------------ choice of experts --
// Shared memory of the experts kernel beside the ring.
struct MoeShared {
    float red[2][MOE_MMA_WARPS][16][MOE_GROUP];    // partial sums of two items
    float probs[MOE_MAX_T * MOE_MAX_K];
    short choice[MOE_MAX_T * MOE_MAX_K];           // slot t * k + j -> expert
    short slot[MOE_MAX_T * MOE_MAX_K];             // slots by expert
    short count[MOE_MAX_E];
    short act[MOE_MAX_E + 32];                     // groups of at most 32 tokens of one expert, by expert:
    short first[MOE_MAX_E + 33];                   // the expert and the first entry of slot[]
    int nact;
    int abort_flag, go;
    uint64_t bar[2 * 24 + 4];
};

// Top k of one token by one warp: each round the largest (key, lowest index) of
// those left; then the softmax weights.  The token's logits are kept in shared
// memory where the partial sums will be (`row`: MOE_MAX_E floats of this warp).
__device__ __forceinline__ void choose_experts(const MoeArgs &p, MoeShared &S, float *row, int t, int lane, bool write)
{
    __syncwarp();
    for (int e = lane; e < p.E; e += 32) row[e] = __ldcg(p.logits + (int64_t)t * p.E + e);
    __syncwarp();
    uint32_t taken = 0;                                        // bit i: this lane's logit i * 32 + lane is chosen
    float peak = 0.0f, w = 0.0f, total = 0.0f;
    for (int j = 0; j < p.top; ++j) {
        uint64_t best = 0;
        for (int e = lane, i = 0; e < p.E; e += 32, ++i) {
            if ((taken >> i) & 1u) continue;
            const uint64_t key = ((uint64_t)logit_key(row[e]) << 32) | (0xffffffffu - (uint32_t)e);
            best = key > best ? key : best;
        }
        __syncwarp();
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const uint64_t other = __shfl_xor_sync(0xffffffffu, best, o);
            best = other > best ? other : best;
        }
        const int e = (int)(0xffffffffu - (uint32_t)best);
        float v = row[e];
        if ((e & 31) == lane) taken |= 1u << (e >> 5);
        if (j == 0) peak = v;
        v = expf(v - peak);
        total += v;
        if (j == lane) w = v;
        if (lane == 0) {
            S.choice[t * p.top + j] = (short)e;
            if (write) p.experts[t * p.top + j] = e;
        }
    }
    if (!p.normalize) {
        total = 0.0f;
        for (int e = lane; e < p.E; e += 32) total += expf(row[e] - peak);
        __syncwarp();
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    if (lane < p.top) {
        w /= total;
        S.probs[t * p.top + lane] = w;
        if (write) p.probs[t * p.top + lane] = w;
    }
}

// The slots of each expert, in groups of at most 32, built by every CTA.
__device__ __forceinline__ void build_lists(const MoeArgs &p, MoeShared &S)
{
    const int tid = threadIdx.x, n_slots = p.T * p.top;
    for (int e = tid; e < p.E; e += MOE_THREADS) {
        int c = 0;
        for (int s = 0; s < n_slots; ++s) c += S.choice[s] == e;
        S.count[e] = (short)c;
    }
    ptx::cta_sync();
    if (tid < 32) {                                            // 32 experts at a time: running sums over the warp
        int n = 0, at = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + tid, c = e < p.E ? S.count[e] : 0, groups = (c + MOE_GROUP - 1) / MOE_GROUP;
            int sum = c, gsum = groups;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, sum, o), gup = __shfl_up_sync(0xffffffffu, gsum, o);
                if (tid >= o) sum += up, gsum += gup;
            }
            for (int g = 0; g < groups; ++g) {
                S.act[n + gsum - groups + g] = (short)e;
                S.first[n + gsum - groups + g] = (short)(at + sum - c + g * MOE_GROUP);
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
    for (int a = tid; a < S.nact; a += MOE_THREADS) {
        const int e = S.act[a];
        if (a > 0 && S.act[a - 1] == e) continue;              // the first group fills the others' entries too
        int at = S.first[a];
        for (int s = 0; s < n_slots; ++s)
            if (S.choice[s] == e) S.slot[at++] = (short)s;
    }
    ptx::cta_sync();
}

// ----------------------------------------------------------------- products --
// A ring stage: 2 boxes of 8 rows, ROW_BYTES of each row; MXFP4: and 2 boxes of
// scales, 4 tiles x 8 rows x 16 bytes.
template <int W>
struct MoeStage {
    static constexpr int KS = W == W_MX ? 512 : 256;           // K of a stage
    static constexpr int ROW_BYTES = W == W_MX ? MOE_ROW_BYTES_MX : MOE_ROW_BYTES;
    static constexpr int BOX = 8 * ROW_BYTES;
    static constexpr int BYTES = 2 * BOX + (W == W_MX ? 1024 : 0);
    // About 128 KB: twice what has to be in flight; the rest of the SM's memory caches the tokens.  A
    // multiple of the product warps: slot i always belongs to warp i % 8.  (A wait for a phase only tells
    // the phase from the one before it, so the warp that waits has to have seen that one end itself.)
    static constexpr int SLOTS = W == W_MX ? 24 : 16;
    static constexpr int SMEM = SLOTS * BYTES + 1024 + (int)sizeof(MoeShared);
    static_assert(2 * SLOTS <= 48 && SLOTS % MOE_MMA_WARPS == 0, "barriers");
};

// One product of the layer as the roles see it.
struct MoeProduct {
    int K, stages;                   // stages of one item
    int tiles;                       // items of one group of tokens
    int rows;                        // rows of one expert's matrix
    int half;                        // row distance between an item's two boxes
    int step;                        // rows from one item to the next
    int limit;                       // rows that the items count over: I or H
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


__device__ __forceinline__ uint4 ld_token(const uint16_t *p, int64_t k, bool have)
{
    return have && p != nullptr ? *reinterpret_cast<const uint4 *>(p + k) : make_uint4(0, 0, 0, 0);
}

// acc += one stage's 16 rows x this lane's token columns, K from k0.  xh / xl:
// this lane's token rows (hi, lo) for each group of eight tokens, null where there
// is no token.  LO: multiply the lo half too.  SPLITW: fp16 weights as two bf16
// halves.  `wait` is called once, after the first tokens are on their way.
template <int W, int NT, bool LO, bool SPLITW, typename Wait>
__device__ __forceinline__ bool stage_mma(float (&acc)[NT][4], uint32_t slot, const uint16_t *const (&xh)[NT],
                                          const uint16_t *const (&xl)[NT], int k0, int K, uint32_t sa_off,
                                          uint32_t sb_off, Wait wait)
{
    const int lane = threadIdx.x & 31, t4 = lane & 3, g = lane >> 2;
    using St = MoeStage<W>;
    const uint32_t row = slot + (uint32_t)g * St::ROW_BYTES + (uint32_t)t4 * 16u;
    if constexpr (W == W_MX) {
        // units of 128 K: 16 bytes = one block of 32 codes to a lane
        constexpr int WB = NT == 1 ? 4 : (NT == 2 ? 2 : 1);    // words of codes whose tokens are loaded together
#pragma unroll 1
        for (int u = 0; u < 4; ++u) {
            const int k = k0 + u * 128 + t4 * 32;
            if (k0 + u * 128 >= K) break;
            const bool have = k < K;                           // token rows are zero up to a multiple of 32
            uint4 h[WB][NT], l[WB][NT];
#pragma unroll
            for (int w = 0; w < WB; ++w)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    h[w][n] = ld_token(xh[n], k + w * 8, have);
                    if constexpr (LO) l[w][n] = ld_token(xl[n], k + w * 8, have);
                }
            if (u == 0 && !wait()) return false;
            const uint4 a = ptx::ld_shared_v4(row + u * 64u), b = ptx::ld_shared_v4(row + St::BOX + u * 64u);
            const uint32_t so = slot + 2 * St::BOX + u * 128u + (uint32_t)g * 16u + (uint32_t)t4;
            uint32_t sa, sb;
            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(sa) : "r"(so + sa_off));
            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(sb) : "r"(so + 512u + sb_off));
            uint32_t ra, rb;
            const uint32_t ma = mx_factor(sa, ra), mb = mx_factor(sb, rb);
            const bool big = __any_sync(0xffffffffu, sa > 128u || sb > 128u);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                if (w > 0 && w % WB == 0) {
#pragma unroll
                    for (int i = 0; i < WB; ++i)
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            h[i][n] = ld_token(xh[n], k + (w + i) * 8, have);
                            if constexpr (LO) l[i][n] = ld_token(xl[n], k + (w + i) * 8, have);
                        }
                }
                uint32_t va[4], vb[4];
                mx_word_bf16(word_of(a, w), ma, va);
                mx_word_bf16(word_of(b, w), mb, vb);
                if (big) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        va[i] = mul_bf16x2(va[i], ra);
                        vb[i] = mul_bf16x2(vb[i], rb);
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint4 x = h[w % WB][n];
                    mma_16816<true>(acc[n], va[0], vb[0], va[1], vb[1], x.x, x.y);
                    mma_16816<true>(acc[n], va[2], vb[2], va[3], vb[3], x.z, x.w);
                    if constexpr (LO) {
                        const uint4 y = l[w % WB][n];
                        mma_16816<true>(acc[n], va[0], vb[0], va[1], vb[1], y.x, y.y);
                        mma_16816<true>(acc[n], va[2], vb[2], va[3], vb[3], y.z, y.w);
                    }
                }
            }
        }
    } else {
        // units of 32 K: 16 bytes to a lane, two instructions
        constexpr bool BF = W == W_BF16 || SPLITW;
        constexpr int UB = NT == 1 ? 4 : (NT == 2 ? 2 : 1);
#pragma unroll 1
        for (int u0 = 0; u0 < 8; u0 += UB) {
            if (k0 + u0 * 32 >= K) break;
            uint4 h[UB][NT], l[UB][NT];
#pragma unroll
            for (int u = 0; u < UB; ++u)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int k = k0 + (u0 + u) * 32 + t4 * 8;
                    h[u][n] = ld_token(xh[n], k, k < K);
                    if constexpr (LO) l[u][n] = ld_token(xl[n], k, k < K);
                }
            if (u0 == 0 && !wait()) return false;
#pragma unroll
            for (int u = 0; u < UB; ++u) {
                const uint4 fa = ptx::ld_shared_v4(row + (u0 + u) * 64u);
                const uint4 fb = ptx::ld_shared_v4(row + St::BOX + (u0 + u) * 64u);
                uint32_t a[4] = {fa.x, fa.y, fa.z, fa.w}, b[4] = {fb.x, fb.y, fb.z, fb.w};
                uint32_t al[4], bl[4];
                if constexpr (SPLITW) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 va = unpack2<OUT_F16>(a[i]), vb = unpack2<OUT_F16>(b[i]);
                        split_pair(va.x, va.y, a[i], al[i]);
                        split_pair(vb.x, vb.y, b[i], bl[i]);
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint4 x = h[u][n];
                    mma_16816<BF>(acc[n], a[0], b[0], a[1], b[1], x.x, x.y);
                    mma_16816<BF>(acc[n], a[2], b[2], a[3], b[3], x.z, x.w);
                    if constexpr (LO) {
                        const uint4 y = l[u][n];
                        mma_16816<BF>(acc[n], a[0], b[0], a[1], b[1], y.x, y.y);
                        mma_16816<BF>(acc[n], a[2], b[2], a[3], b[3], y.z, y.w);
                    }
                    if constexpr (SPLITW) {
                        mma_16816<BF>(acc[n], al[0], bl[0], al[1], bl[1], x.x, x.y);
                        mma_16816<BF>(acc[n], al[2], bl[2], al[3], bl[3], x.z, x.w);
                    }
                }
            }
        }
    }
    return true;
}

// The ring and the item buffers of one CTA.
struct MoePipe {
    Pipe pp;
    uint32_t ring;                   // shared address of the stages
    uint32_t rfull, rempty;          // partial sums: written / read, two buffers each
};

// One warp's part of an item: its stages, then its partial sums to red[buf].
template <int W, int NT, bool LO, bool SPLITW>
__device__ __forceinline__ bool item_mma(MoeShared &S, const MoePipe &m, const MoeProduct &pr, uint32_t base, uint32_t item,
                                         const uint16_t *const (&xh)[NT], const uint16_t *const (&xl)[NT],
                                         uint32_t sa_off, uint32_t sb_off)
{
    using St = MoeStage<W>;
    const int w = (int)(threadIdx.x >> 5) - 1, lane = threadIdx.x & 31, t4 = lane & 3, g = lane >> 2;
    float acc[NT][4] = {};
    for (int s = (int)(((uint32_t)w - base) % MOE_MMA_WARPS); s < pr.stages; s += MOE_MMA_WARPS) {
        const uint32_t use = base + (uint32_t)s, slot = use % St::SLOTS, phase = (use / St::SLOTS) & 1u;
        const bool ok = stage_mma<W, NT, LO, SPLITW>(
            acc, m.ring + slot * St::BYTES, xh, xl, s * St::KS, pr.K, sa_off, sb_off,
            [&] { return mx_warp_wait(m.pp, m.pp.full0 + 8 * slot, phase); });
        if (!ok) return false;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(m.pp.empty0 + 8 * slot);
    }
    const uint32_t buf = item & 1u;
    if (!mx_warp_wait(m.pp, m.rempty + 8 * buf, ((item >> 1) & 1u) ^ 1u)) return false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        *reinterpret_cast<float2 *>(&S.red[buf][w][g][n * 8 + 2 * t4]) = make_float2(acc[n][0], acc[n][1]);
        *reinterpret_cast<float2 *>(&S.red[buf][w][g + 8][n * 8 + 2 * t4]) = make_float2(acc[n][2], acc[n][3]);
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(m.rfull + 8 * buf);
    return true;
}

// This lane's token rows: x by token, h by slot.
template <int XT, int W, bool DOWN, int NT>
__device__ __forceinline__ bool item_product(const MoeArgs &p, MoeShared &S, const MoePipe &m, const MoeProduct &pr,
                                             uint32_t base, uint32_t item, int ai, int row0)
{
    const int g = (threadIdx.x & 31) >> 2, first = S.first[ai], cnt = S.first[ai + 1] - first;
    const uint16_t *xh[NT], *xl[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        xh[n] = xl[n] = nullptr;
        const int c = n * 8 + g;
        if (c >= cnt) continue;
        const int64_t s = S.slot[first + c];
        if constexpr (DOWN) {
            xh[n] = reinterpret_cast<const uint16_t *>(p.h_hi) + s * p.Ip;
            xl[n] = reinterpret_cast<const uint16_t *>(p.h_lo) + s * p.Ip;
        } else if constexpr (W == W_MX) {
            xh[n] = reinterpret_cast<const uint16_t *>(p.x_hi) + s / p.top * p.Hp;
            xl[n] = reinterpret_cast<const uint16_t *>(p.x_lo) + s / p.top * p.Hp;
        } else {
            xh[n] = static_cast<const uint16_t *>(p.x) + s / p.top * p.H;
        }
    }
    // the byte of a row's scale word: its place among the four 32-row groups of a tile
    const uint32_t sa = (uint32_t)(row0 >> 5 & 3) * 4u, sb = (uint32_t)((row0 + pr.half) >> 5 & 3) * 4u;
    constexpr bool LO = DOWN || (W == W_MX && XT == OUT_F16);
    return item_mma<W, NT, LO, DOWN && W == W_F16>(S, m, pr, base, item, xh, xl, sa, sb);
}

template <int XT, int W, bool DOWN>
__device__ __forceinline__ bool mma_phase(const MoeArgs &p, MoeShared &S, const MoePipe &m, const MoeProduct &pr,
                                          uint32_t &base, uint32_t &item)
{
    const int n = S.nact * pr.tiles;
    const int i0 = (int)((int64_t)n * blockIdx.x / gridDim.x), i1 = (int)((int64_t)n * (blockIdx.x + 1) / gridDim.x);
    for (int it = i0; it < i1; ++it, ++item, base += (uint32_t)pr.stages) {
        const int ai = it / pr.tiles, cnt = S.first[ai + 1] - S.first[ai];
        const int row0 = S.act[ai] * pr.rows + (it - ai * pr.tiles) * pr.step;
        const bool ok = cnt <= 8    ? item_product<XT, W, DOWN, 1>(p, S, m, pr, base, item, ai, row0)
                        : cnt <= 16 ? item_product<XT, W, DOWN, 2>(p, S, m, pr, base, item, ai, row0)
                                    : item_product<XT, W, DOWN, 4>(p, S, m, pr, base, item, ai, row0);
        if (!ok) return false;
    }
    return true;
}

// ----------------------------------------------------------------- epilogue --
// Barrier of the epilogue's threads, which may arrive one lane after another.
__device__ __forceinline__ void epilogue_sync()
{
    asm volatile("barrier.sync 1, %0;" ::"n"(MOE_EPI_THREADS) : "memory");
}

__device__ __forceinline__ float red_sum(const MoeShared &S, uint32_t buf, int row, int col)
{
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < MOE_MMA_WARPS; ++w) s += S.red[buf][w][row][col];
    return s;
}

template <int W, bool DOWN>
__device__ __forceinline__ bool epilogue_phase(const MoeArgs &p, MoeShared &S, const MoePipe &m, const MoeProduct &pr,
                                               uint32_t &item)
{
    const int tid = (int)threadIdx.x - 32 * (1 + MOE_MMA_WARPS), lane = threadIdx.x & 31;
    const int n = S.nact * pr.tiles;
    const int i0 = (int)((int64_t)n * blockIdx.x / gridDim.x), i1 = (int)((int64_t)n * (blockIdx.x + 1) / gridDim.x);
    const int step = pr.step, shift = step == 8 ? 3 : 4;
    for (int it = i0; it < i1; ++it, ++item) {
        const int ai = it / pr.tiles, first = S.first[ai], cnt = S.first[ai + 1] - first;
        const int e = S.act[ai], r0 = (it - ai * pr.tiles) * step;
        const uint32_t buf = item & 1u;
        if (!mx_warp_wait(m.pp, m.rfull + 8 * buf, (item >> 1) & 1u)) return false;
        for (int i = tid; i < cnt << shift; i += MOE_EPI_THREADS) {
            const int row = i & (step - 1), c = i >> shift, r = r0 + row;
            if (r >= pr.limit) continue;
            const int64_t s = S.slot[first + c];
            float v = red_sum(S, buf, row, c);
            if constexpr (DOWN) {
                if (p.b2 != nullptr) v += p.b2[(int64_t)e * p.H + r];
                p.part[s * p.H + r] = v;
            } else {
                if (p.b1 != nullptr) v += p.b1[(int64_t)e * p.R1 + r];
                v = act_mx(p.act, v, p.alpha);
                if (p.gated) {
                    float u = red_sum(S, buf, 8 + row, c);
                    if (p.b1 != nullptr) u += p.b1[(int64_t)e * p.R1 + p.I + r];
                    v *= u;
                }
                const int64_t at = s * p.Ip + (W == W_MX ? mx_order(r) : r);
                const __nv_bfloat16 hi = __float2bfloat16_rn(v);
                p.h_hi[at] = hi;
                p.h_lo[at] = __float2bfloat16_rn(v - __bfloat162float(hi));
            }
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(m.rempty + 8 * buf);
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
__device__ __forceinline__ bool produce(const CUtensorMap *w, const CUtensorMap *sc, MoeShared &S, const MoePipe &m,
                                        const MoeProduct &pr, uint32_t &use, uint64_t pol)
{
    using St = MoeStage<W>;
    const int n = S.nact * pr.tiles;
    const int i0 = (int)((int64_t)n * blockIdx.x / gridDim.x), i1 = (int)((int64_t)n * (blockIdx.x + 1) / gridDim.x);
    for (int it = i0; it < i1; ++it) {
        const int ai = it / pr.tiles, row = S.act[ai] * pr.rows + (it - ai * pr.tiles) * pr.step;
        for (int s = 0; s < pr.stages; ++s, ++use) {
            const uint32_t slot = use % St::SLOTS, full = m.pp.full0 + 8 * slot, to = m.ring + slot * St::BYTES;
            if (!mx_warp_wait(m.pp, m.pp.empty0 + 8 * slot, ((use / St::SLOTS) & 1u) ^ 1u)) return false;
            elected_expect_tx(full, (uint32_t)St::BYTES);
            elected_load_2d(to, w, full, s * (St::ROW_BYTES / 2), row, pol);
            elected_load_2d(to + St::BOX, w, full, s * (St::ROW_BYTES / 2), row + pr.half, pol);
            if constexpr (W == W_MX) {
                const int other = row + pr.half;
                elected_load_3d(to + 2 * St::BOX, sc, full, (row & 31) * 4, s * 4, row >> 7);
                elected_load_3d(to + 2 * St::BOX + 512, sc, full, (other & 31) * 4, s * 4, other >> 7);
            }
        }
    }
    return true;
}

template <int XT, int W>
__global__ void __launch_bounds__(MOE_THREADS, 1)
    moe_experts_kernel(const __grid_constant__ CUtensorMap tm1, const __grid_constant__ CUtensorMap ts1,
                       const __grid_constant__ CUtensorMap tm2, const __grid_constant__ CUtensorMap ts2, const MoeArgs p)
{
    using St = MoeStage<W>;
    extern __shared__ __align__(1024) uint8_t smem[];
    MoeShared &S = *reinterpret_cast<MoeShared *>(smem + St::SLOTS * St::BYTES);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    MoePipe m;
    m.ring = ptx::smem_addr(smem);
    m.pp.full0 = ptx::smem_addr(S.bar);
    m.pp.empty0 = m.pp.full0 + 8 * St::SLOTS;
    m.rfull = m.pp.empty0 + 8 * St::SLOTS;
    m.rempty = m.rfull + 16;
    m.pp.abort = reinterpret_cast<volatile uint32_t *>(&S.abort_flag);
    m.pp.status = p.status;
    m.pp.wait_ns = p.wait_ns;
    if (threadIdx.x == 0) {
        ptx::prefetch_tensormap(&tm1);
        ptx::prefetch_tensormap(&tm2);
        for (int s = 0; s < 2 * St::SLOTS; ++s) ptx::mbar_init(m.pp.full0 + 8 * s, 1);
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(m.rfull + 8 * b, MOE_MMA_WARPS);
            ptx::mbar_init(m.rempty + 8 * b, MOE_EPI_WARPS);
        }
        S.abort_flag = 0;
        ptx::fence_mbar_init();
    }
    static_assert(MOE_THREADS / 32 * MOE_MAX_E * 4 <= sizeof(S.red) && MOE_MAX_E <= 32 * 32, "a row of logits to a warp");
    for (int t = warp; t < p.T; t += MOE_THREADS / 32)
        choose_experts(p, S, &S.red[0][0][0][0] + warp * MOE_MAX_E, t, lane, blockIdx.x == 0);
    ptx::cta_sync();
    build_lists(p, S);

    const int per = p.gated ? 8 : 16;
    const MoeProduct up = {p.H, (p.H + St::KS - 1) / St::KS, (p.I + per - 1) / per, p.R1, p.gated ? p.I : 8, per, p.I};
    const MoeProduct down = {p.I, (p.I + St::KS - 1) / St::KS, (p.H + 15) / 16, p.H, 8, 16, p.H};
    bool ok = true;
    if (warp == 0) {
        uint32_t use = 0;
        const uint64_t pol = ptx::createpolicy_evict_first();  // weights are read once
        ok = produce<W>(&tm1, &ts1, S, m, up, use, pol) && produce<W>(&tm2, &ts2, S, m, down, use, pol);
        if (!ok && lane == 0) pipe_fail(m.pp);
        // every copy has landed before the CTA exits
        for (uint32_t u = use > (uint32_t)St::SLOTS ? use - St::SLOTS : 0; u < use; ++u)
            ptx::mbar_wait_bounded(m.pp.full0 + 8 * (u % St::SLOTS), (u / St::SLOTS) & 1u, DRAIN_NS, nullptr);
    } else if (warp <= MOE_MMA_WARPS) {
        uint32_t base = 0, item = 0;
        ok = mma_phase<XT, W, false>(p, S, m, up, base, item);
        // every h is written before any is read
        if (ok) ok = __all_sync(0xffffffffu, lane != 0 || grid_wait(m.pp, p.counters)) != 0;
        if (ok) ok = mma_phase<XT, W, true>(p, S, m, down, base, item);
        if (!ok && lane == 0) pipe_fail(m.pp);
    } else {
        uint32_t item = 0;
        ok = epilogue_phase<W, false>(p, S, m, up, item);
        if (ok) {
            epilogue_sync();
            if (threadIdx.x == 32 * (1 + MOE_MMA_WARPS)) grid_arrive(p.counters);
            ok = epilogue_phase<W, true>(p, S, m, down, item);
        }
        if (!ok && lane == 0) pipe_fail(m.pp);
    }
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

template <int XT, int W>
static cudaError_t launch_experts(const MoeLaunch &L, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)L.grid);
    cfg.blockDim = dim3(MOE_THREADS);
    cfg.dynamicSmemBytes = MoeStage<W>::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;               // the CTAs wait for one another
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, moe_experts_kernel<XT, W>, L.tm1, L.ts1, L.tm2, L.ts2, L.args);
}

template <int XT, int W>
static cudaError_t setup_experts()
{
    return cudaFuncSetAttribute(moe_experts_kernel<XT, W>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                MoeStage<W>::SMEM);
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
    const int groups = (a.T + 7) / 8, extra = a.w_type == W_MX ? a.T : 1;
    const dim3 grid((unsigned)(a.E * groups + extra)), block(MOE_ROUTER_THREADS);
    cudaError_t e = L.x_out == OUT_BF16 ? launch_k(moe_router_kernel<OUT_BF16>, grid, block, 0, stream, a, groups)
                                        : launch_k(moe_router_kernel<OUT_F16>, grid, block, 0, stream, a, groups);
    if (e != cudaSuccess) return e;
    if (a.w_type == W_MX)
        return L.x_out == OUT_BF16 ? launch_experts<OUT_BF16, W_MX>(L, stream) : launch_experts<OUT_F16, W_MX>(L, stream);
    return L.x_out == OUT_BF16 ? launch_experts<OUT_BF16, W_BF16>(L, stream) : launch_experts<OUT_F16, W_F16>(L, stream);
}

}  // namespace mmact
