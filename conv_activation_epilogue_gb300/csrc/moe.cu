// moe.cu -- a whole mixture-of-experts layer for a few tokens (T <= 64) in two
// kernels.
//
//   router kernel    logits[t][e] = x[t] . router[e] + rb[e], the k experts of
//                    the largest logits (ties: the lowest index), their softmax
//                    weights
//   experts kernel   for every chosen expert, read once for all of its tokens:
//                    h = act(g) * u, g and u the two halves of w1[e] x + b1[e]
//                    (or h = act(w1[e] x + b1[e])); a grid barrier; then
//                    o = w2[e] h + b2[e], and y[t] = sum_j p[t][j] o[t, j],
//                    summed over j in order by the last CTA to finish a group
//                    of 16 rows of y
//
// With few tokens every weight is used a handful of times: the time is that of
// reading the chosen experts' weights once.  Products run on mma.sync.m16n8k16
// with the weights as the 16-row operand, straight from global memory to
// registers (each lane one 16-byte load per row and 32 K; which K a lane holds
// does not matter to a sum over K as long as both operands agree), and eight
// tokens as its columns.  The intermediate h is held as two bf16 halves
// hi = bf16(h), lo = bf16(h - hi), 16 bits of it, and multiplied as both, so no
// rounding to 16 bits stands between the two products.  fp16 down weights are
// split the same way (hi + lo is exact), which keeps h's fp32 range.
// MXFP4 weights become bf16 in registers (exactly: a scale is a power of two).
#include "common.cuh"
#include "kernels_mx.h"
#include "mxfp4.cuh"

namespace mmact {

enum : int { W_F16 = 0, W_BF16 = 1, W_MX = 2 };

constexpr int MOE_THREADS = 256, MOE_WARPS = 8;
constexpr int MOE_MAX_T = 64, MOE_MAX_K = 16, MOE_MAX_E = 512;

// ------------------------------------------------------------------ helpers --
// A logit as a key whose unsigned order is the float order, NaN above all, and
// -0 equal to +0; never 0.
__device__ __forceinline__ uint32_t logit_key(float x)
{
    if (x != x) return 0xffffffffu;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ uint4 ld_stream(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
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

// ------------------------------------------------------------------- router --
template <int XT>
__global__ void __launch_bounds__(512) moe_router_kernel(const MoeArgs p)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    extern __shared__ float logits[];
    const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // counters of the experts kernel
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < p.num_counters; i += gridDim.x * blockDim.x)
        p.counters[i] = 0;
    const uint16_t *x = static_cast<const uint16_t *>(p.x) + (int64_t)t * p.H;
    const uint16_t *r = static_cast<const uint16_t *>(p.router);
    for (int e = warp; e < p.E; e += 16) {
        float s = 0.0f;
        for (int k = lane * 8; k < p.H; k += 256) {
            const uint4 a = *reinterpret_cast<const uint4 *>(x + k);
            const uint4 b = *reinterpret_cast<const uint4 *>(r + (int64_t)e * p.H + k);
            const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = unpack2<XT>(aw[j]), g = unpack2<XT>(bw[j]);
                s = fmaf(f.x, g.x, s);
                s = fmaf(f.y, g.y, s);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) logits[e] = s + (p.router_bias != nullptr ? p.router_bias[e] : 0.0f);
    }
    if (p.w_type == W_MX) {
        // x as bf16 (hi, and lo for fp16 x) in the order MXFP4 codes unpack to, zeros up to the block
        for (int k = threadIdx.x; k < p.Hp; k += blockDim.x) {
            const float v = k < p.H ? (XT == OUT_BF16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(x)[k])
                                                      : __half2float(reinterpret_cast<const __half *>(x)[k]))
                                    : 0.0f;
            const __nv_bfloat16 hi = __float2bfloat16_rn(v);
            const int64_t at = (int64_t)t * p.Hp + mx_order(k);
            p.x_hi[at] = hi;
            if (XT == OUT_F16) p.x_lo[at] = __float2bfloat16_rn(v - __bfloat162float(hi));
        }
        // h between I and the end of its last block: zeros (the experts kernel writes [0, I))
        const int pad = p.Ip - p.I;
        for (int i = threadIdx.x; i < pad * p.top; i += blockDim.x) {
            const int64_t at = ((int64_t)t * p.top + i / pad) * p.Ip + p.I + i % pad;
            p.h_hi[at] = p.h_lo[at] = __float2bfloat16_rn(0.0f);
        }
    }
    __syncthreads();
    if (warp != 0) return;
    // top k: each round the largest (key, lowest index) of those left
    float peak = 0.0f, mine = 0.0f, total = 0.0f;
    uint32_t taken = 0;                                        // bit i: this lane's i-th logit is taken
    static_assert(MOE_MAX_E <= 32 * 32, "one bit for each of a lane's logits");
    for (int j = 0; j < p.top; ++j) {
        uint64_t best = 0;
        for (int e = lane, i = 0; e < p.E; e += 32, ++i) {
            if ((taken >> i) & 1u) continue;
            const uint64_t key = ((uint64_t)logit_key(logits[e]) << 32) | (0xffffffffu - (uint32_t)e);
            best = key > best ? key : best;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const uint64_t other = __shfl_xor_sync(0xffffffffu, best, o);
            best = other > best ? other : best;
        }
        const int e = (int)(0xffffffffu - (uint32_t)best);
        const float l = logits[e];
        if ((e & 31) == lane) taken |= 1u << (e >> 5);
        if (j == 0) peak = l;
        const float w = expf(l - peak);
        if (j == lane) {
            mine = w;
            p.experts[(int64_t)t * p.top + j] = e;
        }
        total += w;
    }
    if (!p.normalize) {
        total = 0.0f;
        for (int e = lane; e < p.E; e += 32) total += expf(logits[e] - peak);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    if (lane < p.top) p.probs[(int64_t)t * p.top + lane] = mine / total;
}

// ------------------------------------------------------------------ experts --
// The slots (token t, choice j -> t * k + j) of each expert, built by every CTA
// from the router's choices.
struct MoeLists {
    int nact;
    short act[MOE_MAX_E];            // active experts, ascending
    short first[MOE_MAX_E + 1];      // by active expert: its first entry of slot[]
    short slot[MOE_MAX_T * MOE_MAX_K];
};

__device__ __forceinline__ void build_lists(const MoeArgs &p, MoeLists &L, short *choice, short *count)
{
    const int tid = threadIdx.x, S = p.T * p.top;
    for (int s = tid; s < S; s += MOE_THREADS) choice[s] = (short)p.experts[s];
    __syncthreads();
    for (int e = tid; e < p.E; e += MOE_THREADS) {
        int c = 0;
        for (int s = 0; s < S; ++s) c += choice[s] == e;
        count[e] = (short)c;
    }
    __syncthreads();
    if (tid < 32) {                                            // 32 experts at a time: running sums over the warp
        int n = 0, at = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + tid, c = e < p.E ? count[e] : 0;
            int sum = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, sum, o);
                if (tid >= o) sum += up;
            }
            const uint32_t some = __ballot_sync(0xffffffffu, c != 0);
            if (c != 0) {
                const int i = n + __popc(some & ((1u << tid) - 1u));
                L.act[i] = (short)e;
                L.first[i] = (short)(at + sum - c);
            }
            n += __popc(some);
            at += __shfl_sync(0xffffffffu, sum, 31);
        }
        if (tid == 0) {
            L.first[n] = (short)at;
            L.nact = n;
        }
    }
    __syncthreads();
    for (int a = tid; a < L.nact; a += MOE_THREADS) {
        int at = L.first[a];
        const int e = L.act[a];
        for (int s = 0; s < S; ++s)
            if (choice[s] == e) L.slot[at++] = (short)s;
    }
    __syncthreads();
}

// One unit of K for the weights' type: two rows (this lane's row of the upper
// and of the lower half of the 16) as A fragments.
//   16-bit: 32 K, 2 instructions; MXFP4: 128 K, 8 instructions.
template <int W>
struct Frag {
    static constexpr int STEPS = W == W_MX ? 8 : 2;
    static constexpr int KU = W == W_MX ? 128 : 32;
    uint4 a, b;                      // raw 16 bytes of the two rows
    uint32_t sa, sb;                 // MXFP4: scale bytes
};

// Rows of one expert's weight matrix: base address and K extent.
struct WRows {
    const uint8_t *w;                // the matrix [rows_all, K], all experts
    const uint8_t *s;                // scale tiles (MXFP4)
    int64_t ra, rb;                  // this lane's two rows in it, < 0: no such row (zeros)
    int K, tiles, kb;                // kb: blocks (MXFP4)
};

template <int W>
__device__ __forceinline__ void load_frag(Frag<W> &f, const WRows &r, int u, int t4)
{
    f.a = f.b = make_uint4(0, 0, 0, 0);
    f.sa = f.sb = 0;
    if constexpr (W == W_MX) {
        const int blk = u * 4 + t4;
        if (blk < r.kb) {
            if (r.ra >= 0) {
                f.a = ld_stream(r.w + (r.ra * r.kb + blk) * 16);
                f.sa = r.s[mx_scale_at(r.ra, blk, r.tiles)];
            }
            if (r.rb >= 0) {
                f.b = ld_stream(r.w + (r.rb * r.kb + blk) * 16);
                f.sb = r.s[mx_scale_at(r.rb, blk, r.tiles)];
            }
        }
    } else {
        const int k = u * 32 + t4 * 8;
        if (k < r.K) {
            if (r.ra >= 0) f.a = ld_stream(r.w + (r.ra * r.K + k) * 2);
            if (r.rb >= 0) f.b = ld_stream(r.w + (r.rb * r.K + k) * 2);
        }
    }
}

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

// acc += rows x tokens over one unit.  xh / xl: this lane's token rows (hi, lo)
// for each group of eight tokens, null where there is no token; element offsets
// as the weights'.  LO: multiply the lo half too.  SPLITW: the fp16 weights are
// split into two bf16 halves (the tokens are bf16 hi / lo).
template <int W, int NT, bool LO, bool SPLITW>
__device__ __forceinline__ void unit_mma(float (&acc)[NT][4], const Frag<W> &f, const uint16_t *const (&xh)[NT],
                                         const uint16_t *const (&xl)[NT], int u, int t4, int K, int kb)
{
    if constexpr (W == W_MX) {
        uint32_t ra, rb;
        const uint32_t ma = mx_factor(f.sa, ra), mb = mx_factor(f.sb, rb);
        const bool big = __any_sync(0xffffffffu, f.sa > 128u || f.sb > 128u);
        const bool have = u * 4 + t4 < kb;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t va[4], vb[4];
            mx_word_bf16(word_of(f.a, w), ma, va);
            mx_word_bf16(word_of(f.b, w), mb, vb);
            if (big) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    va[i] = mul_bf16x2(va[i], ra);
                    vb[i] = mul_bf16x2(vb[i], rb);
                }
            }
            const int64_t at = (int64_t)u * 128 + t4 * 32 + w * 8;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                uint4 h = make_uint4(0, 0, 0, 0), l = h;
                if (have && xh[n] != nullptr) {
                    h = *reinterpret_cast<const uint4 *>(xh[n] + at);
                    if constexpr (LO) l = *reinterpret_cast<const uint4 *>(xl[n] + at);
                }
                mma_16816<true>(acc[n], va[0], vb[0], va[1], vb[1], h.x, h.y);
                mma_16816<true>(acc[n], va[2], vb[2], va[3], vb[3], h.z, h.w);
                if constexpr (LO) {
                    mma_16816<true>(acc[n], va[0], vb[0], va[1], vb[1], l.x, l.y);
                    mma_16816<true>(acc[n], va[2], vb[2], va[3], vb[3], l.z, l.w);
                }
            }
        }
    } else {
        const int k = u * 32 + t4 * 8;
        const bool have = k < K;
        uint32_t a[4] = {f.a.x, f.a.y, f.a.z, f.a.w}, b[4] = {f.b.x, f.b.y, f.b.z, f.b.w};
        uint32_t al[4], bl[4];
        if constexpr (SPLITW) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 fa = unpack2<OUT_F16>(a[i]), fb = unpack2<OUT_F16>(b[i]);
                split_pair(fa.x, fa.y, a[i], al[i]);
                split_pair(fb.x, fb.y, b[i], bl[i]);
            }
        }
        constexpr bool BF = W == W_BF16 || SPLITW;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            uint4 h = make_uint4(0, 0, 0, 0), l = h;
            if (have && xh[n] != nullptr) {
                h = *reinterpret_cast<const uint4 *>(xh[n] + k);
                if constexpr (LO) l = *reinterpret_cast<const uint4 *>(xl[n] + k);
            }
            mma_16816<BF>(acc[n], a[0], b[0], a[1], b[1], h.x, h.y);
            mma_16816<BF>(acc[n], a[2], b[2], a[3], b[3], h.z, h.w);
            if constexpr (LO) {
                mma_16816<BF>(acc[n], a[0], b[0], a[1], b[1], l.x, l.y);
                mma_16816<BF>(acc[n], a[2], b[2], a[3], b[3], l.z, l.w);
            }
            if constexpr (SPLITW) {
                mma_16816<BF>(acc[n], al[0], bl[0], al[1], bl[1], h.x, h.y);
                mma_16816<BF>(acc[n], al[2], bl[2], al[3], bl[3], h.z, h.w);
            }
        }
    }
}

// Rows [16] x tokens [NT * 8] of one item over all of K: the CTA's eight warps
// take the K units in turn, and the partial sums meet in shared memory:
// red[warp][row][token].
template <int W, int NT, bool LO, bool SPLITW>
__device__ __forceinline__ void item_product(float *red, const WRows &r, const uint16_t *const (&xh)[NT],
                                             const uint16_t *const (&xl)[NT])
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t4 = lane & 3, g = lane >> 2;
    float acc[NT][4] = {};
    const int units = (r.K + Frag<W>::KU - 1) / Frag<W>::KU;
    constexpr int DEPTH = W == W_MX ? 2 : 4;
    for (int u0 = warp; u0 < units; u0 += MOE_WARPS * DEPTH) {
        Frag<W> f[DEPTH];
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
            if (u0 + d * MOE_WARPS < units) load_frag<W>(f[d], r, u0 + d * MOE_WARPS, t4);
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
            if (u0 + d * MOE_WARPS < units)
                unit_mma<W, NT, LO, SPLITW>(acc, f[d], xh, xl, u0 + d * MOE_WARPS, t4, r.K, r.kb);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float *o = red + ((warp * 16 + g) * NT + n) * 8 + 2 * t4;
        *reinterpret_cast<float2 *>(o) = make_float2(acc[n][0], acc[n][1]);
        *reinterpret_cast<float2 *>(o + 8 * NT * 8) = make_float2(acc[n][2], acc[n][3]);
    }
}

template <int NT>
__device__ __forceinline__ float red_sum(const float *red, int row, int col)
{
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < MOE_WARPS; ++w) s += red[(w * 16 + row) * NT * 8 + col];
    return s;
}

// One item of the up product: tokens [n0, n0 + NT * 8) of active expert `ai`,
// rows tile `tile` (8 rows of h when gated, else 16).
template <int XT, int W, int NT>
__device__ __forceinline__ void up_item(const MoeArgs &p, const MoeLists &L, float *red, int ai, int tile, int n0)
{
    constexpr bool LO = W == W_MX && XT == OUT_F16;
    const int lane = threadIdx.x & 31, g = lane >> 2;
    const int e = L.act[ai], first = L.first[ai], cnt = L.first[ai + 1] - first;
    const int per = p.gated ? 8 : 16, i0 = tile * per;
    WRows r;
    r.w = static_cast<const uint8_t *>(p.w1);
    r.s = static_cast<const uint8_t *>(p.s1);
    r.K = p.H;
    r.kb = (p.H + 31) / 32;
    r.tiles = (p.H + 127) / 128;
    const int64_t base = (int64_t)e * p.R1;
    const int ia = i0 + g, ib = p.gated ? p.I + i0 + g : i0 + 8 + g;
    r.ra = ia < p.I ? base + ia : -1;
    r.rb = (p.gated ? ia < p.I : ib < p.I) ? base + ib : -1;
    const uint16_t *xh[NT], *xl[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int c = n0 + n * 8 + g;
        xh[n] = xl[n] = nullptr;
        if (c < cnt) {
            const int64_t t = L.slot[first + c] / p.top;
            if constexpr (W == W_MX) {
                xh[n] = reinterpret_cast<const uint16_t *>(p.x_hi) + t * p.Hp;
                xl[n] = reinterpret_cast<const uint16_t *>(p.x_lo) + t * p.Hp;
            } else {
                xh[n] = static_cast<const uint16_t *>(p.x) + t * p.H;
            }
        }
    }
    item_product<W, NT, LO, false>(red, r, xh, xl);
    __syncthreads();
    for (int i = threadIdx.x; i < per * NT * 8; i += MOE_THREADS) {
        const int row = i % per, c = i / per;
        if (n0 + c >= cnt || i0 + row >= p.I) continue;
        float v = red_sum<NT>(red, row, c);
        if (p.b1 != nullptr) v += p.b1[base + i0 + row];
        v = act_mx(p.act, v, p.alpha);
        if (p.gated) {
            float u = red_sum<NT>(red, 8 + row, c);
            if (p.b1 != nullptr) u += p.b1[base + p.I + i0 + row];
            v *= u;
        }
        const int k = i0 + row;
        const int64_t at = (int64_t)L.slot[first + n0 + c] * p.Ip + (W == W_MX ? mx_order(k) : k);
        const __nv_bfloat16 hi = __float2bfloat16_rn(v);
        p.h_hi[at] = hi;
        p.h_lo[at] = __float2bfloat16_rn(v - __bfloat162float(hi));
    }
    __syncthreads();
}

// One item of the down product: 16 rows of w2[e] for tokens [n0, n0 + NT * 8).
template <int W, int NT>
__device__ __forceinline__ void down_item(const MoeArgs &p, const MoeLists &L, float *red, int ai, int tile, int n0)
{
    const int lane = threadIdx.x & 31, g = lane >> 2;
    const int e = L.act[ai], first = L.first[ai], cnt = L.first[ai + 1] - first;
    WRows r;
    r.w = static_cast<const uint8_t *>(p.w2);
    r.s = static_cast<const uint8_t *>(p.s2);
    r.K = p.I;
    r.kb = (p.I + 31) / 32;
    r.tiles = (p.I + 127) / 128;
    const int64_t base = (int64_t)e * p.H;
    const int h0 = tile * 16;
    r.ra = h0 + g < p.H ? base + h0 + g : -1;
    r.rb = h0 + 8 + g < p.H ? base + h0 + 8 + g : -1;
    const uint16_t *xh[NT], *xl[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int c = n0 + n * 8 + g;
        xh[n] = xl[n] = nullptr;
        if (c < cnt) {
            const int64_t s = L.slot[first + c];
            xh[n] = reinterpret_cast<const uint16_t *>(p.h_hi) + s * p.Ip;
            xl[n] = reinterpret_cast<const uint16_t *>(p.h_lo) + s * p.Ip;
        }
    }
    item_product<W, NT, true, W == W_F16>(red, r, xh, xl);
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * NT * 8; i += MOE_THREADS) {
        const int row = i & 15, c = i >> 4;
        if (n0 + c >= cnt || h0 + row >= p.H) continue;
        float v = red_sum<NT>(red, row, c);
        if (p.b2 != nullptr) v += p.b2[base + h0 + row];
        p.part[(int64_t)L.slot[first + n0 + c] * p.H + h0 + row] = v;
    }
    __syncthreads();
}

template <int XT, int W>
__global__ void __launch_bounds__(MOE_THREADS) moe_experts_kernel(const MoeArgs p)
{
    __shared__ MoeLists L;
    __shared__ short choice[MOE_MAX_T * MOE_MAX_K], count[MOE_MAX_E];
    __shared__ __align__(16) float red[MOE_WARPS * 16 * 32];
    __shared__ int flag;
    const int tid = threadIdx.x;
    if (tid == 0) flag = 0;
    build_lists(p, L, choice, count);

    const int per = p.gated ? 8 : 16, up_tiles = (p.I + per - 1) / per, down_tiles = (p.H + 15) / 16;
    for (int it = blockIdx.x; it < L.nact * up_tiles; it += gridDim.x) {
        const int ai = it / up_tiles, tile = it - ai * up_tiles;
        const int cnt = L.first[ai + 1] - L.first[ai];
        for (int n0 = 0; n0 < cnt; n0 += 32) {
            if (cnt - n0 <= 8) up_item<XT, W, 1>(p, L, red, ai, tile, n0);
            else if (cnt - n0 <= 16) up_item<XT, W, 2>(p, L, red, ai, tile, n0);
            else up_item<XT, W, 4>(p, L, red, ai, tile, n0);
        }
    }
    // grid barrier: every h is written before any is read
    if (tid == 0) {
        __threadfence();
        atomicAdd(&p.counters[0], 1u);
        const uint64_t t0 = ptx::globaltimer();
        const volatile unsigned int *c = p.counters;
        uint32_t polls = 0;
        while (*c < gridDim.x) {
            if (((++polls & 63u) == 0 && ptx::globaltimer() - t0 > p.wait_ns) || polls >= (1u << 30)) {
                atomicOr(p.status, ST_TIMEOUT);
                flag = 1;
                break;
            }
        }
        __threadfence();
    }
    __syncthreads();
    if (flag != 0) return;

    for (int it = blockIdx.x; it < L.nact * down_tiles; it += gridDim.x) {
        const int tile = it / L.nact, ai = it - tile * L.nact;
        const int cnt = L.first[ai + 1] - L.first[ai];
        for (int n0 = 0; n0 < cnt; n0 += 32) {
            if (cnt - n0 <= 8) down_item<W, 1>(p, L, red, ai, tile, n0);
            else if (cnt - n0 <= 16) down_item<W, 2>(p, L, red, ai, tile, n0);
            else down_item<W, 4>(p, L, red, ai, tile, n0);
        }
        // the last expert of a row tile to finish adds the tile's rows up
        __threadfence();
        __syncthreads();
        if (tid == 0) flag = atomicAdd(&p.counters[1 + tile], 1u) == (unsigned)L.nact - 1u ? 2 : 0;
        __syncthreads();
        if (flag == 2) {
            __threadfence();
            for (int i = tid; i < 16 * p.T; i += MOE_THREADS) {
                const int row = tile * 16 + (i & 15), t = i >> 4;
                if (row >= p.H) continue;
                float y = 0.0f;
                for (int j = 0; j < p.top; ++j)
                    y = fmaf(p.probs[t * p.top + j], __ldcg(p.part + (int64_t)(t * p.top + j) * p.H + row), y);
                const int64_t at = (int64_t)t * p.H + row;
                if constexpr (XT == OUT_BF16) static_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16_rn(y);
                else static_cast<__half *>(p.y)[at] = __float2half_rn(y);
            }
        }
    }
}

template <int XT, int W>
static cudaError_t launch_experts(const MoeArgs &a, int sms, cudaStream_t stream)
{
    int per_sm = 0;
    cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, moe_experts_kernel<XT, W>, MOE_THREADS, 0);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) return cudaErrorLaunchOutOfResources;
    // no more CTAs than the larger of the two products can have items
    const int64_t slots = (int64_t)a.T * a.top;
    const int64_t act = slots < a.E ? slots : a.E;
    const int64_t items = act * ((a.gated ? (a.I + 7) / 8 : (a.I + 15) / 16) > (a.H + 15) / 16
                                     ? (a.gated ? (a.I + 7) / 8 : (a.I + 15) / 16)
                                     : (a.H + 15) / 16);
    int64_t grid = (int64_t)per_sm * sms;
    if (items < grid) grid = items;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(MOE_THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, moe_experts_kernel<XT, W>, a);
}

cudaError_t launch_moe(const MoeArgs &a, int x_out, int sms, cudaStream_t stream)
{
    const size_t smem = (size_t)a.E * 4;
    cudaError_t e = x_out == OUT_BF16 ? launch_k(moe_router_kernel<OUT_BF16>, dim3(a.T), dim3(512), smem, stream, a)
                                      : launch_k(moe_router_kernel<OUT_F16>, dim3(a.T), dim3(512), smem, stream, a);
    if (e != cudaSuccess) return e;
    if (a.w_type == W_MX)
        return x_out == OUT_BF16 ? launch_experts<OUT_BF16, W_MX>(a, sms, stream)
                                 : launch_experts<OUT_F16, W_MX>(a, sms, stream);
    return x_out == OUT_BF16 ? launch_experts<OUT_BF16, W_BF16>(a, sms, stream)
                             : launch_experts<OUT_F16, W_F16>(a, sms, stream);
}

}  // namespace mmact
