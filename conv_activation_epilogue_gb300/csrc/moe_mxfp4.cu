// moe_mxfp4.cu -- the mixture-of-experts layer (moe.cu) for experts' weights in
// MXFP4, on tcgen05.mma.kind::mxf4.
//
// Turning 4-bit weights into 16-bit values is more work than an SM can do in the
// time that it reads them (on mma.sync, with the weights widened in registers, 16
// tokens through 4 of 128 experts of 4096 x 2048 took 265 us where the bytes take
// 102; this form takes 120).  So the weights go to the tensor core as they
// are, and the tokens take their form: a value is written as a sum of eight MXFP4
// terms, the first the value rounded to the 4-bit grid, each next one the
// rounding of what is left, every term with a scale of its own for 32 values (the
// smallest power of two X that keeps the largest of them within 6 X).  The first term
// leaves at most a quarter of the block's largest value; when a term leaves at most X,
// the next leaves at most X / 8 (its own scale is X / 4, or X / 8 and less where less
// than 3 X / 4 is left): eight leave at most 2^-23, the precision of fp32 tokens.  The
// terms are eight columns of the MMA; with few tokens
// the columns are free.  They are also eight rows of 128 bytes, one 1024-byte atom
// of the shared-memory layout for 256 K, which is kept swizzled in global memory
// and moves by one bulk copy a token.
//
//   warp 0       weights: two TMA boxes of 64 rows x 128 bytes (256 K) a stage,
//                running ahead over items and over the grid barrier
//   warp 1       tokens: an atom for each token of the group
//   warp 2       scale copies to tensor memory and MMAs: 128 rows x 8 columns a token
//   warps 4..7   scale tiles of the stage: each thread the words of one row of
//                weights (a row may lie anywhere in the matrix's tiles) and of one
//                term row
//   warps 8..11  the sum over a token's columns, bias, activation, gate times up
//                (through shared memory), the terms of h, stores
//
// Sums, the activation and h are held in fp32 (h as its eight terms between the
// products).  Measured: 16 tokens, 4 of 128 experts of 4096 x 2048 (683 MB) 120 us, 5.7
// TB/s; one token, 8 of 64 experts of 2048 x 1024 33 us with cold caches, most of it the
// chain of router, choice and grid barriers.
#include "moe.cuh"

namespace mmact {

constexpr int MXE_THREADS = 384, MXE_GROUP = 16, MXE_STAGES = 6;
constexpr int MXE_K = 256;                                     // K of a stage
constexpr int MXE_TERMS = 8, MXE_ATOM = MXE_TERMS * 128, MXE_ATOM_SCALES = MXE_TERMS * 8;
constexpr int MXE_W_BYTES = 128 * 128, MXE_T_BYTES = MXE_GROUP * MXE_ATOM, MXE_S_BYTES = 2048;
constexpr int MXE_OFF_T = MXE_STAGES * MXE_W_BYTES, MXE_OFF_S = MXE_OFF_T + MXE_STAGES * MXE_T_BYTES;
constexpr int MXE_OFF_EX = MXE_OFF_S + MXE_STAGES * MXE_S_BYTES;     // [token][row] floats of one item
constexpr int MXE_OFF_SHARED = MXE_OFF_EX + MXE_GROUP * 128 * 4;
constexpr int MXE_SMEM = MXE_OFF_SHARED + (int)sizeof(MoeShared);
constexpr uint32_t MXE_ACC = 128, MXE_SCALE_COL = 256, MXE_TMEM = 512;
static_assert(MXE_SMEM <= CTA_SMEM && MXE_SMEM >= tmem_min_smem((int)MXE_TMEM), "shared memory budget");
static_assert(MXE_SCALE_COL + 16 * MXE_STAGES <= MXE_TMEM, "tensor memory budget");
static_assert(2 * MXE_STAGES + 5 <= MOE_MAX_BARS, "barriers");
static_assert(MOE_MAX_T * MOE_MAX_E * 4 <= MXE_OFF_S, "all logits");
static_assert(MOE_MAX_E * MOE_MAX_T * MOE_MAX_K / 8 <= MXE_OFF_EX - MOE_MAX_T * MOE_MAX_E * 4,
              "a bit for each expert and slot behind the logits");

// -------------------------------------------------------------------- terms --
// Scale byte of a term from the bits of the largest |r|: the smallest power of two
// X with |r| <= 6 X; 255 when it is an infinity or a NaN.
__device__ __forceinline__ uint32_t term_scale_byte(uint32_t amax_bits)
{
    const uint32_t e = amax_bits >> 23;
    if (e == 255u) return 255u;
    const uint32_t b = e + ((amax_bits & 0x7fffffu) > 0x400000u ? 1u : 0u);
    return b > 2u ? b - 2u : 0u;
}

// Where a term's 16 bytes of codes of block `blk` (of a token's row) stand: atom
// blk / 8, row `term`, chunk blk % 8, swizzled; and its scale.
__device__ __forceinline__ int64_t term_codes_at(int64_t token, int stages, int blk, int term)
{
    return (token * stages + (blk >> 3)) * MXE_ATOM + term * 128 + (((blk & 7) ^ term) << 4);
}

__device__ __forceinline__ int64_t term_scale_at(int64_t token, int stages, int blk, int term)
{
    return (token * stages + (blk >> 3)) * MXE_ATOM_SCALES + term * 8 + (blk & 7);
}

// Eight values r of `token` from K = k on, a multiple of 8, as their terms; four
// neighbouring lanes share a block.  (A lane to each value, with a warp maximum and
// three exchanges a term, made the epilogue what a layer with many tokens an expert
// waited for: 64 tokens, 4 of 4 experts of 2048 x 2048, 117 us, 60 so.  Unrolled, the
// terms cost one token 4 us more when the code is not in the SM's cache.)
__device__ __forceinline__ void put_terms(float (&r)[8], uint8_t *codes, uint8_t *scales, int64_t token, int stages, int k,
                                          bool valid)
{
#pragma unroll 1
    for (int j = 0; j < MXE_TERMS; ++j) {
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(r[i]) & 0x7fffffffu);
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const uint32_t b = term_scale_byte(amax);
        const float inv = mx_inv_scale(b == 255u ? 0u : b), x = mx_scale(b);
        float v[8], q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = r[i] * inv;
        const uint32_t c = b == 255u ? 0u : mx_encode8(v);
        mx_decode8(c, q);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = b == 255u ? 0.0f : r[i] - q[i] * x;   // exact
        if (valid) {
            *reinterpret_cast<uint32_t *>(codes + term_codes_at(token, stages, k >> 5, j) + (threadIdx.x & 3) * 4) = c;
            if ((threadIdx.x & 3) == 0) scales[term_scale_at(token, stages, k >> 5, j)] = (uint8_t)b;
        }
    }
}

// ------------------------------------------------------------------- router --
// The CTAs past the logits' prepare what the experts kernel reads: its counters,
// the terms of x up to a whole stage (zeros past H), and zero terms past h's
// blocks.
template <int XT>
__global__ void __launch_bounds__(MOE_ROUTER_THREADS) moe_mxfp4_router_kernel(const MoeArgs p, int token_groups)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    if ((int)blockIdx.x < p.E * token_groups) {
        router_logits<XT>(p, (int)blockIdx.x, token_groups);
        return;
    }
    // MOE_ROUTER_K of one token, 8 values to a thread, four threads to a block
    const int chunks = (p.Hp + MOE_ROUTER_K - 1) / MOE_ROUTER_K, at = (int)blockIdx.x - p.E * token_groups, t = at / chunks;
    const int k = (at - t * chunks) * MOE_ROUTER_K + (int)threadIdx.x * 8, stages = p.Hp / MXE_K;
    if (at == 0 && threadIdx.x < 2) p.counters[threadIdx.x] = 0;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (k < p.H) raw = __ldcg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.x) + (int64_t)t * p.H + k));
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    float r[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<XT>(w[i]);
        r[2 * i] = f.x;
        r[2 * i + 1] = f.y;
    }
    put_terms(r, p.x_codes, p.x_scales, t, stages, k, k < p.Hp);
    fence_proxy_async_all();                                   // bulk copies read the terms
    if (at != t * chunks) return;
    const int blocks = (p.I + 31) / 32, hstages = p.Ip / MXE_K, pad = hstages * 8 - blocks;
    for (int i = threadIdx.x; i < pad * MXE_TERMS * p.top; i += MOE_ROUTER_THREADS) {
        const int j = i % MXE_TERMS, b = blocks + i / MXE_TERMS % pad;
        const int64_t slot = (int64_t)t * p.top + i / (MXE_TERMS * pad);
        *reinterpret_cast<uint4 *>(p.h_codes + term_codes_at(slot, hstages, b, j)) = make_uint4(0, 0, 0, 0);
        p.h_scales[term_scale_at(slot, hstages, b, j)] = 0;
    }
    fence_proxy_async_all();
}

// ------------------------------------------------------------------ experts --
struct MxePipe {
    Pipe pp;                         // full0 (weights, tokens, scales), empty0; tfull0, tempty0: accumulators
    uint32_t ring, tokens, scales;
};

// Items of this CTA: f(group of tokens, tile); false ends them.
template <typename F>
__device__ __forceinline__ bool each_item(const MoeShared &S, const MoeProduct &pr, F f)
{
    const int n = S.nact * pr.tiles;
    for (int i = blockIdx.x; i < n; i += gridDim.x) {
        const int ai = i / pr.tiles;
        if (!f(ai, i - ai * pr.tiles)) return false;
    }
    return true;
}

__device__ __forceinline__ bool mxe_weights(const CUtensorMap *map, const MoeShared &S, const MxePipe &m,
                                            const MoeProduct &pr, uint32_t &use, uint64_t pol)
{
    return each_item(S, pr, [&](int ai, int tile) {
        const int row = S.act[ai] * pr.rows + tile * pr.step;
        // the upper half of the last tile may have no rows (its products are not stored either)
        const bool both = pr.pairs || tile * pr.step + 64 < pr.limit;
        for (int s = 0; s < pr.stages; ++s, ++use) {
            const uint32_t slot = use % MXE_STAGES, full = m.pp.full0 + 8 * slot, to = m.ring + slot * MXE_W_BYTES;
            if (!mx_warp_wait(m.pp, m.pp.empty0 + 8 * slot, ((use / MXE_STAGES) & 1u) ^ 1u)) return false;
            elected_expect_tx(full, both ? 2u * 8192u : 8192u);
            elected_load_2d(to, map, full, s * 64, row, pol);
            if (both) elected_load_2d(to + 8192u, map, full, s * 64, row + pr.half, pol);
        }
        return true;
    });
}

template <bool DOWN>
__device__ __forceinline__ bool mxe_tokens(const MoeArgs &p, const MoeShared &S, const MxePipe &m, const MoeProduct &pr,
                                           uint32_t &use)
{
    const int lane = threadIdx.x & 31;
    return each_item(S, pr, [&](int ai, int) {
        const int first = S.first[ai], cnt = S.first[ai + 1] - first;
        const int64_t slot_of = lane < cnt ? S.slot[first + lane] : 0;
        const uint8_t *from = DOWN ? p.h_codes + slot_of * pr.stages * MXE_ATOM
                                   : p.x_codes + slot_of / p.top * pr.stages * MXE_ATOM;
        for (int s = 0; s < pr.stages; ++s, ++use) {
            const uint32_t slot = use % MXE_STAGES, full = m.pp.full0 + 8 * slot;
            if (!mx_warp_wait(m.pp, m.pp.empty0 + 8 * slot, ((use / MXE_STAGES) & 1u) ^ 1u)) return false;
            elected_expect_tx(full, (uint32_t)cnt * MXE_ATOM);
            __syncwarp();
            if (lane < cnt)
                bulk_load(m.tokens + slot * MXE_T_BYTES + (uint32_t)lane * MXE_ATOM, from + (int64_t)s * MXE_ATOM, MXE_ATOM, full);
            __syncwarp();
        }
        return true;
    });
}

// Thread i of 128: the scale words of weight row i of the tile and of term row i
// (term i % 8 of token i / 8), four stages' loads in flight.
template <bool DOWN>
__device__ __forceinline__ bool mxe_scales(const MoeArgs &p, const MoeShared &S, const MxePipe &m, const MoeProduct &pr,
                                           uint32_t &use)
{
    const int i = (int)threadIdx.x - 128, lane = threadIdx.x & 31;
    const int tiles = (pr.K + 127) / 128;
    const uint8_t *weights = static_cast<const uint8_t *>(DOWN ? p.s2 : p.s1);
    const uint32_t at = (uint32_t)(i & 31) * 16u + (uint32_t)(i >> 5) * 4u;     // row i in a tile of 512 bytes
    return each_item(S, pr, [&](int ai, int tile) {
        const int first = S.first[ai], cnt = S.first[ai + 1] - first;
        const int64_t row = (int64_t)S.act[ai] * pr.rows + tile * pr.step + (i < 64 ? i : pr.half + i - 64);
        const bool has_row = row < (int64_t)p.E * pr.rows, has_term = i < 8 * cnt;
        const uint8_t *wp = weights + (has_row ? mx_scale_at(row, 0, tiles) : 0);
        const int64_t slot_of = has_term ? S.slot[first + (i >> 3)] : 0;
        const uint8_t *tp = (DOWN ? p.h_scales + slot_of * pr.stages * MXE_ATOM_SCALES
                                  : p.x_scales + slot_of / p.top * pr.stages * MXE_ATOM_SCALES) + (i & 7) * 8;
        for (int s0 = 0; s0 < pr.stages; s0 += 4) {
            uint32_t a[4][2];
            uint2 b[4];
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const int s = s0 + d;
                a[d][0] = has_row && 2 * s < tiles ? *reinterpret_cast<const uint32_t *>(wp + (int64_t)s * 1024) : 0u;
                a[d][1] = has_row && 2 * s + 1 < tiles ? *reinterpret_cast<const uint32_t *>(wp + (int64_t)s * 1024 + 512) : 0u;
                b[d] = has_term && s < pr.stages ? __ldcg(reinterpret_cast<const uint2 *>(tp + (int64_t)s * MXE_ATOM_SCALES)) : make_uint2(0, 0);
            }
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                if (s0 + d >= pr.stages) break;
                const uint32_t slot = use % MXE_STAGES, to = m.scales + slot * MXE_S_BYTES + at;
                if (!mx_warp_wait(m.pp, m.pp.empty0 + 8 * slot, ((use / MXE_STAGES) & 1u) ^ 1u)) return false;
                ptx::st_shared_u32(to, a[d][0]);
                ptx::st_shared_u32(to + 512u, a[d][1]);
                if (has_term) {
                    ptx::st_shared_u32(to + 1024u, b[d].x);
                    ptx::st_shared_u32(to + 1536u, b[d].y);
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(m.pp.full0 + 8 * slot);
                ++use;
            }
        }
        return true;
    });
}

__device__ __forceinline__ bool mxe_mma(const MoeShared &S, const MxePipe &m, const MoeProduct &pr, uint32_t &use, uint32_t &item)
{
    const int nk64 = (pr.K + 63) / 64;
    const uint64_t w0 = ptx::smem_desc(m.ring, 16u, 1024u, ptx::SWIZZLE_128B);
    const uint64_t t0 = ptx::smem_desc(m.tokens, 16u, 1024u, ptx::SWIZZLE_128B);
    const uint64_t s0 = ptx::smem_desc(m.scales, 16u, 128u, ptx::SWIZZLE_NONE);
    return each_item(S, pr, [&](int ai, int) {
        const int cnt = S.first[ai + 1] - S.first[ai], n = cnt < 2 ? 16 : (8 * cnt + 15) & ~15;
        const uint32_t id0 = ptx::idesc_mxf4(128, n, 0, 0), id2 = ptx::idesc_mxf4(128, n, 2, 2);
        const uint32_t buf = item & 1u, d = m.pp.tmem + buf * MXE_ACC;
        if (!mx_warp_wait(m.pp, m.pp.tempty0 + 8 * buf, ((item >> 1) & 1u) ^ 1u)) return false;
        ptx::tc_fence_after();
        for (int s = 0; s < pr.stages; ++s, ++use) {
            const uint32_t slot = use % MXE_STAGES;
            if (!mx_warp_wait(m.pp, m.pp.full0 + 8 * slot, (use / MXE_STAGES) & 1u)) return false;
            ptx::tc_fence_after();
            ptx::mma_mxf4_stage(d, w0 + slot * (MXE_W_BYTES >> 4), t0 + slot * (MXE_T_BYTES >> 4), s0 + slot * (MXE_S_BYTES >> 4),
                                m.pp.tmem + MXE_SCALE_COL + slot * 16u, id0, id2, min(4, nk64 - 4 * s), s != 0 ? 1u : 0u);
            ptx::commit_elected(m.pp.empty0 + 8 * slot);
        }
        ptx::commit_elected(m.pp.tfull0 + 8 * buf);
        ++item;
        return true;
    });
}

// Barrier of the four epilogue warps.
__device__ __forceinline__ void mxe_epilogue_sync()
{
    asm volatile("barrier.sync 1, 128;" ::: "memory");
}

// The same, and whether `ok` holds in all of them: either all go on or none.
__device__ __forceinline__ bool mxe_epilogue_all(bool ok)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\tbarrier.red.and.pred p, 1, 128, q;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(r) : "r"((uint32_t)ok) : "memory");
    return r != 0u;
}

template <bool DOWN>
__device__ __forceinline__ bool mxe_epilogue(const MoeArgs &p, const MoeShared &S, const MxePipe &m, const MoeProduct &pr,
                                             float *ex, uint32_t &item)
{
    const int warp = threadIdx.x >> 5, q = warp & 3, lane = threadIdx.x & 31, row = q * 32 + lane;
    return each_item(S, pr, [&](int ai, int tile) {
        const int e = S.act[ai], first = S.first[ai], cnt = S.first[ai + 1] - first;
        const uint32_t buf = item & 1u, taddr = m.pp.tmem + ((uint32_t)(q * 32) << 16) + buf * MXE_ACC;
        // this lane's row of the expert's matrix
        const int r = tile * pr.step + (row < 64 ? row : pr.half + row - 64);
        const bool in = pr.pairs ? tile * pr.step + (row & 63) < pr.limit : r < pr.limit;
        const float *bias = DOWN ? p.b2 : p.b1;
        const float add = bias != nullptr && in ? bias[(int64_t)e * pr.rows + r] : 0.0f;
        const bool full = warp_epi_wait(m.pp, m.pp.tfull0 + 8 * buf, (item >> 1) & 1u);
        if (DOWN ? !full : !mxe_epilogue_all(full)) return false;    // ex of the item before is read, too
        ptx::tc_fence_after();
        for (int c = 0; c < cnt; c += 2) {                     // the sum of a token's terms, the smallest first
            uint32_t d[16];
            ptx::tmem_ld16(taddr + 8 * c, d);
            float v[2] = {};
#pragma unroll
            for (int j = 7; j >= 0; --j) {
                v[0] += __uint_as_float(d[j]);
                v[1] += __uint_as_float(d[8 + j]);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (c + u >= cnt) break;
                v[u] += add;
                if constexpr (DOWN) {
                    if (in) p.part[(int64_t)S.slot[first + c + u] * p.H + r] = v[u];
                } else {
                    ex[(c + u) * 128 + row] = v[u];
                }
            }
            __syncwarp();
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(m.pp.tempty0 + 8 * buf);
        ++item;
        if constexpr (!DOWN) {
            mxe_epilogue_sync();                               // a gate row's up row is another warp's
            // four lanes to a block of a token, eight rows each: with 64 gate rows and 16 tokens one for everyone
            const int blocks = pr.pairs ? 2 : 4, units = cnt * blocks, hstages = p.Ip / MXE_K;
            for (int u0 = q * 8; u0 < units; u0 += 32) {
                const int u = min(u0 + (lane >> 2), units - 1), c = u / blocks, at = (u - c * blocks) * 32 + (lane & 3) * 8;
                const int first_row = tile * pr.step + at;
                float h[8];
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    const float4 g = *reinterpret_cast<const float4 *>(ex + c * 128 + at + i);
                    h[i] = g.x, h[i + 1] = g.y, h[i + 2] = g.z, h[i + 3] = g.w;
                }
                act_mx_all(p.act, h, p.alpha);
                if (pr.pairs)
#pragma unroll
                    for (int i = 0; i < 8; i += 4) {
                        const float4 g = *reinterpret_cast<const float4 *>(ex + c * 128 + 64 + at + i);
                        h[i] *= g.x, h[i + 1] *= g.y, h[i + 2] *= g.z, h[i + 3] *= g.w;
                    }
                if (first_row >= pr.limit)                     // I is a multiple of 8
#pragma unroll
                    for (int i = 0; i < 8; ++i) h[i] = 0.0f;
                __syncwarp();
                put_terms(h, p.h_codes, p.h_scales, S.slot[first + c], hstages, first_row,
                          u0 + (lane >> 2) < units && (first_row & ~31) < p.I);
            }
            __syncwarp();
        }
        return true;
    });
}

template <int XT>
__global__ void __launch_bounds__(MXE_THREADS, 1)
    moe_mxfp4_kernel(const __grid_constant__ CUtensorMap tm1, const __grid_constant__ CUtensorMap tm2, const MoeArgs p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    MoeShared &S = *reinterpret_cast<MoeShared *>(smem + MXE_OFF_SHARED);
    float *ex = reinterpret_cast<float *>(smem + MXE_OFF_EX);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    MxePipe m;
    m.ring = ptx::smem_addr(smem);
    m.tokens = m.ring + MXE_OFF_T;
    m.scales = m.ring + MXE_OFF_S;
    m.pp.full0 = ptx::smem_addr(S.bar);
    m.pp.empty0 = m.pp.full0 + 8 * MXE_STAGES;
    m.pp.tfull0 = m.pp.empty0 + 8 * MXE_STAGES;
    m.pp.tempty0 = m.pp.tfull0 + 16;
    m.pp.drain = m.pp.tempty0 + 16;
    m.pp.abort = reinterpret_cast<volatile uint32_t *>(&S.abort_flag);
    m.pp.status = p.status;
    m.pp.wait_ns = p.wait_ns;
    const bool aligned = (m.ring & 1023u) == 0;                // the swizzle counts rows from multiples of 1024 bytes
    if (threadIdx.x == 0) {
        if (!aligned) atomicOr(p.status, ST_SMEM_ALIGN);
        ptx::prefetch_tensormap(&tm1);
        ptx::prefetch_tensormap(&tm2);
        for (int s = 0; s < MXE_STAGES; ++s) {
            ptx::mbar_init(m.pp.full0 + 8 * s, 6);             // weights, tokens, four warps of scales
            ptx::mbar_init(m.pp.empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(m.pp.tfull0 + 8 * b, 1);
            ptx::mbar_init(m.pp.tempty0 + 8 * b, 4);
        }
        ptx::mbar_init(m.pp.drain, 1);
        S.abort_flag = aligned ? 0 : 1;
        ptx::fence_mbar_init();
    }
    ptx::griddep_wait();                                       // the router's logits and terms
    // tensor memory is taken when the kernels before this one are done; the next may start after that
    if (warp == 2) {
        ptx::tmem_alloc(ptx::smem_addr(&S.tmem), MXE_TMEM);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    plan_experts<MXE_GROUP, MXE_THREADS>(p, S, reinterpret_cast<uint32_t *>(smem),
                                         reinterpret_cast<uint32_t *>(smem + MOE_MAX_T * MOE_MAX_E * 4));
    ptx::tc_fence_after();
    m.pp.tmem = S.tmem;
    ptx::griddep_launch_dependents();

    const MoeProduct up = up_product(p, MXE_K, MXE_K), down = down_product(p, MXE_K, MXE_K);
    bool ok = aligned;
    auto wait_h = [&] {                                        // every h is written before any is read
        const bool all = lane != 0 || grid_wait(m.pp, p.counters);
        __syncwarp();
        return __all_sync(0xffffffffu, all) != 0;
    };
    uint32_t use = 0;
    if (warp == 0) {
        const uint64_t pol = ptx::createpolicy_evict_first();  // weights are read once
        ok = ok && mxe_weights(&tm1, S, m, up, use, pol) && mxe_weights(&tm2, S, m, down, use, pol);
    } else if (warp == 1) {
        fence_proxy_async_all();
        ok = ok && mxe_tokens<false>(p, S, m, up, use) && wait_h();
        fence_proxy_async_all();
        ok = ok && mxe_tokens<true>(p, S, m, down, use);
    } else if (warp == 2) {
        uint32_t item = 0;
        ok = ok && mxe_mma(S, m, up, use, item) && mxe_mma(S, m, down, use, item);
        ptx::commit_elected(m.pp.drain);
        ptx::mbar_wait_bounded(m.pp.drain, 0, DRAIN_NS, nullptr);
    } else if (warp >= 4 && warp < 8) {
        ok = ok && mxe_scales<false>(p, S, m, up, use) && wait_h() && mxe_scales<true>(p, S, m, down, use);
    } else if (warp >= 8) {
        uint32_t item = 0;
        ok = ok && mxe_epilogue<false>(p, S, m, up, ex, item);
        // this CTA's part of h is written
        fence_proxy_async_all();
        __syncwarp();
        mxe_epilogue_sync();
        if (ok && threadIdx.x == 256) grid_arrive(p.counters);
        __syncwarp();
        ok = ok && mxe_epilogue<true>(p, S, m, down, ex, item);
    }
    if (!ok && lane == 0) pipe_fail(m.pp);
    if (warp < 2) {
        // Every copy has landed before the CTA exits.  A stage is complete when all of its parts are; where the
        // others gave up it never is, and the bound is the time its copies have.
        for (uint32_t u = use > (uint32_t)MXE_STAGES ? use - MXE_STAGES : 0; u < use; ++u)
            ptx::mbar_wait_bounded(m.pp.full0 + 8 * (u % MXE_STAGES), (u / MXE_STAGES) & 1u, ok ? DRAIN_NS : 1000000ull, nullptr);
    }
    __syncwarp();
    ptx::tc_fence_before();
    sum_experts<XT, MXE_THREADS>(p, S, m.pp);                  // begins with a barrier of the CTA
    __syncwarp();
    if (warp == 2) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(m.pp.tmem, MXE_TMEM);
    }
}

template <int XT>
static cudaError_t launch_t(const MoeLaunch &L, cudaStream_t stream)
{
    const MoeArgs &a = L.args;
    const int groups = (a.T + 7) / 8;
    const int ctas = a.E * groups + a.T * ((a.Hp + MOE_ROUTER_K - 1) / MOE_ROUTER_K);
    const cudaError_t e =
        launch_k(moe_mxfp4_router_kernel<XT>, dim3((unsigned)ctas), dim3(MOE_ROUTER_THREADS), 0, stream, a, groups);
    if (e != cudaSuccess) return e;
    return launch_cooperative(moe_mxfp4_kernel<XT>, L.grid, MXE_THREADS, MXE_SMEM, stream, L.tm1, L.tm2, a);
}

cudaError_t setup_moe_mxfp4_kernels()
{
    const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    const cudaError_t e = cudaFuncSetAttribute(moe_mxfp4_kernel<OUT_BF16>, attr, MXE_SMEM);
    return e == cudaSuccess ? cudaFuncSetAttribute(moe_mxfp4_kernel<OUT_F16>, attr, MXE_SMEM) : e;
}

cudaError_t launch_moe_mxfp4(const MoeLaunch &L, cudaStream_t stream)
{
    return L.x_out == OUT_BF16 ? launch_t<OUT_BF16>(L, stream) : launch_t<OUT_F16>(L, stream);
}

}  // namespace mmact
