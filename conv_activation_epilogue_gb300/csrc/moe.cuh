// moe.cuh -- what the mixture-of-experts kernels for 16-bit (moe.cu) and MXFP4
// (moe_mxfp4.cu) weights share: the router's logits, the choice of experts, the
// lists of their tokens, grid barriers and the weighted sum.
#pragma once

#include "common.cuh"
#include "kernels_mx.h"
#include "mxfp4.cuh"

namespace mmact {

// A logit as a key whose unsigned order is the float order, NaN above all, and
// -0 equal to +0; never 0.
__device__ __forceinline__ uint32_t logit_key(float x)
{
    if (x != x) return 0xffffffffu;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float key_logit(uint32_t key)
{
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
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
// A CTA is a chain of loads: 16 tokens, 2 of 16 experts of 4096 x 1792 take 56.2 us with 128
// threads, 54 with 256; 512 help no further and cost layers of many experts (64 tokens,
// 8 of 64 experts of 2048 x 1024, MXFP4: 78.8 us with 256, 82.2 with 512).
constexpr int MOE_ROUTER_THREADS = 256, MOE_ROUTER_K = MOE_ROUTER_THREADS * 8;

// Router logits by one CTA, for an expert and eight tokens: its warps share K.
template <int XT>
__device__ __forceinline__ void router_logits(const MoeArgs &p, int block, int token_groups)
{
    __shared__ float red[MOE_ROUTER_THREADS / 32][8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint16_t *xs = static_cast<const uint16_t *>(p.x);
    const int e = block / token_groups, t0 = (block - e * token_groups) * 8, n = min(8, p.T - t0);
    const uint16_t *r = static_cast<const uint16_t *>(p.router) + (int64_t)e * p.H;
    float s[8] = {};
    for (int k = threadIdx.x * 8; k < p.H; k += MOE_ROUTER_K) {
        const uint4 b = *reinterpret_cast<const uint4 *>(r + k);
        const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
        uint4 a[8];                                        // tokens past the last one: the last one again
#pragma unroll
        for (int t = 0; t < 8; ++t) a[t] = *reinterpret_cast<const uint4 *>(xs + (int64_t)(t0 + min(t, n - 1)) * p.H + k);
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
    if (threadIdx.x < n) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < MOE_ROUTER_THREADS / 32; ++w) sum += red[w][threadIdx.x];
        p.logits[(int64_t)(t0 + threadIdx.x) * p.E + e] = sum + (p.router_bias != nullptr ? p.router_bias[e] : 0.0f);
    }
}

// ------------------------------------------------------------ choice of experts --
// Top k of a token by LANES lanes of a warp (32 / LANES tokens side by side; every
// lane of the warp calls it): each round the largest key of those left, then the
// lowest index that has it, whose key becomes 0; then the softmax weights.  `keys`:
// the token's, in shared memory; lane `sub` of the token reads and clears only those
// at sub + i * LANES.
template <int LANES>
__device__ __forceinline__ void choose_experts(const MoeArgs &p, MoeShared &S, uint32_t *keys, int t, bool valid, bool write)
{
    const int sub = threadIdx.x & (LANES - 1);
    short *choice = S.choice + t * p.top;
    float *probs = S.probs + t * p.top;
    for (int j = 0; j < p.top; ++j) {
        uint32_t key = 0, at = 0xffffu;
#pragma unroll 4
        for (int e = sub; e < p.E; e += LANES) {
            const uint32_t k = keys[e];
            if (k > key) key = k, at = (uint32_t)e;
        }
        __syncwarp();
        if constexpr (LANES == 32) {
            const uint32_t best = __reduce_max_sync(0xffffffffu, key);
            at = __reduce_min_sync(0xffffffffu, key == best ? at : 0xffffu);
            key = best;
        } else {
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) {
                const uint32_t k2 = __shfl_xor_sync(0xffffffffu, key, o), at2 = __shfl_xor_sync(0xffffffffu, at, o);
                if (k2 > key || (k2 == key && at2 < at)) key = k2, at = at2;
            }
        }
        if (valid) {
            if ((int)(at & (LANES - 1)) == sub) keys[at] = 0;
            if (sub == 0) choice[j] = (short)at, probs[j] = key_logit(key);
        }
    }
    __syncwarp();
    const float peak = probs[0];
    float total = 0.0f;
    if (!p.normalize) {
        for (int e = sub; e < p.E; e += LANES)
            if (keys[e] != 0) total += expf(key_logit(keys[e]) - peak);
    }
    for (int j = sub; j < p.top; j += LANES) total += expf(probs[j] - peak);
    __syncwarp();
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (!valid) return;
    for (int j = sub; j < p.top; j += LANES) {
        const float w = expf(probs[j] - peak) / total;
        probs[j] = w;
        if (write) {
            p.experts[t * p.top + j] = choice[j];
            p.probs[t * p.top + j] = w;
        }
    }
}

// The slots of each expert, in groups, built by every CTA.  `mask`: for each
// expert one bit for each slot that chose it (in shared memory that is free until
// the rings start, zero before), from which counts and places follow by counting
// bits.
template <int GROUP, int THREADS>
__device__ __forceinline__ void build_lists(const MoeArgs &p, MoeShared &S, uint32_t *mask)
{
    const int tid = threadIdx.x, n_slots = p.T * p.top, words = (n_slots + 31) / 32;
    for (int s = tid; s < n_slots; s += THREADS) atomicOr(&mask[S.choice[s] * words + (s >> 5)], 1u << (s & 31));
    ptx::cta_sync();
    for (int e = tid; e < p.E; e += THREADS) {
        int c = 0;
        for (int w = 0; w < words; ++w) c += __popc(mask[e * words + w]);
        S.count[e] = (short)c;
    }
    ptx::cta_sync();
    if (tid < 32) {                                            // consecutive experts to a lane, one running sum over the warp
        const int per = (p.E + 31) / 32, e0 = tid * per, e1 = min(p.E, e0 + per);
        int sum = 0, gsum = 0;
        for (int e = e0; e < e1; ++e) sum += S.count[e], gsum += (S.count[e] + GROUP - 1) / GROUP;
        __syncwarp();
        int at = sum, n = gsum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, at, o), gup = __shfl_up_sync(0xffffffffu, n, o);
            if (tid >= o) at += up, n += gup;
        }
        const int all = __shfl_sync(0xffffffffu, at, 31), groups = __shfl_sync(0xffffffffu, n, 31);
        at -= sum, n -= gsum;
        for (int e = e0; e < e1; ++e) {
            const int c = S.count[e];
            S.start[e] = (short)at;
            for (int g = 0; g * GROUP < c; ++g, ++n) S.act[n] = (short)e, S.first[n] = (short)(at + g * GROUP);
            at += c;
        }
        if (tid == 0) {
            S.first[groups] = (short)all;
            S.nact = groups;
        }
    }
    ptx::cta_sync();
    for (int s = tid; s < n_slots; s += THREADS) {
        const int e = S.choice[s];
        int at = S.start[e] + __popc(mask[e * words + (s >> 5)] & ((1u << (s & 31)) - 1u));
        for (int w = 0; w < s >> 5; ++w) at += __popc(mask[e * words + w]);
        S.slot[at] = (short)s;
    }
    ptx::cta_sync();
}

// Choice and lists by every thread of an experts kernel: all logits go where the
// rings will be (`keys`: T x E words), the lists' masks to `mask`.  A warp takes a
// token, or with more tokens than warps four at a time, eight lanes to each: the
// rounds are chains of dependent steps and of warp reductions, which an SM does one
// at a time.  8 of 64 experts: one token 1.8 us by a warp, 2.6 by eight lanes; 64
// tokens 12 us by warps, 5.5 by eight lanes each.
template <int GROUP, int THREADS>
__device__ __forceinline__ void plan_experts(const MoeArgs &p, MoeShared &S, uint32_t *keys, uint32_t *mask)
{
    constexpr int WARPS = THREADS / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = p.T * p.E, n4 = n / 4;
    for (int i = threadIdx.x; i < p.E * ((p.T * p.top + 31) / 32); i += THREADS) mask[i] = 0;
    for (int i = threadIdx.x; i < n4; i += 4 * THREADS) {
        float4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (i + u * THREADS < n4) v[u] = __ldcg(reinterpret_cast<const float4 *>(p.logits) + i + u * THREADS);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (i + u * THREADS < n4)
                reinterpret_cast<uint4 *>(keys)[i + u * THREADS] =
                    make_uint4(logit_key(v[u].x), logit_key(v[u].y), logit_key(v[u].z), logit_key(v[u].w));
    }
    if ((int)threadIdx.x < n - 4 * n4) keys[4 * n4 + threadIdx.x] = logit_key(__ldcg(p.logits + 4 * n4 + threadIdx.x));
    ptx::cta_sync();
    const bool write = blockIdx.x == 0;
    if (p.T <= WARPS) {
        if (warp < p.T) choose_experts<32>(p, S, keys + warp * p.E, warp, true, write);
    } else {
        for (int t0 = warp * 4; t0 < p.T; t0 += WARPS * 4) {
            const int t = min(t0 + (lane >> 3), p.T - 1);
            choose_experts<8>(p, S, keys + t * p.E, t, t0 + (lane >> 3) < p.T, write);
        }
    }
    ptx::cta_sync();
    build_lists<GROUP, THREADS>(p, S, mask);
    ptx::fence_proxy_async_smem();                             // before the copies that overwrite both
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
    bool pairs;                      // the halves go together (gate, up)
};

__device__ __forceinline__ MoeProduct up_product(const MoeArgs &p, int stage_k, int token_k)
{
    const int step = p.gated ? p.half_rows : 2 * p.half_rows;
    return {p.H, (p.H + stage_k - 1) / stage_k, (p.H + token_k - 1) / token_k, (p.I + step - 1) / step, p.R1,
            p.gated ? p.I : p.half_rows, step, p.I, p.gated != 0};
}

__device__ __forceinline__ MoeProduct down_product(const MoeArgs &p, int stage_k, int token_k)
{
    const int step = 2 * p.half_rows;
    return {p.I, (p.I + stage_k - 1) / stage_k, (p.I + token_k - 1) / token_k, (p.H + step - 1) / step, p.H,
            p.half_rows, step, p.H, false};
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

// The end of an experts kernel: every o is written before y is summed.
template <int XT, int THREADS>
__device__ __forceinline__ void sum_experts(const MoeArgs &p, MoeShared &S, const Pipe &pp)
{
    ptx::cta_sync();
    if (threadIdx.x == 0) {
        S.go = 0;
        if (*pp.abort == 0u) {
            grid_arrive(p.counters + 1);
            S.go = grid_wait(pp, p.counters + 1) ? 1 : 0;
            if (S.go == 0) pipe_fail(pp);
        }
    }
    ptx::cta_sync();
    if (S.go == 0) return;
    for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < (int64_t)p.T * p.H; i += (int64_t)gridDim.x * THREADS) {
        const int t = (int)(i / p.H), r = (int)(i - (int64_t)t * p.H);
        float y = 0.0f;
        for (int j = 0; j < p.top; ++j)
            y = fmaf(S.probs[t * p.top + j], __ldcg(p.part + (int64_t)(t * p.top + j) * p.H + r), y);
        if constexpr (XT == OUT_BF16) static_cast<__nv_bfloat16 *>(p.y)[i] = __float2bfloat16_rn(y);
        else static_cast<__half *>(p.y)[i] = __float2half_rn(y);
    }
}

// A kernel whose CTAs wait for one another, with its set-up overlapping the end of
// the kernel before it.
template <typename... KArgs, typename... Args>
cudaError_t launch_cooperative(void (*kernel)(KArgs...), int grid, int threads, size_t smem, cudaStream_t stream,
                               Args &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args &&>(args)...);
}

}  // namespace mmact
