// moe.cuh -- what the mixture-of-experts kernels for 16-bit (moe.cu) and MXFP4
// (moe_mxfp4.cu) weights share: the router's logits, the choice of experts, the
// lists of their tokens, grid barriers and the weighted sum.
#pragma once

#include "common.cuh"
#include "kernels_mx.h"
#include "mxfp4.cuh"

namespace mmact {

constexpr int MOE_MAX_T = 64, MOE_MAX_K = 16, MOE_MAX_E = 512;
constexpr int MOE_MIN_GROUP = 16;                              // tokens of an expert that share a read of its weights, at least
constexpr int MOE_MAX_BARS = 40;

// A logit as a key whose unsigned order is the float order, NaN above all, and
// -0 equal to +0; never 0.
__device__ __forceinline__ uint32_t logit_key(float x)
{
    if (x != x) return 0xffffffffu;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
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
constexpr int MOE_ROUTER_THREADS = 128;

// Router logits by one CTA, for an expert and eight tokens: four warps share K.
template <int XT>
__device__ __forceinline__ void router_logits(const MoeArgs &p, int block, int token_groups)
{
    __shared__ float red[4][8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint16_t *xs = static_cast<const uint16_t *>(p.x);
        const int e = block / token_groups, t0 = (block - e * token_groups) * 8, n = min(8, p.T - t0);
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
}

// ------------------------------------------------------------ choice of experts --
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
template <int GROUP, int THREADS>
__device__ __forceinline__ void build_lists(const MoeArgs &p, MoeShared &S, uint32_t *mask)
{
    const int tid = threadIdx.x, n_slots = p.T * p.top, words = (n_slots + 31) / 32;
    for (int i = tid; i < p.E * words; i += THREADS) mask[i] = 0;
    ptx::cta_sync();
    for (int s = tid; s < n_slots; s += THREADS) atomicOr(&mask[S.choice[s] * words + (s >> 5)], 1u << (s & 31));
    ptx::cta_sync();
    for (int e = tid; e < p.E; e += THREADS) {
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
    for (int s = tid; s < n_slots; s += THREADS) {
        const int e = S.choice[s];
        int at = S.start[e] + __popc(mask[e * words + (s >> 5)] & ((1u << (s & 31)) - 1u));
        for (int w = 0; w < s >> 5; ++w) at += __popc(mask[e * words + w]);
        S.slot[at] = (short)s;
    }
    ptx::cta_sync();
}

// Choice and lists by every thread of an experts kernel: all logits go where the
// rings will be (`logits`: T x E floats), the lists' masks to `mask`.
template <int GROUP, int THREADS>
__device__ __forceinline__ void plan_experts(const MoeArgs &p, MoeShared &S, float *logits, uint32_t *mask)
{
    constexpr int WARPS = THREADS / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll 8
    for (int i = threadIdx.x; i < p.T * p.E; i += THREADS) logits[i] = __ldcg(p.logits + i);
    ptx::cta_sync();
    for (int t = warp; t < p.T; t += 4 * WARPS) {
        const int left = (p.T - t + WARPS - 1) / WARPS;        // tokens of this warp from t on
        const bool write = blockIdx.x == 0;
        if (left == 1) choose_experts<1>(p, S, logits, t, WARPS, lane, write);
        else if (left == 2) choose_experts<2>(p, S, logits, t, WARPS, lane, write);
        else if (left == 3) choose_experts<3>(p, S, logits, t, WARPS, lane, write);
        else choose_experts<4>(p, S, logits, t, WARPS, lane, write);
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
