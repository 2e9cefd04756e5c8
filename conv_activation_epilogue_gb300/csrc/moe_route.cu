// moe_route.cu -- a mixture-of-experts router in training: choice of experts,
// probabilities, slots of each expert and balance loss from the logits, and the
// gradient of the logits.
//
// A warp takes a token: lane l holds the NV consecutive logits from column l * NV on,
// so that among equal logits the lowest lane, and in it the lowest register, has the
// lowest index.  A logit becomes an unsigned key of the same order (0 for -inf, which
// is never chosen; the largest for NaN); the choice is `top` times the warp's largest
// key.  The softmax is taken in the same registers, and each lane adds up its own
// columns over all tokens of the warp; warps, then CTAs, are added up in their order,
// so results repeat bit for bit.
#include "common.cuh"
#include "kernels_route.h"
#include "mxfp4.cuh"
#include "row_stores.cuh"

namespace mmact {

constexpr int ROUTE_WARPS = 8;

// NV logits of a row from column c on; columns past E are -inf.  VEC: rows begin on
// 16-byte boundaries (or NV values are fewer bytes, and rows begin on those).
template <int T, int NV, bool VEC>
__device__ __forceinline__ void route_load(const void *p, int64_t row, int E, int c, float (&z)[NV])
{
    constexpr int ES = T == IN_F32 ? 4 : 2, BYTES = NV * ES < 16 ? NV * ES : 16, PER = BYTES / ES;
    const char *at = static_cast<const char *>(p) + (row * E + c) * ES;
#pragma unroll
    for (int g = 0; g < NV / PER; ++g) {
        if constexpr (VEC && BYTES >= 4) {
            uint32_t w[BYTES / 4];
#pragma unroll
            for (int j = 0; j < BYTES / 4; ++j) w[j] = T == IN_F32 ? 0xff800000u : (T == IN_BF16 ? 0xff80ff80u : 0xfc00fc00u);
            if (c + g * PER < E) {
                if constexpr (BYTES == 16) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(at + g * 16);
                    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
                } else if constexpr (BYTES == 8) {
                    const uint2 u = *reinterpret_cast<const uint2 *>(at);
                    w[0] = u.x, w[1] = u.y;
                } else {
                    w[0] = *reinterpret_cast<const uint32_t *>(at);
                }
            }
#pragma unroll
            for (int j = 0; j < BYTES / 4; ++j) {
                if constexpr (T == IN_F32) {
                    z[g * PER + j] = __uint_as_float(w[j]);
                } else {
                    const float2 f = unpack2<T>(w[j]);
                    z[g * PER + 2 * j] = f.x, z[g * PER + 2 * j + 1] = f.y;
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const int i = g * PER + j;
                z[i] = -INFINITY;
                if (c + i < E) {
                    if constexpr (T == IN_F32) z[i] = reinterpret_cast<const float *>(at)[i];
                    else if constexpr (T == IN_BF16) z[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(at)[i]);
                    else z[i] = __half2float(reinterpret_cast<const __half *>(at)[i]);
                }
            }
        }
    }
}

// Unsigned key of a logit's order: -0 and 0 alike, NaN on top, -inf 0.
__device__ __forceinline__ uint32_t route_key(float z)
{
    const uint32_t b = __float_as_uint(z + 0.0f);
    const uint32_t k = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
    return z != z ? 0xffffffffu : (b == 0xff800000u ? 0u : k);
}

__device__ __forceinline__ float route_value(uint32_t key)
{
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}

template <int T, int NV, bool VEC>
__global__ void __launch_bounds__(32 * ROUTE_WARPS) route_kernel(const RouteArgs a)
{
    ptx::griddep_launch_dependents();
    __shared__ float sums[ROUTE_WARPS][32 * NV];
    __shared__ int slots[ROUTE_MAX_EXPERTS + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane * NV, E = a.E;
    for (int i = threadIdx.x; i <= E; i += blockDim.x) slots[i] = 0;
    __syncthreads();
    ptx::griddep_wait();
    float acc[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) acc[j] = 0.0f;
    int tokens = 0;
    for (int64_t t = (int64_t)blockIdx.x * ROUTE_WARPS + warp; t < a.T; t += (int64_t)gridDim.x * ROUTE_WARPS) {
        float z[NV];
        route_load<T, NV, VEC>(a.logits, t, E, c, z);
        const bool on = a.mask == nullptr || a.mask[t] != 0;
        uint32_t key[NV], best = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            key[j] = on ? route_key(z[j]) : 0u;
            best = max(best, key[j]);
        }
        uint32_t mine = 0, first = 0;
        int expert = -1;                                       // lane k: the k-th choice
        for (int k = 0; k < a.top; ++k) {
            const uint32_t top = __reduce_max_sync(0xffffffffu, best);
            if (k == 0) first = top;
            if (top == 0u) break;
            const int owner = __ffs(__ballot_sync(0xffffffffu, best == top)) - 1;
            int at = 0;
            if (lane == owner) {
                best = 0;
                bool taken = false;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    if (!taken && key[j] == top) taken = true, at = c + j, key[j] = 0;
                    best = max(best, key[j]);
                }
            }
            at = __shfl_sync(0xffffffffu, at, owner);
            if (lane == k) expert = at, mine = top;
        }
        float p = 0.0f;
        if (first != 0u) {
            const float peak = route_value(first);
            float ex[NV], sum = 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j) ex[j] = __expf(z[j] - peak), sum += ex[j];
            const float total = warp_sum(sum), inv = 1.0f / total;
#pragma unroll
            for (int j = 0; j < NV; ++j) acc[j] += ex[j] * inv;
            p = expert >= 0 ? __expf(route_value(mine) - peak) : 0.0f;
            p = p / (a.normalize ? warp_sum(p) : total);
            ++tokens;
        }
        if (lane < a.top) {
            a.experts[t * a.top + lane] = expert;
            a.probs[t * a.top + lane] = p;
            if (expert >= 0) atomicAdd(&slots[expert], 1);
        }
    }
    if (lane == 0 && tokens != 0) atomicAdd(&slots[E], tokens);
#pragma unroll
    for (int j = 0; j < NV; ++j) sums[warp][c + j] = acc[j];
    __syncthreads();
    for (int i = threadIdx.x; i <= E; i += blockDim.x) {
        if (i < E) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < ROUTE_WARPS; ++w) s += sums[w][i];
            a.part[(int64_t)blockIdx.x * E + i] = s;
        }
        a.part_counts[(int64_t)blockIdx.x * (E + 1) + i] = slots[i];
    }
}

// Partial sums of all CTAs, a column to a thread, then the loss.
__global__ void __launch_bounds__(ROUTE_MAX_EXPERTS) route_finish_kernel(const RouteArgs a, int grid)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    __shared__ float terms[ROUTE_MAX_EXPERTS / 32];
    __shared__ int tokens;
    const int e = threadIdx.x, E = a.E, lane = e & 31;
    float share = 0.0f;
    int count = 0;
    if (e < E) {
#pragma unroll 8
        for (int g = 0; g < grid; ++g) {
            share += a.part[(int64_t)g * E + e];
            count += a.part_counts[(int64_t)g * (E + 1) + e];
        }
        a.counts[e] = count;
    }
    if (e < 32) {
        int n = 0;
        for (int g = lane; g < grid; g += 32) n += a.part_counts[(int64_t)g * (E + 1) + E];
        n = __reduce_add_sync(0xffffffffu, n);
        if (e == 0) tokens = n, a.counts[E] = n;
    }
    const float term = warp_sum((float)count * share);
    if (lane == 0) terms[e >> 5] = term;
    __syncthreads();
    if (e == 0) {
        float s = 0.0f;
        for (int w = 0; w < (int)(blockDim.x >> 5); ++w) s += terms[w];
        const float n = (float)tokens;
        a.loss[0] = tokens == 0 ? 0.0f : a.coef * (float)E * (s / n) / (n * (float)a.top);
    }
}

// NV values from column c on to a row of dlogits, rounded to its type.
template <int T, int NV, bool VEC>
__device__ __forceinline__ void route_store(void *p, int64_t row, int E, int c, const float (&v)[NV])
{
    constexpr int ES = T == IN_F32 ? 4 : 2, BYTES = NV * ES < 16 ? NV * ES : 16, PER = BYTES / ES;
    const int64_t i0 = row * E + c;
    char *at = static_cast<char *>(p) + i0 * ES;
#pragma unroll
    for (int g = 0; g < NV / PER; ++g) {
        if constexpr (VEC && BYTES >= 4) {
            if (c + g * PER >= E) continue;
            uint32_t w[BYTES / 4];
#pragma unroll
            for (int j = 0; j < BYTES / 4; ++j) {
                if constexpr (T == IN_F32) w[j] = __float_as_uint(v[g * PER + j]);
                else w[j] = pack2<T>(v[g * PER + 2 * j], v[g * PER + 2 * j + 1]);
            }
            if constexpr (BYTES == 16) *reinterpret_cast<uint4 *>(at + g * 16) = make_uint4(w[0], w[1], w[2], w[3]);
            else if constexpr (BYTES == 8) *reinterpret_cast<uint2 *>(at) = make_uint2(w[0], w[1]);
            else *reinterpret_cast<uint32_t *>(at) = w[0];
        } else {
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (c + g * PER + j < E) store1<T>(p, i0 + g * PER + j, v[g * PER + j]);
        }
    }
}

// dz = p (u - p.u) + the chosen probabilities' part, u = coef E / (n^2 top) dloss counts.
template <int T, int NV, bool VEC>
__global__ void __launch_bounds__(32 * ROUTE_WARPS) route_backward_kernel(const RouteBackwardArgs a)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    __shared__ float rows[ROUTE_WARPS][32 * NV];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane * NV, E = a.E;
    float u[NV];
    {
        const float n = (float)a.counts[E];
        const float up = n > 0.0f ? a.coef * (float)E / n / (n * (float)a.top) * (a.dloss != nullptr ? a.dloss[0] : 0.0f) : 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) u[j] = c + j < E ? up * (float)a.counts[c + j] : 0.0f;
    }
    for (int64_t t = (int64_t)blockIdx.x * ROUTE_WARPS + warp; t < a.T; t += (int64_t)gridDim.x * ROUTE_WARPS) {
        float z[NV], peak = -INFINITY, sum = 0.0f, dot = 0.0f;
        route_load<T, NV, VEC>(a.logits, t, E, c, z);
        bool nan = false;
#pragma unroll
        for (int j = 0; j < NV; ++j) peak = fmaxf(peak, z[j]), nan |= z[j] != z[j];
        peak = warp_max(peak);
        if (__any_sync(0xffffffffu, nan)) peak = NAN;
        const bool on = peak != -INFINITY && (a.mask == nullptr || a.mask[t] != 0);
        float v[NV];
        if (!on) {
#pragma unroll
            for (int j = 0; j < NV; ++j) v[j] = 0.0f;
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j) v[j] = __expf(z[j] - peak), sum += v[j];
            const float total = warp_sum(sum), inv = 1.0f / total;
#pragma unroll
            for (int j = 0; j < NV; ++j) v[j] *= inv, dot += v[j] * u[j];
            dot = warp_sum(dot);
            float mine = 0.0f, g = 0.0f;
            int e = -1;
            if (a.dprobs != nullptr && lane < a.top) {
                e = a.experts[t * a.top + lane];
                if (e < 0 || e >= E) e = -1;
                if (e >= 0) {
                    g = a.dprobs[t * a.top + lane];
                    float ze;
                    if constexpr (T == IN_F32) ze = static_cast<const float *>(a.logits)[t * E + e];
                    else if constexpr (T == IN_BF16) ze = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.logits)[t * E + e]);
                    else ze = __half2float(static_cast<const __half *>(a.logits)[t * E + e]);
                    mine = __expf(ze - peak);
                }
            }
            mine /= a.normalize ? warp_sum(mine) : total;
            if (e < 0) mine = 0.0f;                            // no slot at all: 0 / 0
            const float mg = warp_sum(mine * g);
            const float off = a.normalize ? dot : dot + mg;
#pragma unroll
            for (int j = 0; j < NV; ++j) v[j] *= u[j] - off;
            if (a.dprobs != nullptr) {
                float *row = rows[warp];
#pragma unroll
                for (int j = 0; j < NV; ++j) row[c + j] = v[j];
                __syncwarp();
                // the forward pass gives a token an expert once; in another's lists equal entries add up in their order
                const float add = mine * (a.normalize ? g - mg : g);
                for (uint32_t left = __ballot_sync(0xffffffffu, e >= 0); left != 0;) {
                    const uint32_t same = __match_any_sync(0xffffffffu, e) & left;
                    const bool turn = (left >> lane & 1) != 0 && (int)(__ffs(same) - 1) == lane;
                    if (turn) row[e] += add;
                    left &= ~__ballot_sync(0xffffffffu, turn);
                    __syncwarp();
                }
#pragma unroll
                for (int j = 0; j < NV; ++j) v[j] = row[c + j];
                __syncwarp();
            }
        }
        route_store<T, NV, VEC>(a.dlogits, t, E, c, v);
    }
}

int route_grid(int64_t T, int sms)
{
    const int64_t ctas = (T + ROUTE_WARPS - 1) / ROUTE_WARPS;
    return (int)(ctas < 4 * sms ? ctas : 4 * sms);
}

template <int T, int NV>
static bool route_vec(int E)
{
    constexpr int BYTES = NV * (T == IN_F32 ? 4 : 2) < 16 ? NV * (T == IN_F32 ? 4 : 2) : 16;
    return E * (T == IN_F32 ? 4 : 2) % BYTES == 0;
}

template <int T, int NV>
static cudaError_t route_t(const RouteArgs &a, int grid, cudaStream_t s)
{
    auto k = route_vec<T, NV>(a.E) ? route_kernel<T, NV, true> : route_kernel<T, NV, false>;
    if (grid > 0) {                                            // without tokens: zeros
        const cudaError_t e = launch_k(k, dim3((unsigned)grid), dim3(32 * ROUTE_WARPS), 0, s, a);
        if (e != cudaSuccess) return e;
    }
    return launch_k(route_finish_kernel, dim3(1), dim3((unsigned)((a.E + 31) / 32 * 32)), 0, s, a, grid);
}

template <int T, int NV>
static cudaError_t route_backward_t(const RouteBackwardArgs &a, int grid, cudaStream_t s)
{
    auto k = route_vec<T, NV>(a.E) ? route_backward_kernel<T, NV, true> : route_backward_kernel<T, NV, false>;
    return launch_k(k, dim3((unsigned)grid), dim3(32 * ROUTE_WARPS), 0, s, a);
}

template <int T>
static cudaError_t route_e(const RouteArgs &a, int grid, cudaStream_t s)
{
    if (a.E <= 32) return route_t<T, 1>(a, grid, s);
    if (a.E <= 64) return route_t<T, 2>(a, grid, s);
    if (a.E <= 128) return route_t<T, 4>(a, grid, s);
    if (a.E <= 256) return route_t<T, 8>(a, grid, s);
    return route_t<T, 16>(a, grid, s);
}

template <int T>
static cudaError_t route_backward_e(const RouteBackwardArgs &a, int grid, cudaStream_t s)
{
    if (a.E <= 32) return route_backward_t<T, 1>(a, grid, s);
    if (a.E <= 64) return route_backward_t<T, 2>(a, grid, s);
    if (a.E <= 128) return route_backward_t<T, 4>(a, grid, s);
    if (a.E <= 256) return route_backward_t<T, 8>(a, grid, s);
    return route_backward_t<T, 16>(a, grid, s);
}

cudaError_t launch_moe_route(const RouteArgs &a, int type, int grid, cudaStream_t s)
{
    if (type == IN_BF16) return route_e<IN_BF16>(a, grid, s);
    if (type == IN_F16) return route_e<IN_F16>(a, grid, s);
    return route_e<IN_F32>(a, grid, s);
}

cudaError_t launch_moe_route_backward(const RouteBackwardArgs &a, int type, int sms, cudaStream_t s)
{
    const int64_t ctas = (a.T + ROUTE_WARPS - 1) / ROUTE_WARPS;
    const int grid = (int)(ctas < 6 * sms ? ctas : 6 * sms);
    if (type == IN_BF16) return route_backward_e<IN_BF16>(a, grid, s);
    if (type == IN_F16) return route_backward_e<IN_F16>(a, grid, s);
    return route_backward_e<IN_F32>(a, grid, s);
}

}  // namespace mmact
