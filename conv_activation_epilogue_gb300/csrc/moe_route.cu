// moe_route.cu -- a mixture-of-experts router in training: choice of experts,
// probabilities, slots of each expert and balance loss from the logits, and the
// gradient of the logits.
//
// G lanes take a token (8 to 32; 32 / G tokens to a warp), each NV consecutive logits, in
// registers.  A logit becomes an unsigned key of the same order.  The choice: the top-th
// largest of the lanes' largest keys bounds the choice from below, so that few keys
// besides the chosen ones reach it; those go to a list in shared memory, and each one's
// rank in it (by key, then index) is its slot.  Where the list would be long (many equal
// keys), the warp picks the largest key `top` times.  (Picking alone, a
// warp to a token, 131072 x 256 fp32 logits with 8 to choose took 183 us.)  The softmax
// is taken in the same registers, and each lane adds up its own columns over all its
// tokens; groups, warps and CTAs are added up in their order, so results repeat bit for bit.
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

// Unsigned key of a logit's order: -0 and 0 alike, NaN on top, -inf (never chosen) 0.
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

// e^d for d <= 0: the hardware's 2^x; results below 2^-126 are 0.
__device__ __forceinline__ float route_exp(float d)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d * 1.4426950408889634f));
    return r;
}

// Over the G lanes of a token.
template <int G>
__device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int d = G / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v)
{
    if constexpr (G == 32) {
        return __reduce_max_sync(0xffffffffu, v);
    } else {
#pragma unroll
        for (int d = G / 2; d > 0; d >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, d));
        return v;
    }
}

constexpr int ROUTE_LIST = 64;             // keys of a token that are ranked, at most

// A token's choice in shared memory.
struct RouteSlots {
    uint2 list[ROUTE_LIST];                // key, index
    uint2 slot[ROUTE_MAX_TOP];
};

template <int T, int G, int NV, bool VEC>
__global__ void __launch_bounds__(32 * ROUTE_WARPS, 3) route_kernel(const RouteArgs a)
{
    ptx::griddep_launch_dependents();
    constexpr int PER = 32 / G, GROUPS = ROUTE_WARPS * PER;
    __shared__ union {
        RouteSlots s[GROUPS];
        float sums[GROUPS][G * NV];
    } sh;
    __shared__ int slots[ROUTE_MAX_EXPERTS + 1];
    const int lane = threadIdx.x & 31, l = lane % G, c = l * NV, E = a.E, top = a.top, group = threadIdx.x / G;
    const uint32_t mates = G == 32 ? 0xffffffffu : ((1u << (G % 32)) - 1u) << (lane - l);
    RouteSlots &my = sh.s[group];
    for (int i = threadIdx.x; i <= E; i += blockDim.x) slots[i] = 0;
    __syncthreads();
    ptx::griddep_wait();
    float acc[NV], next[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) acc[j] = 0.0f;
    int tokens = 0;
    const int64_t step = (int64_t)gridDim.x * GROUPS, last = a.T - 1;
    // the same number of rounds for every group of a warp; the last token again where there is none left
    const int64_t first = (int64_t)blockIdx.x * GROUPS + group, warp0 = first - lane / G;
    route_load<T, NV, VEC>(a.logits, min(first, last), E, c, next);
    for (int64_t t0 = 0; warp0 + t0 < a.T; t0 += step) {
        const int64_t t = first + t0;
        float z[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) z[j] = next[j];
        if (warp0 + t0 + step < a.T) route_load<T, NV, VEC>(a.logits, min(t + step, last), E, c, next);
        const bool on = t < a.T && (a.mask == nullptr || a.mask[t] != 0);
        uint32_t key[NV], best = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            key[j] = on ? route_key(z[j]) : 0u;
            best = max(best, key[j]);
        }
        const uint32_t peak_key = group_max<G>(best);
        // Lower bound of the choice: lanes' largest keys, equal ones at once, until there are `top`.
        uint32_t bound = peak_key, rest = best;
        {
            int n = 0;
            for (int k = 0; k < top; ++k) {
                const uint32_t same = __ballot_sync(0xffffffffu, rest == bound) & mates;
                if (n < top) n += __popc(same);
                const bool more = n < top && bound != 0u;
                if (!__any_sync(0xffffffffu, more)) break;
                if (rest == bound) rest = 0u;
                const uint32_t m = group_max<G>(rest);
                if (more) bound = m;
            }
        }
        bound = max(bound, 1u);                                // fewer lanes than slots: every key but -inf's
        int mine = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) mine += key[j] >= bound ? 1 : 0;
        int at = mine;
#pragma unroll
        for (int d = 1; d < G; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, at, d, G);
            if (l >= d) at += v;
        }
        const int n = __shfl_sync(0xffffffffu, at, G - 1, G);
        for (int k = l; k < top; k += G) my.slot[k] = make_uint2(0u, 0xffffffffu);
        if (__any_sync(0xffffffffu, n > ROUTE_LIST)) {
            for (int k = 0; k < top; ++k) {
                const uint32_t m = group_max<G>(best);
                const uint32_t same = __ballot_sync(0xffffffffu, best == m) & mates;
                __syncwarp();
                if (m != 0u && lane == __ffs(same) - 1) {
                    best = 0;
                    bool taken = false;
#pragma unroll
                    for (int j = 0; j < NV; ++j) {
                        if (!taken && key[j] == m) taken = true, my.slot[k] = make_uint2(m, (uint32_t)(c + j)), key[j] = 0;
                        best = max(best, key[j]);
                    }
                }
                __syncwarp();
            }
        } else {
            at -= mine;
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (key[j] >= bound) my.list[at++] = make_uint2(key[j], (uint32_t)(c + j));
            __syncwarp();
            for (int i = l; i < n; i += G) {
                const uint2 me = my.list[i];
                int rank = 0;
                for (int j = 0; j < n; ++j) {                  // the list is in the order of the columns
                    const uint32_t other = my.list[j].x;
                    rank += other > me.x || (other == me.x && j < i) ? 1 : 0;
                }
                if (rank < top) my.slot[rank] = me;
            }
            __syncwarp();
        }
        const float peak = route_value(peak_key);
        float ex[NV], sum = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) ex[j] = peak_key != 0u ? route_exp(z[j] - peak) : 0.0f, sum += ex[j];
        const float total = group_sum<G>(sum), inv = peak_key != 0u ? 1.0f / total : 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) acc[j] += ex[j] * inv;
        constexpr int SL = (ROUTE_MAX_TOP + G - 1) / G;        // slots of a lane
        int expert[SL];
        float p[SL], chosen = 0.0f;
#pragma unroll
        for (int i = 0; i < SL; ++i) {
            const int k = l + i * G;
            expert[i] = -1, p[i] = 0.0f;
            if (k < top) {
                const uint2 s = my.slot[k];
                expert[i] = (int)s.y;
                if (expert[i] >= 0) p[i] = route_exp(route_value(s.x) - peak);
            }
            chosen += p[i];
        }
        const float over = a.normalize ? group_sum<G>(chosen) : total;
        if (l == 0 && peak_key != 0u) ++tokens;
#pragma unroll
        for (int i = 0; i < SL; ++i) {
            const int k = l + i * G;
            if (k < top && t < a.T) {
                a.experts[t * top + k] = expert[i];
                a.probs[t * top + k] = expert[i] >= 0 ? p[i] / over : 0.0f;
                if (expert[i] >= 0) atomicAdd(&slots[expert[i]], 1);
            }
        }
        __syncwarp();
    }
    if (tokens != 0) atomicAdd(&slots[E], tokens);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j) sh.sums[group][c + j] = acc[j];
    __syncthreads();
    for (int i = threadIdx.x; i <= E; i += blockDim.x) {
        if (i < E) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < GROUPS; ++w) s += sh.sums[w][i];
            a.part[(int64_t)blockIdx.x * E + i] = s;
        }
        a.part_counts[(int64_t)blockIdx.x * (E + 1) + i] = slots[i];
    }
}

// Partial sums of all CTAs, then the loss: a cluster of 8 CTAs (one, for few partial
// sums), each of which takes every 8th of them; a column to a thread and, for few columns,
// several threads.  Sums over threads, then over CTAs, in their order.
constexpr int ROUTE_FINISH_THREADS = 1024;

__global__ void __launch_bounds__(ROUTE_FINISH_THREADS) route_finish_kernel(const RouteArgs a, int grid, int ctas)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    __shared__ float share[ROUTE_FINISH_THREADS], terms[ROUTE_FINISH_THREADS / 32], loss;
    __shared__ int count[ROUTE_FINISH_THREADS];
    const int E = a.E, rank = ctas > 1 ? (int)ptx::cluster_ctarank() : 0;
    // columns 0..E of counts; column E has no share
    int cols = 32;
    while (cols < E + 1) cols *= 2;                            // at most 1024
    const int per = ROUTE_FINISH_THREADS / cols, col = threadIdx.x & (cols - 1), sub = threadIdx.x / cols;
    float s = 0.0f;
    int n = 0;
    if (col <= E) {
#pragma unroll 8
        for (int g = rank + sub * ctas; g < grid; g += ctas * per) {
            if (col < E) s += a.part[(int64_t)g * E + col];
            n += a.part_counts[(int64_t)g * (E + 1) + col];
        }
    }
    share[threadIdx.x] = s;
    count[threadIdx.x] = n;
    __syncthreads();
    if (sub == 0) {
        for (int i = 1; i < per; ++i) s += share[i * cols + col], n += count[i * cols + col];
        share[col] = s;
        count[col] = n;
    }
    if (ctas > 1) ptx::cluster_sync();
    else __syncthreads();
    if (rank == 0) {
        float term = 0.0f;
        if (sub == 0) {
            for (int r = 1; r < ctas; ++r) {
                s += ptx::ld_cluster_f32(ptx::mapa(ptx::smem_addr(&share[col]), (uint32_t)r));
                n += (int)ptx::ld_cluster_u32(ptx::mapa(ptx::smem_addr(&count[col]), (uint32_t)r));
            }
            if (col <= E) a.counts[col] = n;
            if (col < E) term = (float)n * s;
            if (col == E) loss = (float)n;
        }
        term = group_sum<32>(term);
        if ((threadIdx.x & 31) == 0) terms[threadIdx.x >> 5] = term;
        __syncthreads();
        if (threadIdx.x == 0) {
            float sum = 0.0f;
            for (int w = 0; w < cols / 32; ++w) sum += terms[w];
            const float tokens = loss;
            a.loss[0] = tokens == 0.0f ? 0.0f : a.coef * (float)E * (sum / tokens) / (tokens * (float)a.top);
        }
    }
    if (ctas > 1) ptx::cluster_sync();                         // no CTA leaves while its sums are read
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
template <int T, int G, int NV, bool VEC>
__global__ void __launch_bounds__(32 * ROUTE_WARPS) route_backward_kernel(const RouteBackwardArgs a)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    constexpr int PER = 32 / G, GROUPS = ROUTE_WARPS * PER, SL = (ROUTE_MAX_TOP + G - 1) / G;
    // e^z of a token; what its slots add (zeros but while a token is worked on)
    __shared__ __align__(16) float row[GROUPS][G * NV], extra[GROUPS][G * NV];
    const int lane = threadIdx.x & 31, l = lane % G, c = l * NV, E = a.E, top = a.top, group = threadIdx.x / G;
    float u[NV], next[NV], g_next[SL];
    int e_next[SL];
    {
        const float n = (float)a.counts[E];
        const float up = n > 0.0f ? a.coef * (float)E / n / (n * (float)top) * (a.dloss != nullptr ? a.dloss[0] : 0.0f) : 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) u[j] = c + j < E ? up * (float)a.counts[c + j] : 0.0f, extra[group][c + j] = 0.0f;
    }
    const int64_t step = (int64_t)gridDim.x * GROUPS, last = a.T - 1;
    const int64_t first = (int64_t)blockIdx.x * GROUPS + group, warp0 = first - lane / G;
    auto slots = [&](int64_t t) {
#pragma unroll
        for (int i = 0; i < SL; ++i) {
            const int k = l + i * G;
            e_next[i] = -1, g_next[i] = 0.0f;
            if (a.dprobs == nullptr || k >= top) continue;
            const int e = a.experts[t * top + k];
            g_next[i] = a.dprobs[t * top + k];
            if (e >= 0 && e < E) e_next[i] = e;
        }
    };
    route_load<T, NV, VEC>(a.logits, min(first, last), E, c, next);
    slots(min(first, last));
    for (int64_t t0 = 0; warp0 + t0 < a.T; t0 += step) {
        const int64_t t = first + t0;
        float v[NV], g[SL], peak = -INFINITY, sum = 0.0f, dot = 0.0f;
        int e[SL];
#pragma unroll
        for (int j = 0; j < NV; ++j) v[j] = next[j];
#pragma unroll
        for (int i = 0; i < SL; ++i) e[i] = e_next[i], g[i] = g_next[i];
        if (warp0 + t0 + step < a.T) {
            route_load<T, NV, VEC>(a.logits, min(t + step, last), E, c, next);
            slots(min(t + step, last));
        }
        const bool masked = a.mask != nullptr && a.mask[min(t, last)] == 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) asm("max.NaN.f32 %0, %0, %1;" : "+f"(peak) : "f"(v[j]));
#pragma unroll
        for (int d = G / 2; d > 0; d >>= 1) asm("max.NaN.f32 %0, %0, %1;" : "+f"(peak) : "f"(__shfl_xor_sync(0xffffffffu, peak, d)));
        const bool on = peak != -INFINITY && !masked;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            v[j] = on ? route_exp(v[j] - peak) : 0.0f;
            sum += v[j];
            dot += v[j] * u[j];
        }
        if constexpr (NV % 4 == 0) {
#pragma unroll
            for (int j = 0; j < NV; j += 4) *reinterpret_cast<float4 *>(&row[group][c + j]) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j) row[group][c + j] = v[j];
        }
        __syncwarp();
        const float total = group_sum<G>(sum), inv = on ? 1.0f / total : 0.0f;
        dot = group_sum<G>(dot) * inv;
        float mine[SL], chosen = 0.0f, mg = 0.0f;
#pragma unroll
        for (int i = 0; i < SL; ++i) {
            mine[i] = e[i] >= 0 ? row[group][e[i]] : 0.0f;
            chosen += mine[i];
            mg += mine[i] * g[i];
        }
        const float over = a.normalize ? group_sum<G>(chosen) : total;
        const float inv_over = over != 0.0f ? 1.0f / over : 0.0f;           // 0: a token without slots, or left out
        mg = group_sum<G>(mg) * inv_over;
        const float off = a.normalize ? dot : dot + mg;
#pragma unroll
        for (int i = 0; i < SL; ++i) {
            const float add = mine[i] * inv_over * (a.normalize ? g[i] - mg : g[i]);
            // The forward pass gives a token an expert once; in another's lists equal entries add up in their order.
            const uint32_t same = __match_any_sync(0xffffffffu, e[i] >= 0 ? group * ROUTE_MAX_EXPERTS + e[i] : -1 - lane);
            if (__all_sync(0xffffffffu, same == 1u << lane)) {
                if (e[i] >= 0) extra[group][e[i]] += add;
            } else {
                for (int k = 0; k < G; ++k) {
                    if (l == k && e[i] >= 0) extra[group][e[i]] += add;
                    __syncwarp();
                }
            }
            __syncwarp();
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) v[j] *= inv * (u[j] - off);
        if constexpr (NV % 4 == 0) {
#pragma unroll
            for (int j = 0; j < NV; j += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(&extra[group][c + j]);
                v[j] += x.x, v[j + 1] += x.y, v[j + 2] += x.z, v[j + 3] += x.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j) v[j] += extra[group][c + j];
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < SL; ++i)
            if (e[i] >= 0) extra[group][e[i]] = 0.0f;
        if (t < a.T) route_store<T, NV, VEC>(a.dlogits, t, E, c, v);
        __syncwarp();
    }
}

// Lanes to a token and logits to a lane, by the number of experts: as few lanes as leave
// registers for the logits (a warp takes 32 / G tokens at once, so that its reductions
// and its ranking serve all of them).
int route_lanes(int E) { return E <= 64 ? 8 : (E <= 128 ? 16 : 32); }

int route_grid(int64_t T, int64_t E, int sms)
{
    const int64_t groups = ROUTE_WARPS * 32 / route_lanes((int)E), ctas = (T + groups - 1) / groups;
    return (int)(ctas < 3 * sms ? ctas : 3 * sms);
}

template <int T, int NV>
static bool route_vec(int E)
{
    constexpr int BYTES = NV * (T == IN_F32 ? 4 : 2) < 16 ? NV * (T == IN_F32 ? 4 : 2) : 16;
    return E * (T == IN_F32 ? 4 : 2) % BYTES == 0;
}

template <int T, int G, int NV>
static cudaError_t route_t(const RouteArgs &a, int grid, cudaStream_t s)
{
    auto k = route_vec<T, NV>(a.E) ? route_kernel<T, G, NV, true> : route_kernel<T, G, NV, false>;
    if (grid > 0) {                                            // without tokens: zeros
        const cudaError_t e = launch_k(k, dim3((unsigned)grid), dim3(32 * ROUTE_WARPS), 0, s, a);
        if (e != cudaSuccess) return e;
    }
    const int ctas = grid > 32 ? 8 : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(ROUTE_FINISH_THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, route_finish_kernel, a, grid, ctas);
}

template <int T, int G, int NV>
static cudaError_t route_backward_t(const RouteBackwardArgs &a, int grid, cudaStream_t s)
{
    auto k = route_vec<T, NV>(a.E) ? route_backward_kernel<T, G, NV, true> : route_backward_kernel<T, G, NV, false>;
    return launch_k(k, dim3((unsigned)grid), dim3(32 * ROUTE_WARPS), 0, s, a);
}

template <int T>
static cudaError_t route_e(const RouteArgs &a, int grid, cudaStream_t s)
{
    if (a.E <= 32) return route_t<T, 8, 4>(a, grid, s);
    if (a.E <= 64) return route_t<T, 8, 8>(a, grid, s);
    if (a.E <= 128) return route_t<T, 16, 8>(a, grid, s);
    if (a.E <= 256) return route_t<T, 32, 8>(a, grid, s);
    return route_t<T, 32, 16>(a, grid, s);
}

template <int T>
static cudaError_t route_backward_e(const RouteBackwardArgs &a, int grid, cudaStream_t s)
{
    if (a.E <= 32) return route_backward_t<T, 8, 4>(a, grid, s);
    if (a.E <= 64) return route_backward_t<T, 8, 8>(a, grid, s);
    if (a.E <= 128) return route_backward_t<T, 16, 8>(a, grid, s);
    if (a.E <= 256) return route_backward_t<T, 32, 8>(a, grid, s);
    return route_backward_t<T, 32, 16>(a, grid, s);
}

cudaError_t launch_moe_route(const RouteArgs &a, int type, int grid, cudaStream_t s)
{
    if (type == IN_BF16) return route_e<IN_BF16>(a, grid, s);
    if (type == IN_F16) return route_e<IN_F16>(a, grid, s);
    return route_e<IN_F32>(a, grid, s);
}

cudaError_t launch_moe_route_backward(const RouteBackwardArgs &a, int type, int sms, cudaStream_t s)
{
    const int grid = route_grid(a.T, a.E, sms);
    if (type == IN_BF16) return route_backward_e<IN_BF16>(a, grid, s);
    if (type == IN_F16) return route_backward_e<IN_F16>(a, grid, s);
    return route_backward_e<IN_F32>(a, grid, s);
}

}  // namespace mmact
