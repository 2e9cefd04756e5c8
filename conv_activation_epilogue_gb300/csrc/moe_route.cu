// moe_route.cu -- a mixture-of-experts router in training: choice of experts,
// probabilities, slots of each expert and balance loss from the logits, and the
// gradient of the logits.
//
// G lanes take a token (8 to 32; 32 / G tokens to a warp), NV logits each, in registers.
// The choice: the top-th largest of the lanes' largest logits bounds it from below, so
// that few logits besides the chosen ones reach it; those go to a list in shared
// memory, and each one's rank in it (by value, then index) is its slot.  Where the list
// would be long (many equal logits) or there are NaN, the warp picks the largest of
// them `top` times.  (Picking alone, a warp to a token, 131072 x 256 fp32 logits with 8
// to choose took 183 us.)  The softmax is taken in the same registers, and each lane
// adds up its own columns over all its tokens; groups, warps and CTAs are added up in
// their order, so results repeat bit for bit.
//
// Measured, logits from HBM: 131072 x 256 fp32 with 8 to choose 58 us forward (142 MB; bound
// by instructions, 335 a token), 57 us backward (277 MB, 4.9 TB/s; bound by the
// latency of a warp's reductions); 64 x 64 4.8 us, two launches.
#include "common.cuh"
#include "kernels_route.h"
#include "mxfp4.cuh"
#include "row_stores.cuh"

namespace mmact {

constexpr int ROUTE_WARPS = 8;             // of a CTA of the backward pass
// Of a CTA of the forward pass, one CTA to an SM: as many as have registers for NV
// logits, the next token's and the sums, or 8 when that is one token for each group of
// lanes.  (Several smaller CTAs to an SM are as many partial sums more for the last
// kernel: 131072 x 256 66.6 us with two of 8 warps, 62.9 with one of 16.)
template <int NV>
constexpr int ROUTE_FORWARD_WARPS = NV > 8 ? 16 : 24;


// Values of an access: with VEC (rows begin on 16-byte boundaries, or on those of NV
// values where these are fewer bytes) 16 bytes of them, else one.
template <int T, int NV>
constexpr int ROUTE_BYTES = NV * (T == IN_F32 ? 4 : 2) < 16 ? NV * (T == IN_F32 ? 4 : 2) : 16;
template <int T, int NV, bool VEC>
constexpr int ROUTE_PER = VEC ? ROUTE_BYTES<T, NV> / (T == IN_F32 ? 4 : 2) : 1;

// Column of a lane's j-th logit, rising with j: the lanes' accesses lie side by side.
template <int G, int PER>
__device__ __forceinline__ int route_col(int l, int j)
{
    return (j / PER * G + l) * PER + j % PER;
}

// A lane's logits of a row; columns past E are -inf.
template <int T, int G, int NV, bool VEC>
__device__ __forceinline__ void route_load(const void *p, int64_t row, int E, int l, float (&z)[NV])
{
    constexpr int ES = T == IN_F32 ? 4 : 2, BYTES = ROUTE_BYTES<T, NV>, PER = ROUTE_PER<T, NV, VEC>;
    const char *at = static_cast<const char *>(p) + row * E * ES;
    if constexpr (VEC) {
        static_assert(BYTES >= 8, "two words at least");
#pragma unroll
        for (int g = 0; g < NV / PER; ++g) {
            const int c = route_col<G, PER>(l, g * PER);
            uint32_t w[BYTES / 4];
#pragma unroll
            for (int j = 0; j < BYTES / 4; ++j) w[j] = T == IN_F32 ? 0xff800000u : (T == IN_BF16 ? 0xff80ff80u : 0xfc00fc00u);
            if (c < E) {
                if constexpr (BYTES == 16) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(at + c * ES);
                    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
                } else {
                    const uint2 u = *reinterpret_cast<const uint2 *>(at + c * ES);
                    w[0] = u.x, w[1] = u.y;
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
        }
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = route_col<G, PER>(l, j);
            z[j] = -INFINITY;
            if (c < E) {
                if constexpr (T == IN_F32) z[j] = reinterpret_cast<const float *>(at)[c];
                else if constexpr (T == IN_BF16) z[j] = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(at)[c]);
                else z[j] = __half2float(reinterpret_cast<const __half *>(at)[c]);
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

// max that a NaN wins
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <int G>
__device__ __forceinline__ float group_max_nan(float v)
{
    if constexpr (G == 32) {
        float r;
        asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
        return r;
    } else {
#pragma unroll
        for (int d = G / 2; d > 0; d >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, d));
        return v;
    }
}

// Lower bound of the choice of `top`: the top-th largest of the lanes' largest logits
// (`best`; equal ones may count once), -inf with fewer lanes than slots.  A warp's
// reductions are one instruction each; in less than a warp all lanes compare themselves with all
// others, by shuffles that do not wait for one another.
template <int G>
__device__ __forceinline__ float route_bound(float best, float peak, int top)
{
    if constexpr (G == 32) {
        float bound = peak;
        for (int k = 1; k < top; ++k) {
            if (best == bound) best = -INFINITY;
            bound = group_max_nan<G>(best);
        }
        return bound;
    } else {
        int above = 0;
#pragma unroll
        for (int d = 1; d < G; ++d) above += __shfl_xor_sync(0xffffffffu, best, d) > best ? 1 : 0;
        float bound = above < top ? best : peak;
#pragma unroll
        for (int d = G / 2; d > 0; d >>= 1) bound = fminf(bound, __shfl_xor_sync(0xffffffffu, bound, d));
        return top <= G ? bound : -INFINITY;
    }
}

template <int G>
constexpr int ROUTE_LIST = G == 32 ? 64 : 32;                  // logits of a token that are ranked, at most
constexpr float ROUTE_LOWEST = -3.402823466e38f;               // the lowest logit but -inf

// A token's choice in shared memory: logits (their bits) and indices.
template <int G>
struct RouteSlots {
    uint2 list[ROUTE_LIST<G>];
    uint2 slot[ROUTE_MAX_TOP];
};

// The choice by picking, for every token of a warp: G lanes, `top` times the largest
// logit, of equal ones that of the lowest column.
template <int G, int NV, int PER>
__device__ __forceinline__ void route_pick(const float (&z)[NV], RouteSlots<G> &my, int l, int top)
{
    uint32_t key[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) key[j] = route_key(z[j]);
    for (int k = 0; k < top; ++k) {
        uint32_t best = 0, col = 0xffffffffu;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (key[j] > best) best = key[j], col = (uint32_t)route_col<G, PER>(l, j);   // columns rise with j
        const uint32_t m = group_max<G>(best);
        if (m == 0u || best != m) col = 0xffffffffu;
        const uint32_t at = ~group_max<G>(~col);
        if (at != 0xffffffffu && at == col) {
            my.slot[k] = make_uint2(__float_as_uint(route_value(m)), at);
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (route_col<G, PER>(l, j) == (int)at) key[j] = 0;
        }
    }
    __syncwarp();
}

template <int T, int G, int NV, bool VEC>
__global__ void __launch_bounds__(32 * ROUTE_FORWARD_WARPS<NV>, 1) route_kernel(const RouteArgs a)
{
    ptx::griddep_launch_dependents();
    constexpr int GROUPS = ROUTE_FORWARD_WARPS<NV> * 32 / G, PER = ROUTE_PER<T, NV, VEC>;
    const int groups = blockDim.x / G;                         // GROUPS at most
    __shared__ union {
        RouteSlots<G> s[GROUPS];
        float sums[GROUPS][G * NV];
    } sh;
    __shared__ int slots[ROUTE_MAX_EXPERTS + 1];
    const int lane = threadIdx.x & 31, l = lane % G, E = a.E, top = a.top, group = threadIdx.x / G;
    const uint32_t mates = (G == 32 ? 0xffffffffu : (1u << (G % 32)) - 1u) << (lane - l), below = mates & ((1u << lane) - 1u);
    RouteSlots<G> &my = sh.s[group];
    for (int i = threadIdx.x; i <= E; i += blockDim.x) slots[i] = 0;
    __syncthreads();
    ptx::griddep_wait();
    float acc[NV], next[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) acc[j] = 0.0f;
    int tokens = 0;
    // rounds in which the warp has a token; the last one again where a group has none
    const int64_t step = (int64_t)gridDim.x * groups, last = a.T - 1, first = (int64_t)blockIdx.x * groups + group;
    const int64_t warp0 = first - lane / G;
    const int rounds = warp0 < a.T ? (int)((a.T - warp0 + step - 1) / step) : 0;
    if (rounds > 0) route_load<T, G, NV, VEC>(a.logits, min(first, last), E, l, next);
    int64_t t = first;
    for (int round = 0; round < rounds; ++round, t += step) {
        float z[NV], best = -INFINITY;
#pragma unroll
        for (int j = 0; j < NV; ++j) z[j] = next[j];
        if (round + 1 < rounds) route_load<T, G, NV, VEC>(a.logits, min(t + step, last), E, l, next);
        if (t >= a.T || (a.mask != nullptr && a.mask[t] == 0))
#pragma unroll
            for (int j = 0; j < NV; ++j) z[j] = -INFINITY;
#pragma unroll
        for (int j = 0; j < NV; ++j) best = max_nan(best, z[j]);
        const float peak = group_max_nan<G>(best);
        const float bound = max_nan(route_bound<G>(best, peak, top), ROUTE_LOWEST);
        int mine = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) mine += z[j] >= bound ? 1 : 0;
        // first place in the list of a lane's logits, from the counts' three low bits
        int at = 0, n = 0;
#pragma unroll
        for (int b = 0; b < 3; ++b) {
            const uint32_t set = __ballot_sync(0xffffffffu, (mine >> b & 1) != 0) & mates;
            at += __popc(set & below) << b;
            n += __popc(set) << b;
        }
        for (int k = l; k < top; k += G) my.slot[k] = make_uint2(0u, 0xffffffffu);
        if (__any_sync(0xffffffffu, n > ROUTE_LIST<G> || mine > 7 || peak != peak)) {
            __syncwarp();
            route_pick<G, NV, PER>(z, my, l, top);
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (z[j] >= bound) my.list[at++] = make_uint2(__float_as_uint(z[j]), (uint32_t)route_col<G, PER>(l, j));
            __syncwarp();
            for (int i = l; i < n; i += G) {
                const uint2 me = my.list[i];
                const float v = __uint_as_float(me.x);
                int rank = 0;
#pragma unroll 4
                for (int j = 0; j < n; ++j) {
                    const uint2 other = my.list[j];
                    const float w = __uint_as_float(other.x);
                    rank += w > v || (w == v && other.y < me.y) ? 1 : 0;
                }
                if (rank < top) my.slot[rank] = me;
            }
            __syncwarp();
        }
        const bool some = peak != -INFINITY;
        const float zero = some ? peak : 0.0f;                 // with nothing but -inf: e^-inf
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) z[j] = route_exp(z[j] - zero), sum += z[j];
        const float total = group_sum<G>(sum), inv = some ? __fdividef(1.0f, total) : 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) acc[j] += z[j] * inv;
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
                if (expert[i] >= 0) p[i] = route_exp(__uint_as_float(s.x) - peak);
            }
            chosen += p[i];
        }
        const float over = a.normalize ? __fdividef(1.0f, group_sum<G>(chosen)) : inv;
        if (l == 0 && some) ++tokens;
#pragma unroll
        for (int i = 0; i < SL; ++i) {
            const int k = l + i * G;
            if (k < top && t < a.T) {
                a.experts[t * top + k] = expert[i];
                a.probs[t * top + k] = expert[i] >= 0 ? p[i] * over : 0.0f;
                if (expert[i] >= 0) atomicAdd(&slots[expert[i]], 1);
            }
        }
        __syncwarp();
    }
    if (tokens != 0) atomicAdd(&slots[E], tokens);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j) sh.sums[group][route_col<G, PER>(l, j)] = acc[j];
    __syncthreads();
    for (int i = threadIdx.x; i <= E; i += blockDim.x) {
        if (i < E) {
            float s = 0.0f;
#pragma unroll 8
            for (int w = 0; w < groups; ++w) s += sh.sums[w][i];
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
    __shared__ float share[ROUTE_FINISH_THREADS], terms[ROUTE_FINISH_THREADS / 32];
    __shared__ int count[ROUTE_FINISH_THREADS], tokens;
    const int E = a.E, rank = ctas > 1 ? (int)ptx::cluster_ctarank() : 0, lane = threadIdx.x & 31;
    int cols = 32;
    while (cols < E) cols *= 2;                                // at most 512
    const int per = ROUTE_FINISH_THREADS / cols, col = threadIdx.x & (cols - 1), sub = threadIdx.x / cols;
    float s = 0.0f;
    int n = 0, t = 0;
    ptx::griddep_wait();
    if (col < E) {
#pragma unroll 8
        for (int g = rank + sub * ctas; g < grid; g += ctas * per) {
            s += a.part[(int64_t)g * E + col];
            n += a.part_counts[(int64_t)g * (E + 1) + col];
        }
    }
    if (rank == 0 && threadIdx.x < 32) {
        for (int g = lane; g < grid; g += 32) t += a.part_counts[(int64_t)g * (E + 1) + E];
        t = __reduce_add_sync(0xffffffffu, t);
        if (lane == 0) tokens = t, a.counts[E] = t;
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
            if (col < E) a.counts[col] = n, term = (float)n * s;
        }
        term = group_sum<32>(term);
        if (lane == 0) terms[threadIdx.x >> 5] = term;
        __syncthreads();
        if (threadIdx.x == 0) {
            float sum = 0.0f;
            for (int w = 0; w < cols / 32; ++w) sum += terms[w];
            const float f = (float)tokens;
            a.loss[0] = tokens == 0 ? 0.0f : a.coef * (float)E * (sum / f) / (f * (float)a.top);
        }
    }
    if (ctas > 1) ptx::cluster_sync();                         // no CTA leaves while its sums are read
}

// A lane's values to a row of dlogits, rounded to its type.
template <int T, int G, int NV, bool VEC>
__device__ __forceinline__ void route_store(void *p, int64_t row, int E, int l, const float (&v)[NV])
{
    constexpr int ES = T == IN_F32 ? 4 : 2, BYTES = ROUTE_BYTES<T, NV>, PER = ROUTE_PER<T, NV, VEC>;
    char *at = static_cast<char *>(p) + row * E * ES;
    if constexpr (VEC) {
#pragma unroll
        for (int g = 0; g < NV / PER; ++g) {
            const int c = route_col<G, PER>(l, g * PER);
            if (c >= E) continue;
            uint32_t w[BYTES / 4];
#pragma unroll
            for (int j = 0; j < BYTES / 4; ++j) {
                if constexpr (T == IN_F32) w[j] = __float_as_uint(v[g * PER + j]);
                else w[j] = pack2<T>(v[g * PER + 2 * j], v[g * PER + 2 * j + 1]);
            }
            if constexpr (BYTES == 16) *reinterpret_cast<uint4 *>(at + c * ES) = make_uint4(w[0], w[1], w[2], w[3]);
            else *reinterpret_cast<uint2 *>(at + c * ES) = make_uint2(w[0], w[1]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = route_col<G, PER>(l, j);
            if (c < E) store1<T>(at, c, v[j]);
        }
    }
}

// dz = p (u - p.u) + the chosen probabilities' part, u = coef E / (n^2 top) dloss counts.
template <int T, int G, int NV, bool VEC>
__global__ void __launch_bounds__(32 * ROUTE_WARPS, NV > 8 ? 2 : 4) route_backward_kernel(const RouteBackwardArgs a)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    constexpr int GROUPS = ROUTE_WARPS * 32 / G, PER = ROUTE_PER<T, NV, VEC>, SL = (ROUTE_MAX_TOP + G - 1) / G;
    // e^z of a token; what its slots add (zeros but while a token is worked on)
    __shared__ __align__(16) float row[GROUPS][G * NV], extra[GROUPS][G * NV];
    const int lane = threadIdx.x & 31, l = lane % G, E = a.E, top = a.top, group = threadIdx.x / G;
    float u[NV], next[NV], g_next[SL];
    int e_next[SL];
    {
        const float n = (float)a.counts[E];
        const float up = n > 0.0f ? a.coef * (float)E / n / (n * (float)top) * (a.dloss != nullptr ? a.dloss[0] : 0.0f) : 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = route_col<G, PER>(l, j);
            u[j] = c < E ? up * (float)a.counts[c] : 0.0f;
            extra[group][c] = 0.0f;
        }
    }
    const int64_t step = (int64_t)gridDim.x * GROUPS, last = a.T - 1, first = (int64_t)blockIdx.x * GROUPS + group;
    const int64_t warp0 = first - lane / G;
    const int rounds = warp0 < a.T ? (int)((a.T - warp0 + step - 1) / step) : 0;
    auto slots = [&](int64_t t) {
#pragma unroll
        for (int i = 0; i < SL; ++i) {
            const int k = l + i * G;
            e_next[i] = -1, g_next[i] = 0.0f;
            if (a.dprobs == nullptr || k >= top) continue;
            const int e = a.experts[t * top + k];
            const float g = a.dprobs[t * top + k];
            if (e >= 0 && e < E) e_next[i] = e, g_next[i] = g;             // what stands in a slot of -1 is not looked at
        }
    };
    if (rounds > 0) {
        route_load<T, G, NV, VEC>(a.logits, min(first, last), E, l, next);
        slots(min(first, last));
    }
    int64_t t = first;
    for (int round = 0; round < rounds; ++round, t += step) {
        float v[NV], g[SL], peak = -INFINITY, sum = 0.0f, dot = 0.0f;
        int e[SL];
#pragma unroll
        for (int j = 0; j < NV; ++j) v[j] = next[j];
#pragma unroll
        for (int i = 0; i < SL; ++i) e[i] = e_next[i], g[i] = g_next[i];
        if (round + 1 < rounds) {
            route_load<T, G, NV, VEC>(a.logits, min(t + step, last), E, l, next);
            slots(min(t + step, last));
        }
        const bool masked = a.mask != nullptr && a.mask[min(t, last)] == 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) peak = max_nan(peak, v[j]);
        peak = group_max_nan<G>(peak);
        const bool on = peak != -INFINITY && !masked;
        if (!on)
#pragma unroll
            for (int i = 0; i < SL; ++i) e[i] = -1, g[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            v[j] = on ? route_exp(v[j] - peak) : 0.0f;
            sum += v[j];
            dot += v[j] * u[j];
        }
        if constexpr (PER % 4 == 0) {
#pragma unroll
            for (int j = 0; j < NV; j += 4)
                *reinterpret_cast<float4 *>(&row[group][route_col<G, PER>(l, j)]) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j) row[group][route_col<G, PER>(l, j)] = v[j];
        }
        __syncwarp();
        const float total = group_sum<G>(sum), inv = on ? __fdividef(1.0f, total) : 0.0f;
        dot = group_sum<G>(dot) * inv;
        float mine[SL], chosen = 0.0f, mg = 0.0f;
#pragma unroll
        for (int i = 0; i < SL; ++i) {
            mine[i] = e[i] >= 0 ? row[group][e[i]] : 0.0f;
            chosen += mine[i];
            mg += mine[i] * g[i];
        }
        const float over = a.normalize ? group_sum<G>(chosen) : total;
        const float inv_over = over != 0.0f ? __fdividef(1.0f, over) : 0.0f;           // 0: a token without slots, or left out
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
        for (int j = 0; j < NV; ++j) v[j] = on ? v[j] * (inv * (u[j] - off)) : 0.0f;
        if constexpr (PER % 4 == 0) {
#pragma unroll
            for (int j = 0; j < NV; j += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(&extra[group][route_col<G, PER>(l, j)]);
                v[j] += x.x, v[j + 1] += x.y, v[j + 2] += x.z, v[j + 3] += x.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j) v[j] += extra[group][route_col<G, PER>(l, j)];
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < SL; ++i)
            if (e[i] >= 0) extra[group][e[i]] = 0.0f;
        if (t < a.T) route_store<T, G, NV, VEC>(a.dlogits, t, E, l, v);
        __syncwarp();
    }
}

// Lanes to a token and logits to a lane: as few lanes as leave registers for the logits (a
// warp takes 32 / G tokens at once, so that its reductions and its ranking serve all of
// them), but, for the choice, about twice as many lanes with logits as there are slots,
// or the lanes' largest logits bound it badly.
struct RouteShape {
    int lanes, each;
};

static RouteShape route_shape(int E, int top)
{
    if (E <= 32) return {8, 4};
    if (E <= 64) return top <= 4 ? RouteShape{8, 8} : RouteShape{16, 4};
    if (E <= 128) return top <= 4 ? RouteShape{8, 16} : RouteShape{16, 8};
    if (E <= 256) return top <= 8 ? RouteShape{16, 16} : RouteShape{32, 8};
    return {32, 16};
}

static int route_ctas(int64_t T, int lanes, int warps, int most)
{
    const int64_t groups = warps * 32 / lanes, ctas = (T + groups - 1) / groups;
    return (int)(ctas < most ? ctas : most);
}

// Warps of a CTA of the forward pass.
static int route_warps(int64_t T, RouteShape s, int sms)
{
    if (T * s.lanes <= (int64_t)sms * 8 * 32) return 8;
    return s.each > 8 ? ROUTE_FORWARD_WARPS<16> : ROUTE_FORWARD_WARPS<8>;
}

int route_grid(int64_t T, int64_t E, int64_t top, int sms)
{
    const RouteShape s = route_shape((int)E, (int)top);
    return route_ctas(T, s.lanes, route_warps(T, s, sms), sms);
}

template <int T, int NV>
static bool route_vec(int E)
{
    return E * (T == IN_F32 ? 4 : 2) % ROUTE_BYTES<T, NV> == 0;
}

template <int T, int G, int NV>
static cudaError_t route_t(const RouteArgs &a, int grid, int warps, cudaStream_t s)
{
    auto k = route_vec<T, NV>(a.E) ? route_kernel<T, G, NV, true> : route_kernel<T, G, NV, false>;
    if (grid > 0) {                                            // without tokens: zeros
        const cudaError_t e = launch_k(k, dim3((unsigned)grid), dim3((unsigned)(32 * warps)), 0, s, a);
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
static cudaError_t route_e(const RouteArgs &a, int grid, int sms, cudaStream_t s)
{
    const RouteShape h = route_shape(a.E, a.top);
    const int w = route_warps(a.T, h, sms);
    if (h.lanes == 8) {
        if (h.each == 4) return route_t<T, 8, 4>(a, grid, w, s);
        if (h.each == 8) return route_t<T, 8, 8>(a, grid, w, s);
        return route_t<T, 8, 16>(a, grid, w, s);
    }
    if (h.lanes == 16) {
        if (h.each == 4) return route_t<T, 16, 4>(a, grid, w, s);
        if (h.each == 8) return route_t<T, 16, 8>(a, grid, w, s);
        return route_t<T, 16, 16>(a, grid, w, s);
    }
    return h.each == 8 ? route_t<T, 32, 8>(a, grid, w, s) : route_t<T, 32, 16>(a, grid, w, s);
}

template <int T>
static cudaError_t route_backward_e(const RouteBackwardArgs &a, int sms, cudaStream_t s)
{
    if (a.E <= 32) return route_backward_t<T, 8, 4>(a, route_ctas(a.T, 8, ROUTE_WARPS, 4 * sms), s);
    if (a.E <= 64) return route_backward_t<T, 8, 8>(a, route_ctas(a.T, 8, ROUTE_WARPS, 4 * sms), s);
    if (a.E <= 128) return route_backward_t<T, 16, 8>(a, route_ctas(a.T, 16, ROUTE_WARPS, 4 * sms), s);
    if (a.E <= 256) return route_backward_t<T, 32, 8>(a, route_ctas(a.T, 32, ROUTE_WARPS, 4 * sms), s);
    return route_backward_t<T, 32, 16>(a, route_ctas(a.T, 32, ROUTE_WARPS, 2 * sms), s);
}

cudaError_t launch_moe_route(const RouteArgs &a, int type, int grid, int sms, cudaStream_t s)
{
    if (type == IN_BF16) return route_e<IN_BF16>(a, grid, sms, s);
    if (type == IN_F16) return route_e<IN_F16>(a, grid, sms, s);
    return route_e<IN_F32>(a, grid, sms, s);
}

cudaError_t launch_moe_route_backward(const RouteBackwardArgs &a, int type, int sms, cudaStream_t s)
{
    if (type == IN_BF16) return route_backward_e<IN_BF16>(a, sms, s);
    if (type == IN_F16) return route_backward_e<IN_F16>(a, sms, s);
    return route_backward_e<IN_F32>(a, sms, s);
}

}  // namespace mmact
