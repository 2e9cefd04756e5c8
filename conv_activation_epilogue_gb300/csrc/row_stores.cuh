// row_stores.cuh -- how the dequantisations lay rows of 128-value lines over CTAs and
// store them.
#pragma once

#include <cstdint>
#include <type_traits>

#include "mxfp4.cuh"

namespace mmact {

template <int T>
__device__ __forceinline__ void store1(void *p, int64_t i, float v)
{
    if constexpr (T == IN_F32) static_cast<float *>(p)[i] = v;
    else if constexpr (T == IN_BF16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<__half *>(p)[i] = __float2half_rn(v);
}

// 128 consecutive values (the first n of them) that begin anywhere, i0 values into y, eight
// to each of 16 lanes, `unit` the lanes' number in the block of 256 threads: through
// shared memory, so that the lanes write consecutive words (eight values a lane, one by
// one: 5447 x 3659 bf16 57 us, so 13.8).  Called by whole warps.
template <int T>
__device__ __forceinline__ void store_line_any(void *y, int64_t i0, int n, const float (&v)[8], int unit, int l)
{
    using E = std::conditional_t<T == IN_F32, uint32_t, uint16_t>;
    __shared__ __align__(16) E stage[16][128];
    E *line = stage[unit];
#pragma unroll
    for (int j = 0; j < 8; ++j) store1<T>(line, l * 8 + j, v[j]);
    __syncwarp();
    E *out = static_cast<E *>(y) + i0;
    if constexpr (T == IN_F32) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (q * 16 + l < n) __stcs(out + q * 16 + l, line[q * 16 + l]);
    } else {
        const int odd = (int)(i0 & 1);                         // pairs of values at even offsets
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int e = odd + 2 * (q * 16 + l);
            if (e + 1 < n) __stcs(reinterpret_cast<uint32_t *>(out + e), line[e] | ((uint32_t)line[e + 1] << 16));
        }
        if (l == 0 && odd != 0 && n > 0) out[0] = line[0];
        if (l == 1 && n > odd && ((n - odd) & 1) != 0) out[n - 1] = line[n - 1];
    }
    __syncwarp();
}

// The grid of a dequantisation: a CTA takes as many of a row's tiles as it has, up to
// 16, and U sets of rows; U = 4 once that still leaves four CTAs for each SM, so that
// small calls spread over more SMs and large ones keep more loads in flight.
struct RowGrid {
    int tpr_log2, segs, u;
    int64_t grid;
};

[[maybe_unused]] static RowGrid row_grid(int64_t rows, int64_t K, int sms)
{
    const int64_t tiles = mx_tiles(K);
    RowGrid g;
    g.tpr_log2 = 0;
    while (g.tpr_log2 < 4 && (1 << g.tpr_log2) < tiles) ++g.tpr_log2;
    g.segs = (int)((tiles + (1 << g.tpr_log2) - 1) >> g.tpr_log2);
    const int64_t per = 16 >> g.tpr_log2;
    g.u = (rows + per * 4 - 1) / (per * 4) * g.segs >= 4 * sms ? 4 : 1;
    g.grid = (rows + per * g.u - 1) / (per * g.u) * g.segs;
    return g;
}

}  // namespace mmact
