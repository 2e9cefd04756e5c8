// rows_epilogue.cuh -- the epilogue of the products of few rows: sums over a cluster's
// partial tiles, bias, activation, stores.
#pragma once

#include <cstdint>

#include "common.cuh"
#include "mxfp4.cuh"

namespace mmact {

// C[m0 + j][n] = z[j] for this lane's n and the rows that exist: element stores, a warp
// covering 32 consecutive n.
template <int OUT, int CH, typename Args>
__device__ __forceinline__ void rows_write(const Args &p, int m0, int n, const float (&z)[CH])
{
    if (n >= p.N) return;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        if (m0 + j >= p.M) break;
        const int64_t at = (int64_t)(m0 + j) * p.N + n;
        if constexpr (OUT == OUT_F32) static_cast<float *>(p.C)[at] = z[j];
        else if constexpr (OUT == OUT_BF16) static_cast<__nv_bfloat16 *>(p.C)[at] = __float2bfloat16_rn(z[j]);
        else static_cast<__half *>(p.C)[at] = __float2half_rn(z[j]);
    }
}

// act(z[j] + bias)
template <int CH, typename Args>
__device__ __forceinline__ void rows_activate(const Args &p, float (&z)[CH], float bias)
{
#pragma unroll
    for (int j = 0; j < CH; ++j) z[j] += bias;
    act_mx_all(p.act, z, p.alpha);
}

template <int OUT, int CH, typename Args>
__device__ __forceinline__ void rows_store(const Args &p, int m0, int n, float (&z)[CH], float bias)
{
    rows_activate(p, z, bias);
    rows_write<OUT>(p, m0, n, z);
}

// The same with the output's type at run time.
template <int CH, typename Args>
__device__ __forceinline__ void rows_store(const Args &p, int out, int m0, int n, float (&z)[CH], float bias)
{
    rows_activate(p, z, bias);
    if (out == OUT_F32) rows_write<OUT_F32>(p, m0, n, z);
    else if (out == OUT_BF16) rows_write<OUT_BF16>(p, m0, n, z);
    else rows_write<OUT_F16>(p, m0, n, z);
}

// Sum of CH columns of the cluster's partial tiles at this thread's lane, in rank
// order: all loads of a rank in flight together.
template <int CH>
__device__ __forceinline__ void cluster_columns(uint32_t at, int split, float (&z)[CH])
{
#pragma unroll
    for (int j = 0; j < CH; ++j) z[j] = 0.0f;
#pragma unroll 2
    for (int s = 0; s < split; ++s) {
        const uint32_t from = ptx::mapa(at, (uint32_t)s);
        float v[CH];
#pragma unroll
        for (int j = 0; j < CH; ++j) v[j] = ptx::ld_cluster_f32(from + j * 512u);
#pragma unroll
        for (int j = 0; j < CH; ++j) z[j] += v[j];
    }
}

}  // namespace mmact
