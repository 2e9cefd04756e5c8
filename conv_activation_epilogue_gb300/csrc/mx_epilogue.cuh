// mx_epilogue.cuh -- the epilogue of the CTA-pair products of microscaled operands:
// accumulators from tensor memory, bias, activation, conversion, the output's stores.
#pragma once

#include <cstdint>

#include "common.cuh"
#include "mxfp4.cuh"

namespace mmact {

// One epilogue unit: this warp's 32 rows x one 128-byte row segment (32 fp32 or
// 64 16-bit columns): accumulators from TMEM, + bias, activation, conversion,
// into a 32 x 128 B buffer in the 128-byte swizzled order of a TMA store.
// `loaded` is called when the accumulators are in registers.
template <int OUT, int ACT, typename Loaded>
__device__ __forceinline__ void mx_epi_unit(uint32_t taddr, const float *bias, int nvalid, float alpha, uint32_t buf,
                                            int lane, Loaded loaded)
{
    constexpr int HALVES = OUT == OUT_F32 ? 1 : 2;           // 32 columns at a time
    uint32_t r[HALVES][32];
#pragma unroll
    for (int h = 0; h < HALVES; ++h) ptx::tmem_ld32(taddr + 32 * h, r[h]);
#pragma unroll
    for (int h = 0; h < HALVES; ++h) ptx::tmem_ld_wait(r[h]);
    loaded();
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
        float b[32] = {};
        const float *src = bias + 32 * h;
        if (bias != nullptr) {
            if (nvalid >= 32 * (h + 1) && (reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(src + j);
                    b[j] = f.x, b[j + 1] = f.y, b[j + 2] = f.z, b[j + 3] = f.w;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (32 * h + j < nvalid) b[j] = src[j];
            }
        }
        const uint32_t row = buf + (uint32_t)lane * 128u, sw = (uint32_t)(lane & 7);
        constexpr int PER = OUT == OUT_F32 ? 4 : 8;           // values per 16 bytes
#pragma unroll
        for (int c = 0; c < 32 / PER; ++c) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (OUT == OUT_F32) {
                    const int j = 4 * c + e;
                    w[e] = __float_as_uint(act_mx<ACT>(__uint_as_float(r[h][j]) + b[j], alpha));
                } else {
                    const int j = 8 * c + 2 * e;
                    w[e] = pack2<OUT>(act_mx<ACT>(__uint_as_float(r[h][j]) + b[j], alpha),
                                      act_mx<ACT>(__uint_as_float(r[h][j + 1]) + b[j + 1], alpha));
                }
            }
            ptx::st_shared_v4(row + (((uint32_t)(c + h * (32 / PER)) ^ sw) << 4), w[0], w[1], w[2], w[3]);
        }
    }
}

template <int OUT, typename Loaded>
__device__ __forceinline__ void mx_epi_unit(int act, uint32_t taddr, const float *bias, int nvalid, float alpha,
                                            uint32_t buf, int lane,
                                            Loaded loaded)
{
    switch (act) {
    case ACT_RELU: mx_epi_unit<OUT, ACT_RELU>(taddr, bias, nvalid, alpha, buf, lane, loaded); break;
    case ACT_LEAKY: mx_epi_unit<OUT, ACT_LEAKY>(taddr, bias, nvalid, alpha, buf, lane, loaded); break;
    case ACT_TANH: mx_epi_unit<OUT, ACT_TANH>(taddr, bias, nvalid, alpha, buf, lane, loaded); break;
    case ACT_SIGMOID: mx_epi_unit<OUT, ACT_SIGMOID>(taddr, bias, nvalid, alpha, buf, lane, loaded); break;
    case ACT_GELU: mx_epi_unit<OUT, ACT_GELU>(taddr, bias, nvalid, alpha, buf, lane, loaded); break;
    case ACT_SILU: mx_epi_unit<OUT, ACT_SILU>(taddr, bias, nvalid, alpha, buf, lane, loaded); break;
    default: mx_epi_unit<OUT, ACT_NONE>(taddr, bias, nvalid, alpha, buf, lane, loaded); break;
    }
}

// Element stores of a staged unit (32 rows of 128 bytes in the swizzled order)
// for outputs whose row pitch TMA cannot address.
template <int OUT>
__device__ __forceinline__ void mx_store_elements(void *C, uint32_t buf, int row0, int col0, int M, int N, int lane)
{
    constexpr int ESZ = OUT == OUT_F32 ? 4 : 2, COLS = 128 / ESZ;
    for (int r = 0; r < 32 && row0 + r < M; ++r)
#pragma unroll
        for (int c = lane; c < COLS; c += 32) {
            if (col0 + c >= N) continue;
            const uint32_t b = (uint32_t)c * ESZ;
            const uint32_t at = buf + r * 128u + (((b >> 4) ^ (r & 7)) << 4) + (b & 15u);
            const int64_t i = (int64_t)(row0 + r) * N + col0 + c;
            if constexpr (OUT == OUT_F32) {
                uint32_t v;
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
                static_cast<uint32_t *>(C)[i] = v;
            } else {
                uint16_t v;
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
                static_cast<uint16_t *>(C)[i] = v;
            }
        }
}

}  // namespace mmact
