// mxfp4.cu -- quantisation to the 4-bit microscaled format and back: streaming
// kernels, bound by HBM (2 or 4 bytes read and 0.53 written per value, and the
// other way round).
#include "common.cuh"
#include "kernels_mx.h"
#include "mxfp4.cuh"

namespace mmact {

enum : int { IN_F32 = OUT_F32, IN_F16 = OUT_F16, IN_BF16 = OUT_BF16 };

template <int T>
__device__ __forceinline__ float load1(const void *p, int64_t i)
{
    if constexpr (T == IN_F32) return static_cast<const float *>(p)[i];
    else if constexpr (T == IN_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
    else return __half2float(static_cast<const __half *>(p)[i]);
}

template <int T>
__device__ __forceinline__ void store1(void *p, int64_t i, float v)
{
    if constexpr (T == IN_F32) static_cast<float *>(p)[i] = v;
    else if constexpr (T == IN_BF16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<__half *>(p)[i] = __float2half_rn(v);
}

// Eight consecutive values x[i..i+8) (those at or past `n` are 0).
template <int T, bool VEC>
__device__ __forceinline__ void load8(const void *x, int64_t i, int n, float (&v)[8])
{
    if (VEC && n >= 8) {
        if constexpr (T == IN_F32) {
            const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(x) + i);
            const float4 a = __ldcs(p), b = __ldcs(p + 1);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
            v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
            const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x) + i));
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = unpack2<T>(w[j]);
                v[2 * j] = f.x;
                v[2 * j + 1] = f.y;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < n ? load1<T>(x, i + j) : 0.0f;
    }
}

// x [rows, K] row-major.  Sixteen lanes take one row's 128 values (one scale
// word): each lane 8 values, four lanes a block, whose largest |x| they find by
// two shuffles.  A block of 256 threads covers `tpr` tiles (a power of two, at
// most 16) of 16 / tpr rows; rows past the last one, up to a multiple of 128,
// only get their zero scales.
template <int T, bool VEC>
__global__ void __launch_bounds__(256) quantize_kernel(const void *__restrict__ x, uint8_t *__restrict__ codes,
                                                       uint8_t *__restrict__ scales, int64_t rows, int64_t K,
                                                       int tpr_log2, int segs)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int unit = threadIdx.x >> 4, l = threadIdx.x & 15;
    const int64_t rb = blockIdx.x / segs;
    const int seg = (int)(blockIdx.x - rb * segs);
    const int64_t tiles = mx_tiles(K), kb = mx_blocks(K);
    const int64_t row = (rb << (4 - tpr_log2)) + (unit >> tpr_log2);
    const int64_t tile = ((int64_t)seg << tpr_log2) + (unit & ((1 << tpr_log2) - 1));
    const int64_t k0 = tile * 128 + l * 8;
    float v[8] = {};
    uint32_t amax = 0;
    if (row < rows && k0 < K) {
        load8<T, VEC>(x, row * K + k0, (int)min((int64_t)8, K - k0), v);
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(v[j]) & 0x7fffffffu);
    }
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const uint32_t b = mx_scale_byte(amax);
    const float inv = mx_inv_scale(b == 255u ? 0u : b);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= inv;
    const uint32_t c = b == 255u ? 0u : mx_encode8(v);
    if (row < rows && k0 < kb * 32)
        *reinterpret_cast<uint32_t *>(codes + row * (kb * 16) + tile * 64 + l * 4) = c;
    uint32_t word = b << (8 * (l >> 2));
    word |= __shfl_xor_sync(0xffffffffu, word, 4);
    word |= __shfl_xor_sync(0xffffffffu, word, 8);
    if (l == 0 && tile < tiles && row < ((rows + 127) & ~(int64_t)127))
        *reinterpret_cast<uint32_t *>(scales + mx_scale_at(row, tile * 4, tiles)) = word;
}

// x [K, rows] row-major, blocks along K (the right operand of a row-major
// product).  A warp takes one block of 32 k and 64 columns, two to a lane: 32
// coalesced loads, each column's largest |x| and codes in the lane.  The eight
// warps of a CTA take eight consecutive blocks, and the codes go through shared
// memory so that each row's 128 bytes are written together.
template <int T, bool VEC>
__global__ void __launch_bounds__(256) quantize_trans_kernel(const void *__restrict__ x, uint8_t *__restrict__ codes,
                                                             uint8_t *__restrict__ scales, int64_t rows, int64_t K,
                                                             int col_tiles)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    __shared__ uint32_t sc[64][33];       // [row][8 blocks x 4 words] (+1: the lanes' rows on other banks)
    __shared__ __align__(8) uint8_t ss[64][8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t kt = blockIdx.x / col_tiles;
    const int64_t c0 = (int64_t)(blockIdx.x - kt * col_tiles) * 64;
    const int64_t k0 = kt * 256 + warp * 32, col = c0 + 2 * lane;
    const int64_t tiles = mx_tiles(K), kb = mx_blocks(K);
    float a[32], d[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        a[j] = d[j] = 0.0f;
        if (k0 + j < K) {
            const int64_t i = (k0 + j) * rows + col;
            if (VEC && col + 1 < rows) {
                if constexpr (T == IN_F32) {
                    const float2 f = __ldcs(reinterpret_cast<const float2 *>(static_cast<const float *>(x) + i));
                    a[j] = f.x, d[j] = f.y;
                } else {
                    const float2 f = unpack2<T>(
                        __ldcs(reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(x) + i)));
                    a[j] = f.x, d[j] = f.y;
                }
            } else {
                if (col < rows) a[j] = load1<T>(x, i);
                if (col + 1 < rows) d[j] = load1<T>(x, i + 1);
            }
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t amax = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) amax = max(amax, __float_as_uint(h ? d[j] : a[j]) & 0x7fffffffu);
        const uint32_t b = mx_scale_byte(amax);
        const float inv = mx_inv_scale(b == 255u ? 0u : b);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = (h ? d[8 * q + j] : a[8 * q + j]) * inv;
            sc[2 * lane + h][warp * 4 + q] = b == 255u ? 0u : mx_encode8(v);
        }
        ss[2 * lane + h][warp] = (uint8_t)b;
    }
    __syncthreads();
    // codes: 4 bytes to a thread, a warp writes 128 bytes of one row at a time
    const int64_t word0 = kt * 32;                           // first 4-byte word of the row's segment
#pragma unroll
    for (int r = warp; r < 64; r += 8)
        if (c0 + r < rows && word0 + lane < kb * 4)
            *reinterpret_cast<uint32_t *>(codes + (c0 + r) * (kb * 16) + (word0 + lane) * 4) = sc[r][lane];
    // scales: two words (8 blocks) a row; rows up to a multiple of 128 exist in the tiles
    if (threadIdx.x < 128) {
        const int r = threadIdx.x >> 1, w = threadIdx.x & 1;
        const int64_t tile = kt * 2 + w;
        if (tile < tiles && c0 + r < ((rows + 127) & ~(int64_t)127))
            *reinterpret_cast<uint32_t *>(scales + mx_scale_at(c0 + r, tile * 4, tiles)) =
                *reinterpret_cast<const uint32_t *>(&ss[r][w * 4]);
    }
}

// codes and scales -> y [rows, K]; the same lanes as quantize_kernel.
template <int T, bool VEC>
__global__ void __launch_bounds__(256) dequantize_kernel(const uint8_t *__restrict__ codes,
                                                         const uint8_t *__restrict__ scales, void *__restrict__ y,
                                                         int64_t rows, int64_t K, int tpr_log2, int segs)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int unit = threadIdx.x >> 4, l = threadIdx.x & 15;
    const int64_t rb = blockIdx.x / segs;
    const int seg = (int)(blockIdx.x - rb * segs);
    const int64_t tiles = mx_tiles(K), kb = mx_blocks(K);
    const int64_t row = (rb << (4 - tpr_log2)) + (unit >> tpr_log2);
    const int64_t tile = ((int64_t)seg << tpr_log2) + (unit & ((1 << tpr_log2) - 1));
    const int64_t k0 = tile * 128 + l * 8;
    if (row >= rows || k0 >= K) return;
    const uint32_t c = *reinterpret_cast<const uint32_t *>(codes + row * (kb * 16) + tile * 64 + l * 4);
    const float s = mx_scale(scales[mx_scale_at(row, tile * 4 + (l >> 2), tiles)]);
    float v[8];
    mx_decode8(c, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= s;
    const int64_t i = row * K + k0;
    if (VEC && k0 + 8 <= K) {
        if constexpr (T == IN_F32) {
            float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(y) + i);
            __stcs(p, make_float4(v[0], v[1], v[2], v[3]));
            __stcs(p + 1, make_float4(v[4], v[5], v[6], v[7]));
        } else {
            uint4 u;
            u.x = pack2<T>(v[0], v[1]);
            u.y = pack2<T>(v[2], v[3]);
            u.z = pack2<T>(v[4], v[5]);
            u.w = pack2<T>(v[6], v[7]);
            __stcs(reinterpret_cast<uint4 *>(static_cast<uint16_t *>(y) + i), u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (k0 + j < K) store1<T>(y, i + j, v[j]);
    }
}

// Rows and tiles of one CTA of the row kernels: as many of a row's tiles as it has, up to 16.
struct RowGrid {
    int tpr_log2, segs;
    int64_t grid;
};

static RowGrid row_grid(int64_t rows, int64_t K)
{
    const int64_t tiles = mx_tiles(K);
    RowGrid g;
    g.tpr_log2 = 0;
    while (g.tpr_log2 < 4 && (1 << g.tpr_log2) < tiles) ++g.tpr_log2;
    g.segs = (int)((tiles + (1 << g.tpr_log2) - 1) >> g.tpr_log2);
    const int64_t per = 16 >> g.tpr_log2;
    g.grid = (rows + per - 1) / per * g.segs;
    return g;
}

template <int T>
static cudaError_t quantize_t(const void *x, uint8_t *codes, uint8_t *scales, int64_t rows, int64_t K, bool trans,
                              cudaStream_t s)
{
    const int e = T == IN_F32 ? 4 : 2;
    const int64_t padded = (rows + 127) & ~(int64_t)127;
    if (trans) {
        const int64_t col_tiles = padded / 64, grid = (K + 255) / 256 * col_tiles;
        if (grid > INT32_MAX) return cudaErrorInvalidValue;
        auto k = rows % 2 == 0 ? quantize_trans_kernel<T, true> : quantize_trans_kernel<T, false>;
        return launch_k(k, dim3((unsigned)grid), dim3(256), 0, s, x, codes, scales, rows, K, (int)col_tiles);
    }
    const RowGrid g = row_grid(padded, K);
    if (g.grid > INT32_MAX) return cudaErrorInvalidValue;
    auto k = K * e % 16 == 0 ? quantize_kernel<T, true> : quantize_kernel<T, false>;
    return launch_k(k, dim3((unsigned)g.grid), dim3(256), 0, s, x, codes, scales, rows, K, g.tpr_log2, g.segs);
}

template <int T>
static cudaError_t dequantize_t(const uint8_t *codes, const uint8_t *scales, void *y, int64_t rows, int64_t K,
                                cudaStream_t s)
{
    const int e = T == IN_F32 ? 4 : 2;
    const RowGrid g = row_grid(rows, K);
    if (g.grid > INT32_MAX) return cudaErrorInvalidValue;
    auto k = K * e % 16 == 0 ? dequantize_kernel<T, true> : dequantize_kernel<T, false>;
    return launch_k(k, dim3((unsigned)g.grid), dim3(256), 0, s, codes, scales, y, rows, K, g.tpr_log2, g.segs);
}

template <int T>
__global__ void __launch_bounds__(256) mx_bias_act_kernel(const float *__restrict__ bias, void *__restrict__ out,
                                                          int64_t rows, int64_t cols, int act, float alpha)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int64_t total = rows * cols, stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += stride)
        store1<T>(out, i, act_mx(act, bias == nullptr ? 0.0f : bias[i % cols], alpha));
}

cudaError_t launch_mx_bias_act(const float *bias, void *out, int64_t rows, int64_t cols, int out_kind, int act,
                               float alpha, cudaStream_t s)
{
    const int64_t blocks = (rows * cols + 255) / 256;
    const dim3 grid((unsigned)(blocks < 4096 ? blocks : 4096));
    auto k = out_kind == OUT_BF16 ? mx_bias_act_kernel<OUT_BF16>
                                  : (out_kind == OUT_F16 ? mx_bias_act_kernel<OUT_F16> : mx_bias_act_kernel<OUT_F32>);
    return launch_k(k, grid, dim3(256), 0, s, bias, out, rows, cols, act, alpha);
}

cudaError_t launch_quantize_mxfp4(const void *x, int type, uint8_t *codes, uint8_t *scales, int64_t rows, int64_t K,
                                  bool trans, cudaStream_t s)
{
    if (type == IN_BF16) return quantize_t<IN_BF16>(x, codes, scales, rows, K, trans, s);
    if (type == IN_F16) return quantize_t<IN_F16>(x, codes, scales, rows, K, trans, s);
    return quantize_t<IN_F32>(x, codes, scales, rows, K, trans, s);
}

cudaError_t launch_dequantize_mxfp4(const uint8_t *codes, const uint8_t *scales, void *y, int type, int64_t rows,
                                    int64_t K, cudaStream_t s)
{
    if (type == IN_BF16) return dequantize_t<IN_BF16>(codes, scales, y, rows, K, s);
    if (type == IN_F16) return dequantize_t<IN_F16>(codes, scales, y, rows, K, s);
    return dequantize_t<IN_F32>(codes, scales, y, rows, K, s);
}

}  // namespace mmact
