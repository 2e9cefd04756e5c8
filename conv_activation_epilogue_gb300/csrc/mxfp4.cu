// mxfp4.cu -- quantisation to the 4-bit microscaled format and back: streaming
// kernels, bound by HBM (2 or 4 bytes read and 0.53 written per value, and the
// other way round).  Measured on 8192 x 8192, three inputs in turn: bf16 row-major 26.4
// us (6.4 TB/s), transposed 30.5, the way back 27.8; fp32 61.8 (a lane's 128 bytes in
// eight loads; 4.9 TB/s), 47.4 and 60.1.  Transposed with an odd number of rows, by
// single 16-bit values: 8191 x 8192 bf16 56.
#include <type_traits>

#include "common.cuh"
#include "kernels_mx.h"
#include "mxfp4.cuh"

namespace mmact {

template <int T>
__device__ __forceinline__ void store1(void *p, int64_t i, float v)
{
    if constexpr (T == IN_F32) static_cast<float *>(p)[i] = v;
    else if constexpr (T == IN_BF16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<__half *>(p)[i] = __float2half_rn(v);
}

// x [rows, K] row-major.  A lane takes one block of 32 values: its loads (64 or
// 128 consecutive bytes) are all in flight before the first is used, the largest
// |x| needs no other lane, and 32 lanes write 512 consecutive bytes of codes.
// 2^lanes_log2 consecutive lanes take the blocks of a row; rows past the last
// one, up to a multiple of 128, only get their zero scales.
template <int T, bool VEC>
__global__ void __launch_bounds__(256) quantize_kernel(const void *x, uint8_t *codes,
                                                       uint8_t *scales, int64_t rows, int64_t K,
                                                       int lanes_log2, int segs)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int64_t tiles = mx_tiles(K), kb = mx_blocks(K), padded = (rows + 127) & ~(int64_t)127;
    const int64_t rb = blockIdx.x / segs;
    const int seg = (int)(blockIdx.x - rb * segs);
    const int64_t row = (rb << (8 - lanes_log2)) + (threadIdx.x >> lanes_log2);
    const int64_t blk = ((int64_t)seg << lanes_log2) + (threadIdx.x & ((1 << lanes_log2) - 1)), k0 = blk * 32;
    Raw8<T> r[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < Raw8<T>::WORDS; ++j) r[q].w[j] = 0;
    if (row < rows && blk < kb) {
        const int n = (int)min((int64_t)32, K - k0);
        if constexpr (VEC) {
#pragma unroll
            for (int q = 0; q < 4; ++q) load8<T, true>(x, row * K + k0 + 8 * q, n - 8 * q, r[q]);
        } else {
            load32_any<T>(x, row * K + k0, n, rows * K, r);
        }
    }
    uint32_t amax = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < Raw8<T>::WORDS; ++j) amax = raw_max<T>(amax, r[q].w[j]);
    if constexpr (T != IN_F32) amax = bits_of<T>(max(amax & 0xffffu, amax >> 16));
    const uint32_t b = mx_scale_byte(amax);
    const float inv = mx_inv_scale(b == 255u ? 0u : b);
    uint32_t c[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) c[q] = b == 255u ? 0u : raw_encode<T>(r[q].w, inv);
    if (row < rows && blk < kb) *reinterpret_cast<uint4 *>(codes + (row * kb + blk) * 16) = make_uint4(c[0], c[1], c[2], c[3]);
    uint32_t word = b << (8 * (threadIdx.x & 3));              // blocks that do not exist hold zeros: byte 0
    word |= __shfl_xor_sync(0xffffffffu, word, 1);
    word |= __shfl_xor_sync(0xffffffffu, word, 2);
    if ((threadIdx.x & 3) == 0 && (blk >> 2) < tiles && row < padded)
        *reinterpret_cast<uint32_t *>(scales + mx_scale_at(row, blk, tiles)) = word;
}

// x [K, rows] row-major, blocks along K (the right operand of a row-major
// product).  A warp takes one block of 32 k and 64 columns, two to a lane: 32
// coalesced loads in flight, each column's largest |x| and codes in the lane.
// The eight warps of a CTA take eight consecutive blocks, and the codes go
// through shared memory so that each row's 128 bytes are written together.
template <int T, bool VEC>
__global__ void __launch_bounds__(256) quantize_trans_kernel(const void *x, uint8_t *codes,
                                                             uint8_t *scales, int64_t rows, int64_t K,
                                                             int col_tiles)
{
    constexpr int WPP = T == IN_F32 ? 2 : 1;                   // words of a pair of columns
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    __shared__ uint32_t sc[64][33];       // [row][8 blocks x 4 words] (+1: the lanes' rows on other banks)
    __shared__ __align__(8) uint8_t ss[64][8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t kt = blockIdx.x / col_tiles;
    const int64_t c0 = (int64_t)(blockIdx.x - kt * col_tiles) * 64;
    const int64_t k0 = kt * 256 + warp * 32, col = c0 + 2 * lane;
    const int64_t tiles = mx_tiles(K), kb = mx_blocks(K);
    uint32_t a[32 * WPP];
    if (VEC && c0 + 64 <= rows && k0 + 32 <= K) {              // a whole tile: the same for the warp
        const char *p = static_cast<const char *>(x) + (k0 * rows + col) * (T == IN_F32 ? 4 : 2);
        const int64_t pitch = rows * (T == IN_F32 ? 4 : 2);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if constexpr (T == IN_F32) {
                const uint2 f = __ldcs(reinterpret_cast<const uint2 *>(p + j * pitch));
                a[2 * j] = f.x, a[2 * j + 1] = f.y;
            } else {
                a[j] = __ldcs(reinterpret_cast<const uint32_t *>(p + j * pitch));
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const int64_t i = (k0 + j) * rows + col;
            const bool in0 = k0 + j < K && col < rows, in1 = k0 + j < K && col + 1 < rows;
            if constexpr (T == IN_F32) {
                a[2 * j] = in0 ? static_cast<const uint32_t *>(x)[i] : 0u;
                a[2 * j + 1] = in1 ? static_cast<const uint32_t *>(x)[i + 1] : 0u;
            } else {
                a[j] = in0 ? static_cast<const uint16_t *>(x)[i] : 0u;
                if (in1) a[j] |= (uint32_t) static_cast<const uint16_t *>(x)[i + 1] << 16;
            }
        }
    }
    uint32_t m[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        m[0] = raw_max<T>(m[0], a[WPP * j]);
        if constexpr (T == IN_F32) m[1] = raw_max<T>(m[1], a[2 * j + 1]);
    }
    if constexpr (T != IN_F32) {
        m[1] = bits_of<T>(m[0] >> 16);
        m[0] = bits_of<T>(m[0] & 0xffffu);
    }
    const uint32_t b0 = mx_scale_byte(m[0]), b1 = mx_scale_byte(m[1]);
    const float inv0 = mx_inv_scale(b0 == 255u ? 0u : b0), inv1 = mx_inv_scale(b1 == 255u ? 0u : b1);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float v[8], w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (T == IN_F32) {
                v[j] = __uint_as_float(a[2 * (8 * q + j)]) * inv0;
                w[j] = __uint_as_float(a[2 * (8 * q + j) + 1]) * inv1;
            } else {
                const float2 f = unpack2<T>(a[8 * q + j]);
                v[j] = f.x * inv0;
                w[j] = f.y * inv1;
            }
        }
        sc[2 * lane][warp * 4 + q] = b0 == 255u ? 0u : mx_encode8(v);
        sc[2 * lane + 1][warp * 4 + q] = b1 == 255u ? 0u : mx_encode8(w);
    }
    ss[2 * lane][warp] = (uint8_t)b0;
    ss[2 * lane + 1][warp] = (uint8_t)b1;
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

// codes and scales -> y [rows, K].  Sixteen lanes take one row's 128 values, 8 to a
// lane; a block of 256 threads covers `tpr` tiles (a power of two, at most 16) of
// 16 / tpr rows, U times (U sets of loads in flight).
template <int T, bool VEC, int U>
__global__ void __launch_bounds__(256) dequantize_kernel(const uint8_t *codes,
                                                         const uint8_t *scales, void *y,
                                                         int64_t rows, int64_t K, int tpr_log2, int segs)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int unit = threadIdx.x >> 4, l = threadIdx.x & 15;
    const int64_t rb = blockIdx.x / segs;
    const int seg = (int)(blockIdx.x - rb * segs);
    const int64_t tiles = mx_tiles(K), kb = mx_blocks(K);
    const int per = 16 >> tpr_log2;
    const int64_t row0 = rb * (per * U) + (unit >> tpr_log2);
    const int64_t tile = ((int64_t)seg << tpr_log2) + (unit & ((1 << tpr_log2) - 1));
    const int64_t k0 = tile * 128 + l * 8;
    if (VEC && k0 >= K) return;
    uint32_t c[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t row = row0 + u * per;
        c[u] = b[u] = 0;
        if (row >= rows || k0 >= K) continue;
        c[u] = __ldcs(reinterpret_cast<const uint32_t *>(codes + row * (kb * 16) + tile * 64 + l * 4));
        b[u] = scales[mx_scale_at(row, tile * 4 + (l >> 2), tiles)];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t row = row0 + u * per;
        if (VEC && row >= rows) break;
        const float s = mx_scale(b[u]);
        float v[8];
        mx_decode8(c[u], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= s;
        const int64_t i = row * K + k0;
        if constexpr (!VEC) {
            // Rows that begin anywhere: through shared memory, so that 16 lanes write consecutive words (eight values
            // a lane, one by one: 5447 x 3659 bf16 57 us, so 13.8).
            using E = std::conditional_t<T == IN_F32, uint32_t, uint16_t>;
            __shared__ __align__(16) E stage[16][128];
            E *line = stage[unit];
#pragma unroll
            for (int j = 0; j < 8; ++j) store1<T>(line, l * 8 + j, v[j]);
            __syncwarp();
            const int n = row < rows ? (int)min((int64_t)128, K - tile * 128) : 0;
            const int64_t i0 = i - l * 8;
            E *out = static_cast<E *>(y) + i0;
            if constexpr (T == IN_F32) {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (q * 16 + l < n) __stcs(out + q * 16 + l, line[q * 16 + l]);
            } else {
                const int odd = (int)(i0 & 1);                 // pairs of values at even offsets
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int e = odd + 2 * (q * 16 + l);
                    if (e + 1 < n) __stcs(reinterpret_cast<uint32_t *>(out + e), line[e] | ((uint32_t)line[e + 1] << 16));
                }
                if (l == 0 && odd != 0 && n > 0) out[0] = line[0];
                if (l == 1 && n > odd && ((n - odd) & 1) != 0) out[n - 1] = line[n - 1];
            }
            __syncwarp();
        } else if (k0 + 8 <= K) {
            if constexpr (T == IN_F32) {
                float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(y) + i);
                __stcs(p, make_float4(v[0], v[1], v[2], v[3]));
                __stcs(p + 1, make_float4(v[4], v[5], v[6], v[7]));
            } else {
                uint4 w;
                w.x = pack2<T>(v[0], v[1]);
                w.y = pack2<T>(v[2], v[3]);
                w.z = pack2<T>(v[4], v[5]);
                w.w = pack2<T>(v[6], v[7]);
                __stcs(reinterpret_cast<uint4 *>(static_cast<uint16_t *>(y) + i), w);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (k0 + j < K) store1<T>(y, i + j, v[j]);
        }
    }
}

// The grid of dequantize_kernel: a CTA takes as many of a row's tiles as it has, up to
// 16, and U sets of rows; U = 4 once that still leaves four CTAs for each SM, so that
// small calls spread over more SMs and large ones keep more loads in flight.
struct RowGrid {
    int tpr_log2, segs, u;
    int64_t grid;
};

static RowGrid row_grid(int64_t rows, int64_t K, int sms)
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
    // a CTA: the blocks of a row (whole tiles) on a power of two of its 256 lanes
    const int64_t blocks = mx_tiles(K) * 4;
    int lanes_log2 = 2;
    while (lanes_log2 < 8 && (1 << lanes_log2) < blocks) ++lanes_log2;
    const int64_t segs = (blocks + (1 << lanes_log2) - 1) >> lanes_log2, per = 256 >> lanes_log2;
    const int64_t grid = (padded + per - 1) / per * segs;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    auto k = K * e % 16 == 0 ? quantize_kernel<T, true> : quantize_kernel<T, false>;
    return launch_k(k, dim3((unsigned)grid), dim3(256), 0, s, x, codes, scales, rows, K, lanes_log2, (int)segs);
}

template <int T>
static cudaError_t dequantize_t(const uint8_t *codes, const uint8_t *scales, void *y, int64_t rows, int64_t K, int sms,
                                cudaStream_t s)
{
    const int e = T == IN_F32 ? 4 : 2;
    const RowGrid g = row_grid(rows, K, sms);
    if (g.grid > INT32_MAX) return cudaErrorInvalidValue;
    const bool vec = K * e % 16 == 0;
    auto k = g.u == 4 ? (vec ? dequantize_kernel<T, true, 4> : dequantize_kernel<T, false, 4>)
                      : (vec ? dequantize_kernel<T, true, 1> : dequantize_kernel<T, false, 1>);
    return launch_k(k, dim3((unsigned)g.grid), dim3(256), 0, s, codes, scales, y, rows, K, g.tpr_log2, g.segs);
}

template <int T>
__global__ void __launch_bounds__(256) mx_bias_act_kernel(const float *bias, void *out,
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
                                    int64_t K, int sms, cudaStream_t s)
{
    if (type == IN_BF16) return dequantize_t<IN_BF16>(codes, scales, y, rows, K, sms, s);
    if (type == IN_F16) return dequantize_t<IN_F16>(codes, scales, y, rows, K, sms, s);
    return dequantize_t<IN_F32>(codes, scales, y, rows, K, sms, s);
}

}  // namespace mmact
