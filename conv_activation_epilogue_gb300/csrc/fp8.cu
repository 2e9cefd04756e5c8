// fp8.cu -- quantisation to 8-bit floating point with a scale for each block of 128,
// and back: streaming kernels, bound by HBM (2 or 4 bytes read and 1.01 written per
// value, and the other way round).  Measured on 8192 x 8192 bf16, inputs in turn: rows to
// E4M3 29 us (7.0 TB/s, a part of the codes stays in L2), turned round in blocks of 128 x 128
// and back to values 62.6 (6.45 TB/s).
#include "common.cuh"
#include "fp8.cuh"
#include "kernels_fp8.h"
#include "row_stores.cuh"

namespace mmact {

// x [rows, K] row-major, blocks of one row.  A lane takes 32 values (its 64 or 128
// bytes of loads are all in flight before the first is used), four lanes a block.
// 2^lanes_log2 consecutive lanes take a row, whole scale tiles of it; rows past the
// last one, up to a multiple of 128, only get their zero scales.
template <int T, int F8, bool VEC>
__global__ void __launch_bounds__(256) quantize_f8_kernel(const void *x, uint8_t *codes, uint8_t *scales, int64_t rows,
                                                          int64_t K, int lanes_log2, int segs)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int64_t tiles = f8_tiles(K), pitch = f8_pitch(K), padded = (rows + 127) & ~(int64_t)127;
    const int64_t rb = blockIdx.x / segs;
    const int seg = (int)(blockIdx.x - rb * segs);
    const int64_t row = (rb << (8 - lanes_log2)) + (threadIdx.x >> lanes_log2);
    const int64_t part = ((int64_t)seg << lanes_log2) + (threadIdx.x & ((1 << lanes_log2) - 1)), k0 = part * 32;
    const int n = (int)max((int64_t)0, min((int64_t)32, K - k0));
    Raw8<T> r[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < Raw8<T>::WORDS; ++j) r[q].w[j] = 0;
    if (row < rows && n > 0) {
        const int64_t at = row * K + k0;
        if constexpr (VEC) {
#pragma unroll
            for (int q = 0; q < 4; ++q) load8<T, true>(x, at + 8 * q, n - 8 * q, r[q]);
        } else {
            load32_any<T>(x, at, n, rows * K, r);
        }
    }
    uint32_t amax = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < Raw8<T>::WORDS; ++j) amax = raw_max<T>(amax, r[q].w[j]);
    if constexpr (T != IN_F32) amax = max(amax & 0xffffu, amax >> 16);
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    if constexpr (T != IN_F32) amax = bits_of<T>(amax);
    const uint32_t b = f8_scale_byte<F8>(amax);
    const float inv = mx_inv_scale(b == 255u ? 0u : b);
    if (row < rows) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (k0 + 16 * h >= pitch) break;
            const uint2 u = f8_raw_encode<T, F8>(r[2 * h].w, inv), v = f8_raw_encode<T, F8>(r[2 * h + 1].w, inv);
            *reinterpret_cast<uint4 *>(codes + row * pitch + k0 + 16 * h) =
                b == 255u ? make_uint4(0, 0, 0, 0) : make_uint4(u.x, u.y, v.x, v.y);
        }
    }
    uint32_t word = b << (8 * ((threadIdx.x >> 2) & 3));       // blocks that do not exist hold zeros: byte 0
    word |= __shfl_xor_sync(0xffffffffu, word, 4);
    word |= __shfl_xor_sync(0xffffffffu, word, 8);
    if ((threadIdx.x & 15) == 0 && (part >> 4) < tiles && row < padded)
        *reinterpret_cast<uint32_t *>(scales + mx_scale_at(row, part >> 2, tiles)) = word;
}

// x [rows, K] row-major, blocks of 128 x 128: a block to a CTA, 32 values of a row to a
// thread.  A CTA past the last block of K writes its column's zero scales.
template <int T, int F8, bool VEC>
__global__ void __launch_bounds__(512) quantize_f8_square_kernel(const void *x, uint8_t *codes, uint8_t *scales, int64_t rows,
                                                                 int64_t K, int kbs)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    __shared__ uint32_t part[16];
    const int64_t tiles = f8_tiles(K), pitch = f8_pitch(K), rb = blockIdx.x / kbs;
    const int kb = (int)(blockIdx.x - rb * kbs);
    const int64_t row = rb * 128 + (threadIdx.x >> 2), k0 = (int64_t)kb * 128 + (threadIdx.x & 3) * 32;
    const int n = (int)max((int64_t)0, min((int64_t)32, K - k0));
    Raw8<T> r[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < Raw8<T>::WORDS; ++j) r[q].w[j] = 0;
    if (row < rows && n > 0) {
        const int64_t at = row * K + k0;
        if constexpr (VEC) {
#pragma unroll
            for (int q = 0; q < 4; ++q) load8<T, true>(x, at + 8 * q, n - 8 * q, r[q]);
        } else {
            load32_any<T>(x, at, n, rows * K, r);
        }
    }
    uint32_t amax = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < Raw8<T>::WORDS; ++j) amax = raw_max<T>(amax, r[q].w[j]);
    if constexpr (T != IN_F32) amax = max(amax & 0xffffu, amax >> 16);
    amax = __reduce_max_sync(0xffffffffu, amax);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 16; ++j) amax = max(amax, part[j]);
    if constexpr (T != IN_F32) amax = bits_of<T>(amax);
    const uint32_t b = f8_scale_byte<F8>(amax);
    const float inv = mx_inv_scale(b == 255u ? 0u : b);
    if (row < rows) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (k0 + 16 * h >= pitch) break;
            const uint2 u = f8_raw_encode<T, F8>(r[2 * h].w, inv), v = f8_raw_encode<T, F8>(r[2 * h + 1].w, inv);
            *reinterpret_cast<uint4 *>(codes + row * pitch + k0 + 16 * h) =
                b == 255u ? make_uint4(0, 0, 0, 0) : make_uint4(u.x, u.y, v.x, v.y);
        }
    }
    if ((threadIdx.x & 3) == 0) scales[mx_scale_at(row, kb, tiles)] = (uint8_t)(row < rows ? b : 0u);
}

// ------------------------------------------------------ tiles of 128 K x 128 columns --
// x [K, cols] row-major.  A CTA of 8 warps takes 128 K of 128 columns, a warp 32 K of 64
// columns, two to a lane: 32 coalesced loads in flight, values in registers as raw words.
template <int T>
constexpr int PAIR_WORDS = T == IN_F32 ? 2 : 1;                // words of a pair of columns

struct TileSmem {
    uint32_t codes[128][33];                                   // [column][32 words] (+1: the lanes' columns on other banks)
    uint32_t amax[4][128];
};

// `vec`: an even number of columns, so that pairs are aligned and whole.  Values that do
// not exist are 0.
template <int T>
__device__ __forceinline__ void load_pairs(const void *x, int64_t K, int64_t cols, int64_t k0, int64_t col, bool vec,
                                           uint32_t (&a)[32 * PAIR_WORDS<T>])
{
    constexpr int ES = T == IN_F32 ? 4 : 2;
    const char *p = static_cast<const char *>(x) + (k0 * cols + col) * ES;
    const int64_t line = cols * ES;
    const int n = col < cols ? (int)max((int64_t)0, min((int64_t)32, K - k0)) : 0;
    if (vec && __all_sync(0xffffffffu, n == 32)) {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if constexpr (T == IN_F32) {
                const uint2 f = __ldcs(reinterpret_cast<const uint2 *>(p + j * line));
                a[2 * j] = f.x, a[2 * j + 1] = f.y;
            } else {
                a[j] = __ldcs(reinterpret_cast<const uint32_t *>(p + j * line));
            }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 32 * PAIR_WORDS<T>; ++j) a[j] = 0;
    if (vec) {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (j >= n) continue;
            if constexpr (T == IN_F32) {
                const uint2 f = __ldcs(reinterpret_cast<const uint2 *>(p + j * line));
                a[2 * j] = f.x, a[2 * j + 1] = f.y;
            } else {
                a[j] = __ldcs(reinterpret_cast<const uint32_t *>(p + j * line));
            }
        }
    } else {
        const bool two = col + 1 < cols;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (j >= n) continue;
            if constexpr (T == IN_F32) {
                const uint32_t *q = reinterpret_cast<const uint32_t *>(p + j * line);
                a[2 * j] = q[0];
                if (two) a[2 * j + 1] = q[1];
            } else {
                const uint16_t *q = reinterpret_cast<const uint16_t *>(p + j * line);
                a[j] = q[0];
                if (two) a[j] |= (uint32_t)q[1] << 16;
            }
        }
    }
}

// The pair of values of row j of the tile.
template <int T>
__device__ __forceinline__ float2 pair_of(const uint32_t (&a)[32 * PAIR_WORDS<T>], int j)
{
    if constexpr (T == IN_F32) return make_float2(__uint_as_float(a[2 * j]), __uint_as_float(a[2 * j + 1]));
    else return unpack2<T>(a[j]);
}

// The tile turned round, blocks along K: row `col` of codes [cols, K].  Each column's
// (SQUARE: the tile's) largest |x| and the codes go through shared memory, and each
// row's 128 bytes of codes are written together.
template <int T, int F8, bool SQUARE>
__device__ __forceinline__ void store_columns(const uint32_t (&a)[32 * PAIR_WORDS<T>], TileSmem &sh, uint8_t *codes,
                                              uint8_t *scales, int64_t rows, int64_t K, int64_t kt, int64_t c0)
{
    constexpr int WPP = PAIR_WORDS<T>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, kq = warp & 3, c = (warp >> 2) * 64 + 2 * lane;
    const int64_t tiles = f8_tiles(K), pitch = f8_pitch(K), col = c0 + c;
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
    if constexpr (SQUARE) {
        m[0] = __reduce_max_sync(0xffffffffu, max(m[0], m[1]));
        if (lane == 0) sh.amax[0][warp] = m[0];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) m[0] = max(m[0], sh.amax[0][j]);
        m[1] = m[0];
    } else {
        *reinterpret_cast<uint2 *>(&sh.amax[kq][c]) = make_uint2(m[0], m[1]);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint2 u = *reinterpret_cast<const uint2 *>(&sh.amax[j][c]);
            m[0] = max(m[0], u.x);
            m[1] = max(m[1], u.y);
        }
    }
    const uint32_t b0 = f8_scale_byte<F8>(m[0]), b1 = f8_scale_byte<F8>(m[1]);
    const float inv0 = mx_inv_scale(b0 == 255u ? 0u : b0), inv1 = mx_inv_scale(b1 == 255u ? 0u : b1);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        float2 f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = pair_of<T>(a, 4 * q + j);
        sh.codes[c][kq * 8 + q] = b0 == 255u ? 0u : f8_encode4<F8>(f[0].x * inv0, f[1].x * inv0, f[2].x * inv0, f[3].x * inv0);
        sh.codes[c + 1][kq * 8 + q] = b1 == 255u ? 0u : f8_encode4<F8>(f[0].y * inv1, f[1].y * inv1, f[2].y * inv1, f[3].y * inv1);
    }
    __syncthreads();
    // codes: 4 bytes to a thread, a warp writes 128 bytes of one row at a time
#pragma unroll 4
    for (int r = warp; r < 128; r += 8)
        if (c0 + r < rows && kt * 128 + lane * 4 < pitch)
            *reinterpret_cast<uint32_t *>(codes + (c0 + r) * pitch + kt * 128 + lane * 4) = sh.codes[r][lane];
    // scales: a byte a row, and zeros for rows and blocks that do not exist
    if (kq == 0) {
        const int64_t last = kt == f8_blocks(K) - 1 ? tiles * 4 : kt + 1;
        for (int64_t b = kt; b < last; ++b) {
            scales[mx_scale_at(col, b, tiles)] = (uint8_t)(b == kt && col < rows ? b0 : 0u);
            scales[mx_scale_at(col + 1, b, tiles)] = (uint8_t)(b == kt && col + 1 < rows ? b1 : 0u);
        }
    }
}

template <int T, int F8, bool SQUARE>
__global__ void __launch_bounds__(256) quantize_f8_trans_kernel(const void *x, uint8_t *codes, uint8_t *scales, int64_t rows,
                                                                int64_t K, int col_tiles, bool vec)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    __shared__ TileSmem sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t kt = blockIdx.x / col_tiles, c0 = (int64_t)(blockIdx.x - kt * col_tiles) * 128;
    uint32_t a[32 * PAIR_WORDS<T>];
    load_pairs<T>(x, K, rows, kt * 128 + (warp & 3) * 32, c0 + (warp >> 2) * 64 + 2 * lane, vec, a);
    store_columns<T, F8, SQUARE>(a, sh, codes, scales, rows, K, kt, c0);
}

// The tile as it is, blocks along its 128 columns: rows of codes [K, cols].  A row's
// largest |x| is the warp's (one reduction instruction a row), then that of the two
// warps that share the row.  The codes go through shared memory, 16 bytes to a store
// (two bytes a lane straight to memory: the gradients of 333 x 1000 x 776 14.6 us, so 13.8).
struct RowSmem {
    uint32_t amax[2][128];
    float inv[8][32];
    __align__(16) uint8_t codes[128][144];
};

template <int T, int F8>
__device__ __forceinline__ void store_rows(const uint32_t (&a)[32 * PAIR_WORDS<T>], RowSmem &sh, uint8_t *codes, uint8_t *scales,
                                           int64_t rows, int64_t cols, int64_t rt, int64_t ct)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, kq = warp & 3, half = warp >> 2;
    const int64_t tiles = f8_tiles(cols), pitch = f8_pitch(cols), row = rt * 128 + kq * 32 + lane;
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        uint32_t v;
        if constexpr (T == IN_F32) {
            v = max(a[2 * j] & 0x7fffffffu, a[2 * j + 1] & 0x7fffffffu);
        } else {
            const uint32_t w = a[j] & 0x7fff7fffu;
            v = max(w & 0xffffu, w >> 16);
        }
        v = __reduce_max_sync(0xffffffffu, v);
        if (lane == j) m = v;
    }
    sh.amax[half][kq * 32 + lane] = m;
    __syncthreads();
    m = max(m, sh.amax[half ^ 1][kq * 32 + lane]);
    if constexpr (T != IN_F32) m = bits_of<T>(m);
    const uint32_t b = f8_scale_byte<F8>(m);
    sh.inv[warp][lane] = b == 255u ? -1.0f : mx_inv_scale(b);  // -1: codes 0
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        const float s = sh.inv[warp][j];
        const float2 f = pair_of<T>(a, j);
        const uint32_t v = f8_encode4<F8>(f.x * s, f.y * s, 0.0f, 0.0f);
        *reinterpret_cast<uint16_t *>(&sh.codes[kq * 32 + j][half * 64 + 2 * lane]) = (uint16_t)(s < 0.0f ? 0u : v);
    }
    if (half == 0) {
        const int64_t last = ct == f8_blocks(cols) - 1 ? tiles * 4 : ct + 1;
        for (int64_t k = ct; k < last; ++k) scales[mx_scale_at(row, k, tiles)] = (uint8_t)(k == ct && row < rows ? b : 0u);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int chunk = i * 256 + (int)threadIdx.x, r = chunk >> 3, c = (chunk & 7) * 16;
        if (rt * 128 + r < rows && ct * 128 + c < pitch)
            *reinterpret_cast<uint4 *>(codes + (rt * 128 + r) * pitch + ct * 128 + c) = *reinterpret_cast<const uint4 *>(&sh.codes[r][c]);
    }
}

// What the backward pass of a linear layer makes of dy [M, N] and x [M, K], in one
// launch: dy by rows (for dx), dy turned round and its column sums (dw, db), x turned round
// (dw): dy is read once.  The first CTAs take tiles of dy, the others of x.  8192 x 4096
// bf16 of each: 55 us (134 MB read, 101 written: 4.3 TB/s; 35 us at the copy rate): a tile is
// reduced twice, by rows and by columns, and three CTAs of an SM overlap little of that
// (two: 67 us).
template <int T, int F8>
__global__ void __launch_bounds__(256, T == IN_F32 ? 2 : 3) quantize_f8_grads_kernel(const F8Grads g)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    __shared__ TileSmem sh;
    __shared__ RowSmem rows;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, kq = warp & 3, c = (warp >> 2) * 64 + 2 * lane;
    uint32_t a[32 * PAIR_WORDS<T>];
    if ((int64_t)blockIdx.x >= g.dy_tiles) {
        const int64_t i = blockIdx.x - g.dy_tiles, tk = (g.K + 127) / 128, rt = i / tk, c0 = (i - rt * tk) * 128;
        load_pairs<T>(g.x, g.M, g.K, rt * 128 + kq * 32, c0 + c, g.K % 2 == 0, a);
        store_columns<T, F8_E4M3, false>(a, sh, g.xt_codes, g.xt_scales, g.K, g.M, rt, c0);
        return;
    }
    const int64_t tn = (g.N + 127) / 128, rt = blockIdx.x / tn, ct = blockIdx.x - rt * tn, c0 = ct * 128;
    load_pairs<T>(g.dy, g.M, g.N, rt * 128 + kq * 32, c0 + c, g.N % 2 == 0, a);
    if (g.row_codes != nullptr) store_rows<T, F8>(a, rows, g.row_codes, g.row_scales, g.M, g.N, rt, ct);
    if (g.part != nullptr) {                                   // rows in order, then quarters of the tile
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const float2 f = pair_of<T>(a, j);
            sum.x += f.x, sum.y += f.y;
        }
        float(*sums)[128] = reinterpret_cast<float(*)[128]>(&sh.codes[0][0]);
        sums[kq][c] = sum.x, sums[kq][c + 1] = sum.y;
        __syncthreads();
        const int64_t col = c0 + threadIdx.x;
        if (threadIdx.x < 128 && col < g.N)
            g.part[rt * g.N + col] = sums[0][threadIdx.x] + sums[1][threadIdx.x] + sums[2][threadIdx.x] + sums[3][threadIdx.x];
        __syncthreads();
    }
    if (g.col_codes != nullptr) store_columns<T, F8, false>(a, sh, g.col_codes, g.col_scales, g.N, g.M, rt, c0);
}

// codes and scales -> y [rows, K].  Sixteen lanes take one row's block of 128 values, 8
// to a lane; a CTA of 256 threads covers 2^bpr_log2 blocks (at most 16) of 16 >> bpr_log2
// rows, U times (U sets of loads in flight).
template <int T, int F8, bool VEC, int U>
__global__ void __launch_bounds__(256) dequantize_f8_kernel(const uint8_t *codes, const uint8_t *scales, void *y, int64_t rows,
                                                            int64_t K, int bpr_log2, int segs)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int unit = threadIdx.x >> 4, l = threadIdx.x & 15;
    const int64_t rb = blockIdx.x / segs;
    const int seg = (int)(blockIdx.x - rb * segs);
    const int64_t tiles = f8_tiles(K), pitch = f8_pitch(K);
    const int per = 16 >> bpr_log2;
    const int64_t row0 = rb * (per * U) + (unit >> bpr_log2);
    const int64_t blk = ((int64_t)seg << bpr_log2) + (unit & ((1 << bpr_log2) - 1)), k0 = blk * 128 + l * 8;
    if (VEC && k0 >= K) return;
    uint2 c[U];
    uint32_t b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t row = row0 + u * per;
        c[u] = make_uint2(0, 0);
        b[u] = 0;
        if (row >= rows || k0 >= K) continue;
        c[u] = __ldcs(reinterpret_cast<const uint2 *>(codes + row * pitch + k0));
        b[u] = scales[mx_scale_at(row, blk, tiles)];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t row = row0 + u * per;
        if (VEC && row >= rows) break;
        const float s = mx_scale(b[u]);
        const float4 lo = f8_decode4<F8>(c[u].x), hi = f8_decode4<F8>(c[u].y);
        const float v[8] = {lo.x * s, lo.y * s, lo.z * s, lo.w * s, hi.x * s, hi.y * s, hi.z * s, hi.w * s};
        const int64_t i = row * K + k0;
        if constexpr (!VEC) {
            const int n = row < rows ? (int)max((int64_t)0, min((int64_t)128, K - blk * 128)) : 0;
            store_line_any<T>(y, i - l * 8, n, v, unit, l);
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

// db from the tiles' column sums: 32 columns to a CTA, every 8th row block to a warp, then
// the warps in order.
__global__ void __launch_bounds__(256) column_sum_kernel(const float *part, float *out, int64_t blocks, int64_t cols)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    __shared__ float sums[8][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float sum = 0.0f;
    if (c < cols)
#pragma unroll 8
        for (int64_t b = warp; b < blocks; b += 8) sum += part[b * cols + c];
    sums[warp][lane] = sum;
    __syncthreads();
    if (warp != 0 || c >= cols) return;
#pragma unroll
    for (int w = 1; w < 8; ++w) sum += sums[w][lane];
    out[c] = sum;
}

template <int T, int F8>
static cudaError_t quantize_t(const void *x, uint8_t *codes, uint8_t *scales, int64_t rows, int64_t K, bool square, bool trans,
                              cudaStream_t s)
{
    const int e = T == IN_F32 ? 4 : 2;
    const int64_t padded = (rows + 127) & ~(int64_t)127;
    if (trans) {
        const int64_t col_tiles = padded / 128, grid = f8_blocks(K) * col_tiles;
        if (grid > INT32_MAX) return cudaErrorInvalidValue;
        auto k = square ? quantize_f8_trans_kernel<T, F8, true> : quantize_f8_trans_kernel<T, F8, false>;
        return launch_k(k, dim3((unsigned)grid), dim3(256), 0, s, x, codes, scales, rows, K, (int)col_tiles, rows % 2 == 0);
    }
    const bool vec = K * e % 16 == 0;
    if (square) {
        const int64_t kbs = f8_tiles(K) * 4, grid = padded / 128 * kbs;
        if (grid > INT32_MAX) return cudaErrorInvalidValue;
        auto k = vec ? quantize_f8_square_kernel<T, F8, true> : quantize_f8_square_kernel<T, F8, false>;
        return launch_k(k, dim3((unsigned)grid), dim3(512), 0, s, x, codes, scales, rows, K, (int)kbs);
    }
    // a CTA: the lanes of a row (whole scale tiles) on a power of two of its 256
    const int64_t lanes = f8_tiles(K) * 16;
    int lanes_log2 = 4;
    while (lanes_log2 < 8 && (1 << lanes_log2) < lanes) ++lanes_log2;
    const int64_t segs = (lanes + (1 << lanes_log2) - 1) >> lanes_log2, per = 256 >> lanes_log2;
    const int64_t grid = (padded + per - 1) / per * segs;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    auto k = vec ? quantize_f8_kernel<T, F8, true> : quantize_f8_kernel<T, F8, false>;
    return launch_k(k, dim3((unsigned)grid), dim3(256), 0, s, x, codes, scales, rows, K, lanes_log2, (int)segs);
}

template <int T, int F8>
static cudaError_t dequantize_t(const uint8_t *codes, const uint8_t *scales, void *y, int64_t rows, int64_t K, int sms,
                                cudaStream_t s)
{
    const RowGrid g = row_grid(rows, K, sms);
    if (g.grid > INT32_MAX) return cudaErrorInvalidValue;
    const bool vec = K * (T == IN_F32 ? 4 : 2) % 16 == 0;
    auto k = g.u == 4 ? (vec ? dequantize_f8_kernel<T, F8, true, 4> : dequantize_f8_kernel<T, F8, false, 4>)
                      : (vec ? dequantize_f8_kernel<T, F8, true, 1> : dequantize_f8_kernel<T, F8, false, 1>);
    return launch_k(k, dim3((unsigned)g.grid), dim3(256), 0, s, codes, scales, y, rows, K, g.tpr_log2, g.segs);
}

template <int F8>
static cudaError_t quantize_f8(const void *x, int type, uint8_t *codes, uint8_t *scales, int64_t rows, int64_t K, bool square,
                               bool trans, cudaStream_t s)
{
    if (type == IN_BF16) return quantize_t<IN_BF16, F8>(x, codes, scales, rows, K, square, trans, s);
    if (type == IN_F16) return quantize_t<IN_F16, F8>(x, codes, scales, rows, K, square, trans, s);
    return quantize_t<IN_F32, F8>(x, codes, scales, rows, K, square, trans, s);
}

cudaError_t launch_quantize_fp8(const void *x, int type, uint8_t *codes, uint8_t *scales, int64_t rows, int64_t K, int f8,
                                bool square, bool trans, cudaStream_t s)
{
    return f8 == F8_E4M3 ? quantize_f8<F8_E4M3>(x, type, codes, scales, rows, K, square, trans, s)
                         : quantize_f8<F8_E5M2>(x, type, codes, scales, rows, K, square, trans, s);
}

template <int F8>
static cudaError_t dequantize_f8(const uint8_t *codes, const uint8_t *scales, void *y, int type, int64_t rows, int64_t K,
                                 int sms, cudaStream_t s)
{
    if (type == IN_BF16) return dequantize_t<IN_BF16, F8>(codes, scales, y, rows, K, sms, s);
    if (type == IN_F16) return dequantize_t<IN_F16, F8>(codes, scales, y, rows, K, sms, s);
    return dequantize_t<IN_F32, F8>(codes, scales, y, rows, K, sms, s);
}

cudaError_t launch_dequantize_fp8(const uint8_t *codes, const uint8_t *scales, void *y, int type, int64_t rows, int64_t K,
                                  int f8, int sms, cudaStream_t s)
{
    return f8 == F8_E4M3 ? dequantize_f8<F8_E4M3>(codes, scales, y, type, rows, K, sms, s)
                         : dequantize_f8<F8_E5M2>(codes, scales, y, type, rows, K, sms, s);
}

cudaError_t launch_quantize_fp8_grads(F8Grads g, int type, int f8, cudaStream_t s)
{
    const int64_t tm = (g.M + 127) / 128, tn = (g.N + 127) / 128, tk = (g.K + 127) / 128;
    g.dy_tiles = g.row_codes != nullptr || g.col_codes != nullptr || g.part != nullptr ? tm * tn : 0;
    const int64_t grid = g.dy_tiles + (g.xt_codes != nullptr ? tm * tk : 0);
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    if (grid == 0) return cudaSuccess;
    void (*k)(const F8Grads);
    if (f8 == F8_E4M3)
        k = type == IN_BF16 ? quantize_f8_grads_kernel<IN_BF16, F8_E4M3>
                            : (type == IN_F16 ? quantize_f8_grads_kernel<IN_F16, F8_E4M3> : quantize_f8_grads_kernel<IN_F32, F8_E4M3>);
    else
        k = type == IN_BF16 ? quantize_f8_grads_kernel<IN_BF16, F8_E5M2>
                            : (type == IN_F16 ? quantize_f8_grads_kernel<IN_F16, F8_E5M2> : quantize_f8_grads_kernel<IN_F32, F8_E5M2>);
    return launch_k(k, dim3((unsigned)grid), dim3(256), 0, s, g);
}

cudaError_t launch_column_sums(const float *part, float *out, int64_t rows, int64_t cols, cudaStream_t s)
{
    return launch_k(column_sum_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(256), 0, s, part, out, (rows + 127) / 128, cols);
}

}  // namespace mmact
