// fp8.cuh -- 8-bit floating point with a scale for each block of 128: layout,
// conversions, tensor-core instructions.
//
// 128 consecutive values along K share the scale X = 2^(b - 127), b one byte (255 =
// NaN); a value is X times an E4M3 or E5M2 number.  Quantisation: X is the smallest
// power of two, 2^-127 at least, with which the block's largest |x| / X does not pass
// the type's largest value (448 or 57344, both 1.75 times a power of two), so nothing
// saturates and the division by X is exact; values are rounded to nearest even.  A
// power of two costs a floating-point code no precision (but at the subnormal end),
// and the tensor core applies it by itself.
//
// A quantised matrix [rows, K] is two arrays:
//   codes   [rows][KP] bytes, KP = K rounded up to 16; codes past K are 0
//   scales  tiles of 512 bytes, [ceil(rows / 128)][ceil(KB / 4)], KB = ceil(K / 128):
//           the scale of row r, block b is byte (r % 32) * 16 + (r % 128) / 32 * 4 + b % 4
//           of its tile; bytes of rows or blocks that do not exist are 0.
// Square blocks (128 rows share the scale too) are the same arrays with equal bytes.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "mxfp4.cuh"

namespace mmact {

enum : int { F8_E4M3 = 0, F8_E5M2 = 1 };       // also the operand formats of the instruction descriptor

__host__ __device__ constexpr int64_t f8_pitch(int64_t k) { return (k + 15) / 16 * 16; }
__host__ __device__ constexpr int64_t f8_blocks(int64_t k) { return (k + 127) / 128; }
__host__ __device__ constexpr int64_t f8_tiles(int64_t k) { return (k + 511) / 512; }

// Scale byte of a block from the bits of its largest |x| (as fp32): 1.75 * 2^8 and
// 1.75 * 2^15 are the types' largest values, so a fraction above 0.75 takes the next
// power of two.  255 when the block holds an infinity or a NaN; a block of zeros gets 0.
template <int F8>
__device__ __forceinline__ uint32_t f8_scale_byte(uint32_t amax_bits)
{
    constexpr int TOP = F8 == F8_E4M3 ? 8 : 15;
    const int e = (int)(amax_bits >> 23);
    if (e == 255) return 255u;
    return (uint32_t)max(0, e - TOP + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0));
}

// Four values, already divided by X, to four codes (v0 in the low byte).
template <int F8>
__device__ __forceinline__ uint32_t f8_encode4(float v0, float v1, float v2, float v3)
{
    uint32_t r;
    if constexpr (F8 == F8_E4M3)
        asm("{\n\t.reg .b16 a, b;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
            "mov.b32 %0, {a, b};\n\t}"
            : "=r"(r)
            : "f"(v0), "f"(v1), "f"(v2), "f"(v3));
    else
        asm("{\n\t.reg .b16 a, b;\n\t"
            "cvt.rn.satfinite.e5m2x2.f32 a, %2, %1;\n\t"
            "cvt.rn.satfinite.e5m2x2.f32 b, %4, %3;\n\t"
            "mov.b32 %0, {a, b};\n\t}"
            : "=r"(r)
            : "f"(v0), "f"(v1), "f"(v2), "f"(v3));
    return r;
}

// Four codes to four values.
template <int F8>
__device__ __forceinline__ float4 f8_decode4(uint32_t c)
{
    uint32_t h0, h1;
    if constexpr (F8 == F8_E4M3)
        asm("{\n\t.reg .b16 a, b;\n\t"
            "mov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(h0), "=r"(h1)
            : "r"(c));
    else
        asm("{\n\t.reg .b16 a, b;\n\t"
            "mov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e5m2x2 %0, a;\n\t"
            "cvt.rn.f16x2.e5m2x2 %1, b;\n\t}"
            : "=r"(h0), "=r"(h1)
            : "r"(c));
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&h0));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&h1));
    return make_float4(a.x, a.y, b.x, b.y);
}

// Codes of eight values held as raw words, times `inv` (a word of codes each four).
template <int T, int F8>
__device__ __forceinline__ uint2 f8_raw_encode(const uint32_t (&w)[Raw8<T>::WORDS], float inv)
{
    float v[8];
    if constexpr (T == IN_F32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]) * inv;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = unpack2<T>(w[j]);
            v[2 * j] = f.x * inv;
            v[2 * j + 1] = f.y * inv;
        }
    }
    return make_uint2(f8_encode4<F8>(v[0], v[1], v[2], v[3]), f8_encode4<F8>(v[4], v[5], v[6], v[7]));
}

namespace ptx {

// Instruction descriptor for kind::mxf8f6f4: operand formats (F8_*), scales UE8M0, M and
// N extents.  The byte of the 32-bit scale columns that holds this instruction's
// scales is added by f8_scale_id.
__host__ __device__ constexpr uint32_t idesc_f8(int a, int b, int M, int N)
{
    return ((uint32_t)a << 7) | ((uint32_t)b << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 7) << 27);
}

__device__ __forceinline__ uint32_t f8_scale_id(int kb) { return ((uint32_t)(kb & 3) << 4) | ((uint32_t)(kb & 3) << 29); }

// One ring stage of 128 K over a CTA pair (issued in the even CTA by the whole warp,
// one elected lane): with `copy`, the scale tiles of the CTA's A rows (512 bytes at `s`)
// and of all B rows (two tiles behind it) to 12 columns of tensor memory from `ts` on,
// B's first; then a K = 32 MMA for each 32 bytes of the operands' rows, `n` of them.
__device__ __forceinline__ void mma_f8_stage_pair(uint32_t d, uint64_t a, uint64_t b, uint64_t s, uint32_t ts, uint32_t id,
                                                  int n, uint32_t accumulate, uint32_t copy)
{
    asm volatile(
        "{\n\t.reg .pred p, q, c, n1, n2, n3;\n\t.reg .b64 a1, a2, a3, b1, b2, b3, s1, s2;\n\t"
        ".reg .b32 t1, t2;\n\t"
        "setp.ne.b32 p, %7, 0;\n\t"
        "add.s64 s1, %3, 32;\n\tadd.s64 s2, %3, 64;\n\t"
        "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
        "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
        "add.s32 t1, %4, 4;\n\tadd.s32 t2, %4, 8;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.ne.and.b32 c, %8, 0, q;\n\t"
        "setp.gt.and.s32 n1, %6, 1, q;\n\tsetp.gt.and.s32 n2, %6, 2, q;\n\tsetp.gt.and.s32 n3, %6, 3, q;\n\t"
        "@c tcgen05.cp.cta_group::2.32x128b.warpx4 [%4], s1;\n\t"
        "@c tcgen05.cp.cta_group::2.32x128b.warpx4 [t1], s2;\n\t"
        "@c tcgen05.cp.cta_group::2.32x128b.warpx4 [t2], %3;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %5, [t2], [%4], p;\n\t"
        "@n1 tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a1, b1, %5, [t2], [%4], 1;\n\t"
        "@n2 tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a2, b2, %5, [t2], [%4], 1;\n\t"
        "@n3 tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a3, b3, %5, [t2], [%4], 1;\n\t"
        "}" ::"r"(d),
        "l"(a), "l"(b), "l"(s), "r"(ts), "r"(id), "r"(n), "r"(accumulate), "r"(copy)
        : "memory");
}

// The same on one CTA: 128 rows (A) by a tile (B) of at most 128, A's scale tile (at `sa`),
// then B's (`sb`), to 8 columns from `ts` on.
__device__ __forceinline__ void mma_f8_stage(uint32_t d, uint64_t a, uint64_t b, uint64_t sa, uint64_t sb, uint32_t ts,
                                             uint32_t id, int n, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, q, n1, n2, n3;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
        ".reg .b32 t1;\n\t"
        "setp.ne.b32 p, %7, 0;\n\t"
        "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
        "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
        "add.s32 t1, %4, 4;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.gt.and.s32 n1, %6, 1, q;\n\tsetp.gt.and.s32 n2, %6, 2, q;\n\tsetp.gt.and.s32 n3, %6, 3, q;\n\t"
        "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%4], %3;\n\t"
        "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [t1], %8;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %5, [%4], [t1], p;\n\t"
        "@n1 tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a1, b1, %5, [%4], [t1], 1;\n\t"
        "@n2 tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a2, b2, %5, [%4], [t1], 1;\n\t"
        "@n3 tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a3, b3, %5, [%4], [t1], 1;\n\t"
        "}" ::"r"(d),
        "l"(a), "l"(b), "l"(sa), "r"(ts), "r"(id), "r"(n), "r"(accumulate), "l"(sb)
        : "memory");
}

}  // namespace ptx

}  // namespace mmact
