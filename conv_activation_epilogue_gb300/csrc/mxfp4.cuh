// mxfp4.cuh -- the 4-bit microscaled format: layout, conversions, tensor-core
// instructions; and the activations of the operators that use it.
//
// MXFP4 (OCP Microscaling Formats specification 1.0): 32 consecutive values
// along K share the scale X = 2^(b - 127) with b one byte (255 = NaN); a value
// is X times an E2M1 number, one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign.
// Quantisation: b = max(floor(log2(amax)) - 2 + 127, 0), values rounded to
// nearest even on the E2M1 grid, those past 6 set to 6.
//
// A quantised matrix [rows, K] is two arrays:
//   codes   [rows][KB * 16] bytes, KB = ceil(K / 32): two codes to a byte, the
//           even k in the low half; codes past K are 0
//   scales  tiles of 512 bytes, [ceil(rows / 128)][ceil(KB / 4)]: the scale of
//           row r, block b is byte (r % 32) * 16 + (r % 128) / 32 * 4 + b % 4 of
//           its tile; bytes of rows or blocks that do not exist are 0.
// A tile is what one tcgen05.cp.32x128b.warpx4 moves into tensor memory: 32
// lanes x 16 bytes, column c holding the four scales of row lane + 32 c.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace mmact {

constexpr int MX_BLOCK = 32;

__host__ __device__ constexpr int64_t mx_blocks(int64_t k) { return (k + 31) / 32; }
__host__ __device__ constexpr int64_t mx_tiles(int64_t k) { return (k + 127) / 128; }

// Byte offset of the scale of row r, block b (tiles = mx_tiles(K)).
__device__ __forceinline__ int64_t mx_scale_at(int64_t r, int64_t b, int64_t tiles)
{
    return ((r >> 7) * tiles + (b >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3);
}

// Scale byte of a block from the bits of its largest |x| (as fp32): the
// exponent field minus 2, at least 0; 255 when the block holds an infinity or
// a NaN.  A block of zeros gets 0.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits)
{
    const uint32_t e = amax_bits >> 23;
    return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}

// 1 / X for a finite block (b <= 252): exact.
__device__ __forceinline__ float mx_inv_scale(uint32_t b)
{
    return __uint_as_float((254u - b) << 23);
}

// X of a scale byte: 2^-127 is subnormal, 255 is NaN.
__device__ __forceinline__ float mx_scale(uint32_t b)
{
    return __uint_as_float(b == 0u ? 0x00400000u : (b == 255u ? 0x7fc00000u : b << 23));
}

// Eight values, already divided by X, to eight codes (v[0] in the low bits):
// round to nearest even, saturating at +-6.
__device__ __forceinline__ uint32_t mx_encode8(const float (&v)[8])
{
    uint32_t r;
    asm("{\n\t.reg .b8 c0, c1, c2, c3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c3, %8, %7;\n\t"
        "mov.b32 %0, {c0, c1, c2, c3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Eight codes to eight E2M1 values.
__device__ __forceinline__ void mx_decode8(uint32_t c, float (&v)[8])
{
    uint32_t h[4];
    asm("{\n\t.reg .b8 c0, c1, c2, c3;\n\t"
        "mov.b32 {c0, c1, c2, c3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, c0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, c1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, c3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(c));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// ------------------------------------------------------------- quantisation --
enum : int { IN_F32 = OUT_F32, IN_F16 = OUT_F16, IN_BF16 = OUT_BF16 };

// Eight consecutive values x[i..i+8) as raw 32-bit words, two 16-bit values or
// one fp32 to a word (values at or past `n` are 0).  (Here and in the kernels no input
// is read through the read-only path: a kernel is on its SMs before griddep_wait
// returns, while the one before it may still write what it will read.)
template <int T>
struct Raw8 {
    static constexpr int WORDS = T == IN_F32 ? 8 : 4;
    uint32_t w[WORDS];
};

template <int T, bool VEC>
__device__ __forceinline__ void load8(const void *x, int64_t i, int n, Raw8<T> &r)
{
    if (VEC && n >= 8) {
#pragma unroll
        for (int j = 0; j < Raw8<T>::WORDS / 4; ++j) {
            const char *p = static_cast<const char *>(x) + i * (T == IN_F32 ? 4 : 2) + 16 * j;
            const uint4 u = *reinterpret_cast<const uint4 *>(p);
            r.w[4 * j] = u.x, r.w[4 * j + 1] = u.y, r.w[4 * j + 2] = u.z, r.w[4 * j + 3] = u.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (T == IN_F32) {
                r.w[j] = j < n ? static_cast<const uint32_t *>(x)[i + j] : 0u;
            } else {
                const uint32_t v = j < n ? static_cast<const uint16_t *>(x)[i + j] : 0u;
                r.w[j / 2] = j % 2 == 0 ? v : r.w[j / 2] | (v << 16);
            }
        }
    }
}

// A block of n <= 32 consecutive values x[at..at+n) (the rest 0) that begins anywhere,
// of a tensor of `total` values: the aligned 16 bytes that hold them, shifted into
// place.  (By single values, 32 lanes each 64 bytes from the next, rows that are not a
// multiple of 16 bytes took three times as long: 5447 x 3659 bf16 35.8 us, 11.6 so.)
// Where those reach past the end of the tensor, by single values.
template <int T>
__device__ __forceinline__ void load32_any(const void *x, int64_t at, int n, int64_t total, Raw8<T> (&r)[4])
{
    constexpr int ES = T == IN_F32 ? 4 : 2, WORDS = 8 * ES, PER = WORDS / 4;
    const int shift = (int)(at * ES) & 15, bytes = shift + n * ES;
    const int64_t from = at * ES - shift;
    if (from + ((bytes + 15) & ~15) > total * ES) {
#pragma unroll
        for (int q = 0; q < 4; ++q) load8<T, false>(x, at + 8 * q, n - 8 * q, r[q]);
        return;
    }
    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const char *>(x) + from);
    uint32_t u[WORDS + 4];
#pragma unroll
    for (int c = 0; c <= WORDS / 4; ++c) {
        const uint4 v = 16 * c < bytes ? p[c] : make_uint4(0, 0, 0, 0);
        u[4 * c] = v.x, u[4 * c + 1] = v.y, u[4 * c + 2] = v.z, u[4 * c + 3] = v.w;
    }
    if (shift & 8)
#pragma unroll
        for (int j = 0; j < WORDS + 2; ++j) u[j] = u[j + 2];
    if (shift & 4)
#pragma unroll
        for (int j = 0; j < WORDS + 1; ++j) u[j] = u[j + 1];
#pragma unroll
    for (int j = 0; j < WORDS; ++j) {
        uint32_t w = u[j];
        if constexpr (T == IN_F32) {
            if (j >= n) w = 0;
        } else {
            if (shift & 2) w = __funnelshift_r(u[j], u[j + 1], 16);
            if (2 * j >= n) w = 0;
            else if (2 * j + 1 >= n) w &= 0xffffu;
        }
        r[j / PER].w[j % PER] = w;
    }
}

// The largest |value| of raw words so far: of 16-bit types in each half of `m`
// (their magnitudes order as unsigned integers, infinities and NaN on top).
template <int T>
__device__ __forceinline__ uint32_t raw_max(uint32_t m, uint32_t w)
{
    if constexpr (T == IN_F32) return max(m, w & 0x7fffffffu);
    else return __vmaxu2(m, w & 0x7fff7fffu);
}

// The fp32 bits of a 16-bit magnitude.
template <int T>
__device__ __forceinline__ uint32_t bits_of(uint32_t h)
{
    if constexpr (T == IN_BF16) return h << 16;
    else return __float_as_uint(__half2float(__ushort_as_half((unsigned short)h)));
}

// Codes of eight values held as raw words, times `inv`.
template <int T>
__device__ __forceinline__ uint32_t raw_encode(const uint32_t (&w)[Raw8<T>::WORDS], float inv)
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
    return mx_encode8(v);
}

// -------------------------------------------------------------- activations --
enum : int { ACT_SILU = ACT_GELU + 1 };

// z * sigma(z) = z / (1 + e^-z): one hardware exponential and one fast divide, a
// few ulp each.  Below z = -87 the divisor passes 2^126, where __fdividef gives 0 or
// (e^-z = inf) NaN; the value, above -1e-36 there, is cut off to -0.  At z = -inf
// it is NaN, as the formula's -inf / inf.
__device__ __forceinline__ float silu_f32(float z)
{
    return z < -87.0f ? z * 0.0f : __fdividef(z, 1.0f + __expf(-z));
}

// max(z, 0), NaN for a NaN: a block that the quantiser marked must not come out as zeros.
__device__ __forceinline__ float relu_f32(float z)
{
    float r;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(z));
    return r;
}

template <int ACT>
__device__ __forceinline__ float act_mx(float z, float alpha)
{
    if constexpr (ACT == ACT_SILU) return silu_f32(z);
    else if constexpr (ACT == ACT_RELU) return relu_f32(z);
    else return act_f32<ACT>(z, alpha);
}

__device__ __forceinline__ float act_mx(int act, float z, float alpha)
{
    switch (act) {
    case ACT_RELU: return act_mx<ACT_RELU>(z, alpha);
    case ACT_LEAKY: return act_mx<ACT_LEAKY>(z, alpha);
    case ACT_TANH: return act_mx<ACT_TANH>(z, alpha);
    case ACT_SIGMOID: return act_mx<ACT_SIGMOID>(z, alpha);
    case ACT_GELU: return act_mx<ACT_GELU>(z, alpha);
    case ACT_SILU: return act_mx<ACT_SILU>(z, alpha);
    default: return z;
    }
}

// The same over an array, the activation looked up once.
template <int ACT, int N>
__device__ __forceinline__ void act_mx_all(float (&v)[N], float alpha)
{
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = act_mx<ACT>(v[i], alpha);
}

template <int N>
__device__ __forceinline__ void act_mx_all(int act, float (&v)[N], float alpha)
{
    switch (act) {
    case ACT_RELU: act_mx_all<ACT_RELU>(v, alpha); break;
    case ACT_LEAKY: act_mx_all<ACT_LEAKY>(v, alpha); break;
    case ACT_TANH: act_mx_all<ACT_TANH>(v, alpha); break;
    case ACT_SIGMOID: act_mx_all<ACT_SIGMOID>(v, alpha); break;
    case ACT_GELU: act_mx_all<ACT_GELU>(v, alpha); break;
    case ACT_SILU: act_mx_all<ACT_SILU>(v, alpha); break;
    default: break;
    }
}

// -------------------------------------------------- tensor-core instructions --
namespace ptx {

// The tcgen05 instructions below are executed by a whole converged warp and
// issued by one elected lane of it (always the same one, so that a commit covers
// the MMAs before it).  A warp-uniform loop keeps descriptors and addresses in
// uniform registers; the same loop run by a single lane moves them there before
// every instruction, and was measured at 108 cycles an instruction where a
// 256 x 256 x 64 MMA of a CTA pair takes 128 (133 with this form, the scale
// copies of its stage included).
#define MMACT_ELECTED "{\n\t.reg .pred p, q;\n\telect.sync _|q, 0xffffffff;\n\t"

// D[tmem] (+)= (A x scale_A)(B x scale_B), kind::mxf4: E2M1 operands packed two
// to a byte, K-major, K = 64 per instruction, one UE8M0 scale per row and 32 K
// (two per row and instruction), scales in tensor memory at columns that are a
// multiple of four.
__device__ __forceinline__ void mma_mxf4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t sa_tmem, uint32_t sb_tmem, uint32_t accumulate)
{
    asm volatile(
        MMACT_ELECTED
        "setp.ne.b32 p, %6, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate)
        : "memory");
}

// The same over a CTA pair (issued in the even CTA): M = 256, each CTA holds its
// 128 rows of A, half of B's rows, its own A rows' scales and all of B's scales.
__device__ __forceinline__ void mma_mxf4_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                              uint32_t sa_tmem, uint32_t sb_tmem, uint32_t accumulate)
{
    asm volatile(
        MMACT_ELECTED
        "setp.ne.b32 p, %6, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate)
        : "memory");
}

// Copy 32 rows x 16 bytes of shared memory (an unswizzled descriptor, 8-row
// groups of 128 bytes) to four 32-bit columns of all four lane quarters of
// tensor memory: one scale tile.  Ordered before the MMAs issued after it.
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint64_t sdesc)
{
    asm volatile(MMACT_ELECTED "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr), "l"(sdesc)
                 : "memory");
}

// The same in both CTAs of a pair, each from its own shared memory to its own
// tensor memory (issued in the even CTA).
__device__ __forceinline__ void tmem_cp_scales_pair(uint32_t taddr, uint64_t sdesc)
{
    asm volatile(MMACT_ELECTED "@q tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr), "l"(sdesc)
                 : "memory");
}

// Arrive once on `bar` when every MMA and copy issued so far is done; on a pair,
// on the barrier of every CTA in `mask`.
__device__ __forceinline__ void commit_elected(uint32_t bar)
{
    asm volatile(MMACT_ELECTED
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
                 : "memory");
}

__device__ __forceinline__ void commit_elected_pair(uint32_t bar, uint16_t mask)
{
    asm volatile(MMACT_ELECTED
                 "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], "
                 "%1;\n\t}" ::"r"(bar),
                 "h"(mask)
                 : "memory");
}

#undef MMACT_ELECTED

// One ring stage of 256 K of a product of 128 rows (A) by a tile (B) of at most 128:
// four scale tiles of 512 bytes (A's two, then B's) to 16 columns of tensor memory
// from `ts` on, and a K = 64 MMA for each 32 bytes of the operands' rows; `n` of them,
// 4 but in the last stage.  `a`, `b`, `s` are the descriptors of the stage's parts.
// The usual case is one block with one election: descriptors made one by one, with a
// branch around each MMA, took 640 clocks a stage, as long as a stage's weights come
// in.
__device__ __forceinline__ void mma_mxf4_stage(uint32_t d, uint64_t a, uint64_t b, uint64_t s, uint32_t ts, uint32_t id0,
                                               uint32_t id2, int n, uint32_t accumulate)
{
    if (n == 4) {
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .b64 a1, a2, a3, b1, b2, b3, s1, s2, s3;\n\t"
            ".reg .b32 t1, t2, t3;\n\t"
            "setp.ne.b32 p, %7, 0;\n\t"
            "add.s64 s1, %3, 32;\n\tadd.s64 s2, %3, 64;\n\tadd.s64 s3, %3, 96;\n\t"
            "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
            "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
            "add.s32 t1, %4, 4;\n\tadd.s32 t2, %4, 8;\n\tadd.s32 t3, %4, 12;\n\t"
            "elect.sync _|q, 0xffffffff;\n\t"
            "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%4], %3;\n\t"
            "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [t1], s1;\n\t"
            "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [t2], s2;\n\t"
            "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [t3], s3;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %5, [%4], [t2], p;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], a1, b1, %6, [%4], [t2], 1;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], a2, b2, %5, [t1], [t3], 1;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], a3, b3, %6, [t1], [t3], 1;\n\t"
            "}" ::"r"(d),
            "l"(a), "l"(b), "l"(s), "r"(ts), "r"(id0), "r"(id2), "r"(accumulate)
            : "memory");
        return;
    }
#pragma unroll 1
    for (int j = 0; j < 4; ++j) tmem_cp_scales(ts + 4 * j, s + 32 * j);
#pragma unroll 1
    for (int k = 0; k < n; ++k)
        mma_mxf4(d, a + 2 * k, b + 2 * k, k & 1 ? id2 : id0, ts + 4 * (k >> 1), ts + 8 + 4 * (k >> 1), accumulate | (uint32_t)k);
}

// Instruction descriptor for kind::mxf4: A and B E2M1 (format 1), scales UE8M0,
// M and N extents; sa and sb (0 or 2) say which two bytes of the 32-bit scale
// columns hold this instruction's scales.
__host__ __device__ constexpr uint32_t idesc_mxf4(int M, int N, uint32_t sa, uint32_t sb)
{
    return (sb << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
           ((uint32_t)(M >> 7) << 27) | (sa << 29);
}

// Non-binding copy of a tensor box to L2.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap *m, int x, int y)
{
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(m)),
                 "r"(x), "r"(y)
                 : "memory");
}

// 32-bit float load from another CTA's shared memory (address from mapa).
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// 32 lanes x 16 consecutive 32-bit columns: thread i gets lane (base + i).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

}  // namespace ptx

// A pipeline wait of a whole warp with one verdict for it.
__device__ __forceinline__ bool mx_warp_wait(const Pipe &pp, uint32_t bar, uint32_t parity)
{
    return __all_sync(0xffffffffu, pipe_wait(pp, bar, parity)) != 0;
}

}  // namespace mmact
