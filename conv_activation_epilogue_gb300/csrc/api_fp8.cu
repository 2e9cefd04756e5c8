// api_fp8.cu -- the C ABI of the 8-bit floating-point operators (include/mmact.h):
// argument validation and launch planning.  As in api.cu, every check happens on the
// host before anything is enqueued.
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <utility>

#include <cuda.h>
#include <cuda_runtime.h>

#include "api_checks.h"
#include "api_internal.h"
#include "fp8.cuh"
#include "kernels_fp8.h"
#include "kernels_mx.h"
#include "mmact.h"

#define MMACT_EXPORT extern "C" __attribute__((visibility("default")))

namespace mmact {
namespace {

bool valid_f8(mmact_dtype d) { return d == MMACT_E4M3 || d == MMACT_E5M2; }
int f8_kind(mmact_dtype d) { return d == MMACT_E5M2 ? F8_E5M2 : F8_E4M3; }

std::atomic<int> g_f8_kernel{0};   // 0: chosen per shape; 1: rows kernel; 2: pair kernel

// The current device, with this file's kernels set up on it (once per device).
struct F8Context {
    DeviceContext dev;
    int max_pairs;                   // CTA pairs of the pair kernel resident at once
    const int *max_clusters;         // [i]: clusters of 2^i CTAs of the rows kernel
};

mmact_status f8_context(F8Context *out)
{
    static std::mutex mutex;
    static std::atomic<bool> ready[MAX_DEVICES];
    static int pairs[MAX_DEVICES], clusters[MAX_DEVICES][4];
    const mmact_status s = device_context(&out->dev);
    if (s != MMACT_OK) return s;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEVICES) return MMACT_ERR_CUDA;
    if (!ready[dev].load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> lock(mutex);
        // once: other threads read pairs and clusters as soon as `ready` says so
        if (!ready[dev].load(std::memory_order_relaxed) &&
            (setup_fp8_pair_kernels(&pairs[dev]) != cudaSuccess || setup_fp8_rows_kernels(clusters[dev]) != cudaSuccess))
            return MMACT_ERR_CUDA;
        ready[dev].store(true, std::memory_order_release);
    }
    out->max_pairs = pairs[dev];
    out->max_clusters = clusters[dev];
    return MMACT_OK;
}

int64_t f8_codes_bytes(int64_t rows, int64_t K) { return rows * f8_pitch(K); }
int64_t f8_scales_bytes(int64_t rows, int64_t K) { return (rows + 127) / 128 * f8_tiles(K) * 512; }

// A matrix in 8 bits.
struct F8Matrix {
    const void *codes, *scales;
    mmact_dtype type;
};

mmact_status f8_gemm_check(const F8Matrix &A, const F8Matrix &B, const float *bias, const void *C, int64_t M, int64_t N,
                           int64_t K, mmact_dtype cd, mmact_act act)
{
    if (!mx_dims(M, K) || !mx_dims(N, K)) return MMACT_ERR_INVALID_ARG;
    if (((A.codes == nullptr || A.scales == nullptr) && M * K != 0) ||
        ((B.codes == nullptr || B.scales == nullptr) && N * K != 0) || (C == nullptr && M * N != 0))
        return MMACT_ERR_INVALID_ARG;
    if (!valid_f8(A.type) || !valid_f8(B.type) || !valid_float(cd) || !valid_act(act)) return MMACT_ERR_INVALID_ARG;
    if (bias != nullptr && !aligned4(bias)) return MMACT_ERR_INVALID_ARG;
    if (!aligned16(A.codes) || !aligned16(A.scales) || !aligned16(B.codes) || !aligned16(B.scales) || !aligned16(C))
        return MMACT_ERR_UNSUPPORTED;
    if (((M + 127) / 128) * ((N + 127) / 128) > MAX_DIM) return MMACT_ERR_UNSUPPORTED;
    return MMACT_OK;
}

// Tensor maps of an 8-bit matrix: its codes as 16-bit words (box 64 words = 128 codes x
// `box_rows` rows, 128-byte swizzle) and its scale tiles as 32-bit words (box 128 words = a
// tile, of `box_tiles` rows of tiles).  Rows, codes and tiles past the end arrive as zeros.
bool f8_encode(CUtensorMap *mc, CUtensorMap *ms, const F8Matrix &m, int64_t rows, int64_t K, uint32_t box_rows,
               uint32_t box_tiles)
{
    const uint64_t dc[2] = {(uint64_t)f8_pitch(K) / 2, (uint64_t)rows}, sc[1] = {(uint64_t)f8_pitch(K)};
    const uint32_t bc[2] = {64, box_rows};
    const uint64_t ds[2] = {(uint64_t)f8_tiles(K) * 128, (uint64_t)(rows + 127) / 128};
    const uint64_t ss[1] = {(uint64_t)f8_tiles(K) * 512};
    const uint32_t bs[2] = {128, box_tiles};
    return encode_tensor_map(mc, MMACT_BF16, 2, m.codes, dc, sc, bc, true) &&
           encode_tensor_map(ms, MMACT_F32, 2, m.scales, ds, ss, bs, false);
}

// K blocks whose products an accumulator takes, at most, when the output is fp32 (gemm_fp8.cu).
constexpr int F8_CHUNK_KB = 16;

// Plan of one product: either kernel's launch.
struct F8Plan {
    bool pair, quantize;             // quantize: x first, by a kernel of its own
    F8Problem P;
    F8RowsProblem R;                 // but its bt-wide tiles, which the launch lays out
    F8Matrix A, B;
    int x_type;                      // OUT_* of R.x; < 0: A is quantised
};

int64_t f8_row_tiles(int64_t M, int64_t N) { return ((M + 127) / 128) * ((N + 127) / 128); }

// Whether a product runs on the pair kernel: when the rows kernel would have more tiles
// (128 x 128) than there are SMs, or K is short for the tiles there are.  Measured (us, rows
// and pair): 256 tiles of K = 4096 28.7 and 15.7, 160 28.0 and 15.2; 128 tiles of K = 4096 14.7 and
// 14.9, 2048 10.2 and 10.0, 1024 7.8 and 7.2; 64 of 8192 16.4 and 22.7, 4096 12.0 and 14.7, 2048 9.7 and
// 9.3, 1024 8.1 and 7.1, 512 7.1 and 6.0; 16 of 2048 7.7 and 9.1, 1024 6.9 and 6.9, 512 6.9 and 5.9.
bool f8_choose_pair(const F8Context &c, int64_t M, int64_t N, int64_t K)
{
    const int mode = g_f8_kernel.load();
    if (c.max_pairs < 1 || mode == 1) return false;
    if (mode == 2) return true;
    const int64_t tiles = f8_row_tiles(M, N);
    return M > 128 && (tiles > c.dev.sm_count || K <= 16 * std::max<int64_t>(tiles, 48));
}

// Rows of x up to which the rows kernel quantises them itself.  Measured (us, inside and by
// a kernel before): 1 x 8192 x 8192 14.3 and 16.2, 8 rows 15.3 and 16.6, 8 x 4096 x 4096 6.7 and 8.5.
constexpr int64_t F8_FUSED_ROWS = 8;

enum : int { F8_ANY, F8_ROWS, F8_PAIR };   // kernel of a plan; F8_ANY: the product's own choice

// The kernel of both gradients, so that they share a launch, or F8_ANY: each its own.  When the two
// would choose different ones, that of the rows kernel (m x n, over k) has few tiles and many K blocks, the other
// (`other_tiles`, `other_kb`) the reverse.  A shared launch ends no earlier than the few tiles: from some 40 K blocks on that is
// later than two launches do.  Measured (us, the whole backward pass, M x N x K: own kernels, both rows, both pair):
//   few tiles, long K    8192 x 512 x 512 (16 tiles of 64 K blocks) 31, 41, 41; 131072 x 512 x 512 251, 987, 512;
//                        18000 x 64 x 100 29, 53, 64; 8192 x 512 x 1024 (32 tiles) 36, 72, 43; 256 x 8192 x 1024 32, 48, 38
//   shorter              4096 x 512 x 512 (32 K blocks) 27, 25, 28; 1024 x 4096 x 512 30, 32, 26
//   more tiles           8192 x 1024 x 1024 (64 tiles) 48, 90, 49; 8192 x 768 x 2048 (96) 70, 146, 53
// With m (the tokens, or dw's rows) 128 or less the other product is all stores and keeps the pairs busy for longer:
// 100 x 6500 x 2000 (16 tiles of 51 K blocks) 33, 59, 38, but 128 x 6144 x 4096 (32 of 48) 44, 83, 41; from about
// 112 K blocks on its tiles are no longer long enough: 128 x 12288 x 4096 (32 of 96) 68, 154, 65; 16384 x 64 x 4096 (32 of
// 128) 98, 209, 110; 64 x 16384 x 8192 (64 of 128) 137, 357, 168.
// A shared launch is of pairs when a product has more tiles than SMs or there is much to do (K blocks of both
// products' tiles together): 2048 x 1024 x 1024 (2048) 30, 25, 21; 1024 x 4096 x 512 (2048) above; 4096 x 512 x 512
// (1024) above; 2048 x 512 x 512 (512) 24, 16, 18.
int f8_shared_kernel(const F8Context &c, int64_t m, int64_t n, int64_t k, int64_t other_tiles, int64_t other_kb)
{
    const int64_t tiles = f8_row_tiles(m, n), kb = f8_blocks(k);
    if (tiles <= c.max_pairs / (m <= 128 ? 4 : 2) && kb >= 40 + tiles / 2) return F8_ANY;
    if (m <= 128 && tiles <= c.max_pairs && kb >= 112) return F8_ANY;
    return std::max(tiles, other_tiles) > c.dev.sm_count || tiles * kb + other_tiles * other_kb >= 10 * c.dev.sm_count ? F8_PAIR : F8_ROWS;
}

// `x` (or null): A [M, K] in x_type, to be quantised into A, as by f8_gemm_launch, or
// by the rows kernel on the way.
mmact_status f8_gemm_plan(F8Plan &plan, const F8Matrix &A, const F8Matrix &B, const float *bias, void *C, int64_t M,
                          int64_t N, int64_t K, mmact_dtype cd, mmact_act act, float alpha, const void *x = nullptr,
                          mmact_dtype x_type = MMACT_F32, int kernel = F8_ANY)
{
    F8Context c;
    const mmact_status st = f8_context(&c);
    if (st != MMACT_OK) return st;
    const int nk32 = (int)((K + 31) / 32), num_kb = (int)f8_blocks(K);
    plan.pair = kernel == F8_ANY ? f8_choose_pair(c, M, N, K) : kernel == F8_PAIR;
    plan.A = A;
    plan.B = B;
    plan.x_type = -1;
    plan.quantize = x != nullptr && plan.pair;
    if (plan.pair) {
        F8Problem &L = plan.P;
        std::memset(&L, 0, sizeof(L));
        L.M = (int)M;
        L.N = (int)N;
        L.nk32 = nk32;
        L.num_kb = num_kb;
        L.chunk_kb = cd == MMACT_F32 ? F8_CHUNK_KB : (num_kb + 3) & ~3;
        L.tiles_m = (int)((M + 255) / 256);
        L.tiles_n = (int)((N + 255) / 256);
        L.num_tiles = L.tiles_m * L.tiles_n;
        L.group_m = 8;
        L.act = (int)act;
        L.alpha = alpha;
        L.bias = bias;
        L.C = C;
        L.idesc = ptx::idesc_f8(f8_kind(A.type), f8_kind(B.type), 256, 256);
        const int ce = elem_bytes(cd);
        L.c_tma = N * ce % 16 == 0 ? 1 : 0;
        L.out = out_kind(cd);
        if (!f8_encode(&L.tmA, &L.tmSA, A, M, K, 128, 1) || !f8_encode(&L.tmB, &L.tmSB, B, N, K, 128, 2)) return MMACT_ERR_CUDA;
        if (L.c_tma) {
            const uint64_t dC[2] = {(uint64_t)N, (uint64_t)M}, sC[1] = {(uint64_t)N * ce};
            const uint32_t bC[2] = {(uint32_t)(128 / ce), 32};
            if (!encode_tensor_map(&L.tmC, cd, 2, C, dC, sC, bC, true)) return MMACT_ERR_CUDA;
        }
        return MMACT_OK;
    }
    F8RowsProblem &a = plan.R;
    std::memset(&a, 0, sizeof(a));
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.nk32 = nk32;
    a.num_kb = num_kb;
    a.tiles_n = (int)((N + 127) / 128);
    a.act = (int)act;
    a.out = out_kind(cd);
    a.alpha = alpha;
    a.bias = bias;
    a.C = C;
    if ((int64_t)a.tiles_n * ((M + 15) / 16) * 8 > MAX_DIM) return MMACT_ERR_UNSUPPORTED;
    plan.quantize = x != nullptr && M > F8_FUSED_ROWS;
    if (x != nullptr && !plan.quantize) {
        a.x = x;
        plan.x_type = out_kind(x_type);
    }
    return MMACT_OK;
}

// K blocks of a CTA from which on the rings are deep, so that an SM holds one CTA.  Measured
// for 1 and 16 rows: 64 of 128 weight rows' tiles of K = 8192 (32 K blocks a CTA) 15.8 and 17.6
// us with rings of ten stages, 16.1 and 19.2 with five and two CTAs to an SM; 16 tiles of the same
// K 9.0 and 8.0, 64 tiles of K = 2048 7.4 and 6.9.
constexpr int F8_DEEP_KB = 24;

// Lays out the tiles of one or two products on the rows kernel.
mmact_status f8_rows_layout(F8RowsLaunch &L, const F8Context &c, const F8Plan &one, const F8Plan *two)
{
    std::memset(&L, 0, sizeof(L));
    F8RowsArgs &a = L.args;
    a.prob[0] = one.R;
    if (two != nullptr) a.prob[1] = two->R;
    const int n = two != nullptr ? 2 : 1, sms = c.dev.sm_count;
    // the narrowest tile that takes every row (a narrower one than 128 has to be the only one)
    int bt = 16, num_kb = a.prob[0].num_kb;
    int64_t tiles = 0;
    for (int i = 0; i < n; ++i) {
        while (bt < 128 && bt < a.prob[i].M) bt *= 2;
        num_kb = std::min(num_kb, a.prob[i].num_kb);
    }
    for (int i = 0; i < n; ++i) {
        a.prob[i].num_tiles = a.prob[i].tiles_n * ((a.prob[i].M + bt - 1) / bt);
        tiles += a.prob[i].num_tiles;
    }
    if (tiles * 8 > MAX_DIM) return MMACT_ERR_UNSUPPORTED;
    // CTAs to a tile: as long as that leaves no cluster waiting for SMs and each CTA two K blocks;
    // of few rows and short K blocks, two CTAs to an SM.
    int split = 1, log2 = 0;
    while (split < 8 && tiles * split * 2 <= sms && tiles <= c.max_clusters[log2 + 1] && num_kb >= split * 4) split *= 2, ++log2;
    if (bt == 16)
        while (split < 8 && tiles * split * 2 <= 2 * sms && num_kb >= split * 4 && num_kb < split * F8_DEEP_KB) split *= 2;
    // of two products, no CTA of the longer one with more than 32 K blocks (gradients of 8192 x 2048 x 128, 64 tiles of 16 K blocks
    // and 16 of 64: 39.7 us, 45.5 without; one product alone is the slower for it: 128 x 8192 x 16384 36.4, 29.6 without)
    for (int i = 0; i < n && n == 2; ++i)
        while (split < 8 && a.prob[i].num_kb > split * 32) split *= 2;
    // no CTA without a K block
    auto idle = [&](int s) {
        for (int i = 0; i < n; ++i) {
            const int kb = a.prob[i].num_kb, per = (kb + s - 1) / s;
            if ((s - 1) * per >= kb) return true;
        }
        return false;
    };
    while (split > 1 && idle(split)) split /= 2;
    int most = 0;
    for (int i = 0; i < n; ++i) {
        F8RowsProblem &p = a.prob[i];
        F8RowsMaps &m = a.maps[i];
        const F8Plan &plan = i == 0 ? one : *two;
        p.kb_per = (p.num_kb + split - 1) / split;
        p.chunk_kb = p.out == OUT_F32 ? F8_CHUNK_KB : p.num_kb;
        L.chunks = L.chunks || p.kb_per > p.chunk_kb;
        most = std::max(most, p.kb_per);
        // the operands change sides: B's rows are the instruction's A
        p.idesc = ptx::idesc_f8(f8_kind(plan.B.type), f8_kind(plan.A.type), 128, bt);
        if (!f8_encode(&m.tmW, &m.tmSW, plan.B, p.N, p.K, 128, 1)) return MMACT_ERR_CUDA;
        if (plan.x_type < 0 && !f8_encode(&m.tmT, &m.tmST, plan.A, p.M, p.K, (uint32_t)bt, 1)) return MMACT_ERR_CUDA;
    }
    a.stages = std::min(bt <= 32 && most < F8_DEEP_KB ? 5 : F8_ROWS_STAGES(bt), most);
    a.split = split;
    a.status = c.dev.status;
    a.wait_ns = c.dev.wait_ns;
    L.bt = bt;
    L.x_type = one.x_type;
    L.grid = (int)(tiles * split);
    return MMACT_OK;
}

// What one or two products enqueue: at most one launch of each kernel.
struct F8Launch {
    bool rows;
    int pairs;                       // 0: none of the pair kernel
    F8GemmArgs P;
    F8RowsLaunch R;
};

// Lays out a product, or two that do not depend on each other (`other`, or null).
mmact_status f8_gemm_layout(F8Launch &L, const F8Plan &plan, const F8Plan *other)
{
    F8Context c;
    const mmact_status s = f8_context(&c);
    if (s != MMACT_OK) return s;
    const F8Plan *on[2] = {nullptr, nullptr}, *few[2] = {nullptr, nullptr};    // of the pair kernel; of the rows kernel
    int non = 0, nfew = 0;
    for (const F8Plan *q : {&plan, other})
        if (q != nullptr) (q->pair ? on[non++] : few[nfew++]) = q;
    L.rows = nfew != 0;
    L.pairs = 0;
    if (non != 0) {
        F8GemmArgs &a = L.P;
        std::memset(&a, 0, sizeof(a));
        // the one with the longer tiles first: the others fill the last round
        if (non == 2 && on[1]->P.num_kb > on[0]->P.num_kb) std::swap(on[0], on[1]);
        for (int i = 0; i < non; ++i) {
            a.prob[i] = on[i]->P;
            a.tiles[i] = a.prob[i].num_tiles;
        }
        if (non == 2) a.lead = std::max(1, (a.prob[0].num_kb + a.prob[1].num_kb / 2) / a.prob[1].num_kb);
        a.status = c.dev.status;
        a.wait_ns = c.dev.wait_ns;
        L.pairs = (int)std::min<int64_t>((int64_t)a.tiles[0] + a.tiles[1], c.max_pairs);
    }
    return nfew != 0 ? f8_rows_layout(L.R, c, *few[0], few[1]) : MMACT_OK;
}

cudaError_t f8_gemm_launch(const F8Launch &L, cudaStream_t stream)
{
    const cudaError_t e = L.pairs != 0 ? launch_gemm_fp8_pair(L.P, L.pairs, stream) : cudaSuccess;
    return e == cudaSuccess && L.rows ? launch_gemm_fp8_rows(L.R, stream) : e;
}

cudaError_t quantize_launch(const void *x, const F8Matrix &m, int64_t rows, int64_t K, mmact_dtype xd, bool square,
                            bool transposed, cudaStream_t stream)
{
    return launch_quantize_fp8(x, out_kind(xd), static_cast<uint8_t *>(const_cast<void *>(m.codes)),
                               static_cast<uint8_t *>(const_cast<void *>(m.scales)), rows, K, f8_kind(m.type), square,
                               transposed, stream);
}

// Takes consecutive parts of a workspace, each from a multiple of 512 bytes.
struct Parts {
    char *base;
    int64_t at = 0;
    void *take(int64_t bytes)
    {
        char *here = base + at;
        at += round_up(bytes, 512);
        return here;
    }
    F8Matrix matrix(int64_t rows, int64_t K, mmact_dtype type)
    {
        void *codes = take(f8_codes_bytes(rows, K));
        return F8Matrix{codes, take(f8_scales_bytes(rows, K)), type};
    }
};

int64_t linear_bytes(int64_t M, int64_t K)
{
    return round_up(f8_codes_bytes(M, K), 512) + f8_scales_bytes(M, K);
}

// More tiles of 128 x 128 than are counted in 32 bits.
bool backward_too_large(int64_t M, int64_t N, int64_t K)
{
    const int64_t tm = (M + 127) / 128, tn = (N + 127) / 128, tk = (K + 127) / 128;
    return tm * tk > MAX_DIM || tn * tk > MAX_DIM || tm * tn > MAX_DIM;
}

// dy by rows, dy and x by columns, partial column sums
int64_t backward_bytes(int64_t M, int64_t N, int64_t K)
{
    return linear_bytes(M, N) + linear_bytes(N, M) + linear_bytes(K, M) + round_up((M + 127) / 128 * N * 4, 512);
}

}  // namespace
}  // namespace mmact

using namespace mmact;

MMACT_EXPORT mmact_status mmact_fp8_size(int64_t rows, int64_t K, int64_t *codes_bytes, int64_t *scales_bytes)
{
    if (!mx_dims(rows, K) || codes_bytes == nullptr || scales_bytes == nullptr) return MMACT_ERR_INVALID_ARG;
    *codes_bytes = f8_codes_bytes(rows, K);
    *scales_bytes = f8_scales_bytes(rows, K);
    return MMACT_OK;
}

MMACT_EXPORT mmact_status mmact_quantize_fp8(const void *x, void *codes, void *scales, int64_t rows, int64_t K,
                                             mmact_dtype x_dtype, mmact_dtype code_dtype, int64_t block_rows, int transposed,
                                             void *stream)
{
    if (!mx_dims(rows, K) || !valid_float(x_dtype) || !valid_f8(code_dtype)) return MMACT_ERR_INVALID_ARG;
    if (block_rows != 1 && block_rows != 128) return MMACT_ERR_INVALID_ARG;
    if (rows == 0 || K == 0) return MMACT_OK;
    if (x == nullptr || codes == nullptr || scales == nullptr) return MMACT_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return MMACT_ERR_UNSUPPORTED;
    return enqueued(quantize_launch(x, F8Matrix{codes, scales, code_dtype}, rows, K, x_dtype, block_rows == 128,
                                    transposed != 0, static_cast<cudaStream_t>(stream)));
}

MMACT_EXPORT mmact_status mmact_dequantize_fp8(const void *codes, const void *scales, void *y, int64_t rows, int64_t K,
                                               mmact_dtype code_dtype, mmact_dtype y_dtype, void *stream)
{
    if (!mx_dims(rows, K) || !valid_float(y_dtype) || !valid_f8(code_dtype)) return MMACT_ERR_INVALID_ARG;
    if (rows == 0 || K == 0) return MMACT_OK;
    if (codes == nullptr || scales == nullptr || y == nullptr) return MMACT_ERR_INVALID_ARG;
    if (!aligned16(codes) || !aligned16(scales) || !aligned16(y)) return MMACT_ERR_UNSUPPORTED;
    DeviceContext dev;
    const mmact_status st = device_context(&dev);
    if (st != MMACT_OK) return st;
    return enqueued(launch_dequantize_fp8(static_cast<const uint8_t *>(codes), static_cast<const uint8_t *>(scales), y,
                                          out_kind(y_dtype), rows, K, f8_kind(code_dtype), dev.sm_count,
                                          static_cast<cudaStream_t>(stream)));
}

MMACT_EXPORT mmact_status mmact_gemm_fp8(const void *a_codes, const void *a_scales, const void *b_codes, const void *b_scales,
                                         const float *bias, void *C, int64_t M, int64_t N, int64_t K, mmact_dtype a_dtype,
                                         mmact_dtype b_dtype, mmact_dtype c_dtype, mmact_act act, float alpha, void *stream)
{
    const F8Matrix A{a_codes, a_scales, a_dtype}, B{b_codes, b_scales, b_dtype};
    mmact_status s = f8_gemm_check(A, B, bias, C, M, N, K, c_dtype, act);
    if (s != MMACT_OK) return s;
    if (M == 0 || N == 0) return MMACT_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (K == 0) return enqueued(launch_mx_bias_act(bias, C, M, N, out_kind(c_dtype), (int)act, alpha, st));
    F8Plan plan;
    F8Launch L;
    if ((s = f8_gemm_plan(plan, A, B, bias, C, M, N, K, c_dtype, act, alpha)) != MMACT_OK) return s;
    if ((s = f8_gemm_layout(L, plan, nullptr)) != MMACT_OK) return s;
    return enqueued(f8_gemm_launch(L, st));
}

MMACT_EXPORT mmact_status mmact_set_gemm_fp8_kernel(int mode)
{
    if (mode < 0 || mode > 2) return MMACT_ERR_INVALID_ARG;
    g_f8_kernel.store(mode);
    return MMACT_OK;
}

MMACT_EXPORT mmact_status mmact_linear_fp8_workspace_bytes(int64_t M, int64_t K, int64_t *bytes)
{
    if (!mx_dims(M, K) || bytes == nullptr) return MMACT_ERR_INVALID_ARG;
    *bytes = linear_bytes(M, K);
    return MMACT_OK;
}

MMACT_EXPORT mmact_status mmact_linear_fp8(const void *x, const void *w_codes, const void *w_scales, const float *bias,
                                           void *C, int64_t M, int64_t N, int64_t K, mmact_dtype x_dtype, mmact_dtype w_dtype,
                                           mmact_dtype c_dtype, mmact_act act, float alpha, void *workspace, void *stream)
{
    if (!mx_dims(M, K) || !valid_float(x_dtype)) return MMACT_ERR_INVALID_ARG;
    if ((x == nullptr || workspace == nullptr) && M * K != 0) return MMACT_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(workspace)) return MMACT_ERR_UNSUPPORTED;
    Parts ws{static_cast<char *>(workspace)};
    const F8Matrix A = M * K != 0 ? ws.matrix(M, K, MMACT_E4M3) : F8Matrix{workspace, workspace, MMACT_E4M3};
    const F8Matrix W{w_codes, w_scales, w_dtype};
    mmact_status s = f8_gemm_check(A, W, bias, C, M, N, K, c_dtype, act);
    if (s != MMACT_OK) return s;
    if (M == 0 || N == 0) return MMACT_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (K == 0) return enqueued(launch_mx_bias_act(bias, C, M, N, out_kind(c_dtype), (int)act, alpha, st));
    F8Plan plan;
    F8Launch L;
    if ((s = f8_gemm_plan(plan, A, W, bias, C, M, N, K, c_dtype, act, alpha, x, x_dtype)) != MMACT_OK) return s;
    if ((s = f8_gemm_layout(L, plan, nullptr)) != MMACT_OK) return s;
    if (plan.quantize && (s = enqueued(quantize_launch(x, A, M, K, x_dtype, false, false, st))) != MMACT_OK) return s;
    return enqueued(f8_gemm_launch(L, st));
}

MMACT_EXPORT mmact_status mmact_linear_fp8_backward_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t *bytes)
{
    if (!mx_dims(M, K) || !mx_dims(N, K) || bytes == nullptr) return MMACT_ERR_INVALID_ARG;
    if (backward_too_large(M, N, K)) return MMACT_ERR_UNSUPPORTED;
    *bytes = backward_bytes(M, N, K);
    return MMACT_OK;
}

MMACT_EXPORT mmact_status mmact_linear_fp8_backward(const void *dy, const void *x, const void *wt_codes, const void *wt_scales,
                                                    void *dx, void *dw, float *db, int64_t M, int64_t N, int64_t K,
                                                    mmact_dtype x_dtype, mmact_dtype wt_dtype, mmact_dtype grad_dtype,
                                                    mmact_dtype dw_dtype, void *workspace, void *stream)
{
    if (!mx_dims(M, K) || !mx_dims(N, K)) return MMACT_ERR_INVALID_ARG;
    if (!valid_float(x_dtype) || !valid_f8(wt_dtype) || !valid_f8(grad_dtype) || !valid_float(dw_dtype))
        return MMACT_ERR_INVALID_ARG;
    const bool any = dx != nullptr || dw != nullptr || db != nullptr;
    if (any && (dy == nullptr || workspace == nullptr) && M * N != 0) return MMACT_ERR_INVALID_ARG;
    if (dx != nullptr && (wt_codes == nullptr || wt_scales == nullptr) && M != 0 && N * K != 0) return MMACT_ERR_INVALID_ARG;
    if (dw != nullptr && (x == nullptr || workspace == nullptr) && M * K != 0 && N != 0) return MMACT_ERR_INVALID_ARG;
    if (db != nullptr && !aligned4(db)) return MMACT_ERR_INVALID_ARG;
    if (!aligned16(dy) || !aligned16(x) || !aligned16(wt_codes) || !aligned16(wt_scales) || !aligned16(dx) ||
        !aligned16(dw) || !aligned16(workspace))
        return MMACT_ERR_UNSUPPORTED;
    if (backward_too_large(M, N, K)) return MMACT_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    mmact_status s = MMACT_OK;
    const bool want_dx = dx != nullptr && M * K != 0, want_dw = dw != nullptr && N * K != 0, want_db = db != nullptr && N != 0;
    // sums over nothing are zeros
    if (want_dx && N == 0) return enqueued(launch_mx_bias_act(nullptr, dx, M, K, out_kind(x_dtype), 0, 0.0f, st));
    if (M == 0) {
        if (want_dw) s = enqueued(launch_mx_bias_act(nullptr, dw, N, K, out_kind(dw_dtype), 0, 0.0f, st));
        if (s == MMACT_OK && want_db) s = enqueued(launch_mx_bias_act(nullptr, db, 1, N, OUT_F32, 0, 0.0f, st));
        return s;
    }
    Parts ws{static_cast<char *>(workspace)};
    const F8Matrix gy = ws.matrix(M, N, grad_dtype), gyt = ws.matrix(N, M, grad_dtype), xt = ws.matrix(K, M, MMACT_E4M3);
    float *part = static_cast<float *>(ws.take(0));
    F8Plan X, W;
    int kernel = F8_ANY;
    if (want_dx && want_dw) {
        F8Context c;
        if ((s = f8_context(&c)) != MMACT_OK) return s;
        const bool dx_pair = f8_choose_pair(c, M, K, N), dw_pair = f8_choose_pair(c, N, K, M);
        if (dw_pair && !dx_pair) kernel = f8_shared_kernel(c, M, K, N, f8_row_tiles(N, K), f8_blocks(M));
        if (dx_pair && !dw_pair) kernel = f8_shared_kernel(c, N, K, M, f8_row_tiles(M, K), f8_blocks(N));
    }
    if (want_dx && (s = f8_gemm_plan(X, gy, F8Matrix{wt_codes, wt_scales, wt_dtype}, nullptr, dx, M, K, N, x_dtype,
                                     MMACT_ACT_NONE, 0.0f, nullptr, MMACT_F32, kernel)) != MMACT_OK)
        return s;
    if (want_dw && (s = f8_gemm_plan(W, gyt, xt, nullptr, dw, N, K, M, dw_dtype, MMACT_ACT_NONE, 0.0f, nullptr,
                                     MMACT_F32, kernel)) != MMACT_OK)
        return s;
    F8Launch L;
    const bool products = want_dx || want_dw;
    if (products && (s = f8_gemm_layout(L, want_dw ? W : X, want_dw && want_dx ? &X : nullptr)) != MMACT_OK) return s;
    F8Grads g;
    std::memset(&g, 0, sizeof(g));
    g.dy = dy;
    g.x = x;
    g.M = M;
    g.N = N;
    g.K = K;
    auto bytes = [](const void *p) { return static_cast<uint8_t *>(const_cast<void *>(p)); };
    if (want_dx) g.row_codes = bytes(gy.codes), g.row_scales = bytes(gy.scales);
    if (want_dw) {
        g.col_codes = bytes(gyt.codes), g.col_scales = bytes(gyt.scales);
        g.xt_codes = bytes(xt.codes), g.xt_scales = bytes(xt.scales);
    }
    if (want_db) g.part = part;
    if ((s = enqueued(launch_quantize_fp8_grads(g, out_kind(x_dtype), f8_kind(grad_dtype), st))) != MMACT_OK) return s;
    if (want_db && (s = enqueued(launch_column_sums(part, db, M, N, st))) != MMACT_OK) return s;
    return products ? enqueued(f8_gemm_launch(L, st)) : MMACT_OK;
}
