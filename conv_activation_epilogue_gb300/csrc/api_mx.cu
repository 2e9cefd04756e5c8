// api_mx.cu -- the C ABI of the MXFP4 and mixture-of-experts operators
// (include/mmact.h): argument validation and launch planning.  As in api.cu,
// every check happens on the host before anything is enqueued.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>

#include "api_checks.h"
#include "api_internal.h"
#include "common.cuh"
#include "kernels_mx.h"
#include "mmact.h"
#include "mxfp4.cuh"

#define MMACT_EXPORT extern "C" __attribute__((visibility("default")))

namespace mmact {
namespace {

std::atomic<int> g_mx_kernel{0};   // 0: chosen per shape; 1: rows kernel; 2: pair kernel

// The current device, with this file's kernels set up on it (once per device).
struct MxContext {
    DeviceContext dev;
    int max_pairs;                   // CTA pairs of the pair kernel resident at once
    const int *max_clusters;         // [i]: clusters of 2^i CTAs of the rows kernel
};

mmact_status mx_context(MxContext *out)
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
            (setup_mxfp4_pair_kernels(&pairs[dev]) != cudaSuccess || setup_mxfp4_rows_kernels(clusters[dev]) != cudaSuccess ||
             setup_moe_kernels() != cudaSuccess || setup_moe_mxfp4_kernels() != cudaSuccess))
            return MMACT_ERR_CUDA;
        ready[dev].store(true, std::memory_order_release);
    }
    out->max_pairs = pairs[dev];
    out->max_clusters = clusters[dev];
    return MMACT_OK;
}

int64_t mx_codes_bytes(int64_t rows, int64_t K) { return rows * (mx_blocks(K) * 16); }
int64_t mx_scales_bytes(int64_t rows, int64_t K) { return (rows + 127) / 128 * mx_tiles(K) * 512; }

mmact_status mx_gemm_check(const void *ac, const void *as, const void *bc, const void *bs, const float *bias,
                           const void *C, int64_t M, int64_t N, int64_t K, mmact_dtype cd, mmact_act act)
{
    if (!mx_dims(M, K) || !mx_dims(N, K)) return MMACT_ERR_INVALID_ARG;
    if (((ac == nullptr || as == nullptr) && M * K != 0) || ((bc == nullptr || bs == nullptr) && N * K != 0) ||
        (C == nullptr && M * N != 0))
        return MMACT_ERR_INVALID_ARG;
    if (!valid_float(cd) || !valid_act(act)) return MMACT_ERR_INVALID_ARG;
    if (bias != nullptr && !aligned4(bias)) return MMACT_ERR_INVALID_ARG;
    if (!aligned16(ac) || !aligned16(as) || !aligned16(bc) || !aligned16(bs) || !aligned16(C))
        return MMACT_ERR_UNSUPPORTED;
    if (((M + 127) / 128) * ((N + 127) / 128) > MAX_DIM) return MMACT_ERR_UNSUPPORTED;
    return MMACT_OK;
}

// Tensor maps of an MXFP4 matrix: its codes as 16-bit words (box 64 words = 256
// codes x `box_rows` rows, 128-byte swizzle) and its scale tiles as 32-bit words
// (box 256 words = two tiles = 256 K, of `box_tiles` rows of tiles).  Rows, codes and tiles past the
// end arrive as zeros.
bool mx_encode(CUtensorMap *mc, CUtensorMap *ms, const void *codes, const void *scales, int64_t rows, int64_t K,
               uint32_t box_rows, uint32_t box_tiles)
{
    const uint64_t dc[2] = {(uint64_t)mx_blocks(K) * 8, (uint64_t)rows}, sc[1] = {(uint64_t)mx_blocks(K) * 16};
    const uint32_t bc[2] = {64, box_rows};
    const uint64_t ds[2] = {(uint64_t)mx_tiles(K) * 128, (uint64_t)(rows + 127) / 128};
    const uint64_t ss[1] = {(uint64_t)mx_tiles(K) * 512};
    const uint32_t bs[2] = {256, box_tiles};
    return encode_tensor_map(mc, MMACT_BF16, 2, codes, dc, sc, bc, true) &&
           encode_tensor_map(ms, MMACT_F32, 2, scales, ds, ss, bs, false);
}

// Plan of one product: either kernel's launch.
struct MxPlan {
    bool pair, quantize;             // quantize: x first, by a kernel of its own
    MxGemmLaunch P;
    MxRowsLaunch R;
};

// Whether a product runs on the pair kernel: when the rows kernel would have more
// tiles (128 x 128) than there are SMs.  Measured on GB300 for M from 160 to 4096,
// N from 256 to 8192 and K of 256, 1024 and 4096: up to one tile an SM the rows
// kernel is 15 % faster (K = 256: 5.4 against 6.2 us), equal (K = 1024) or up to
// 25 % faster (K = 4096: 8.0 against 10.2); past that the pair kernel is up to
// twice and more as fast (1024 x 4096 x 4096: 11.3 against 20.8 us).
bool mx_choose_pair(const MxContext &c, int64_t M, int64_t N)
{
    const int mode = g_mx_kernel.load();
    if (c.max_pairs < 1 || mode == 1) return false;
    if (mode == 2) return true;
    return M > 128 && ((M + 127) / 128) * ((N + 127) / 128) > c.dev.sm_count;
}

// Rows of x up to which the rows kernel quantises them itself (gemm_mxfp4_rows.cu
// has both sides' times).
constexpr int64_t MX_FUSED_ROWS = 8;

// `x` (or null): A [M, K] in x_type, to be quantised into ac, as by mx_gemm_launch,
// or by the rows kernel on the way.
mmact_status mx_gemm_plan(MxPlan &plan, const void *ac, const void *as, const void *bc, const void *bs,
                          const float *bias, void *C, int64_t M, int64_t N, int64_t K, mmact_dtype cd, mmact_act act,
                          float alpha, const void *x = nullptr, mmact_dtype x_type = MMACT_F32)
{
    MxContext c;
    const mmact_status st = mx_context(&c);
    if (st != MMACT_OK) return st;
    const int nk64 = (int)((mx_blocks(K) + 1) / 2), num_kb = (int)((K + 255) / 256);
    plan.pair = mx_choose_pair(c, M, N);
    plan.quantize = x != nullptr && plan.pair;
    if (plan.pair) {
        MxGemmLaunch &L = plan.P;
        std::memset(&L, 0, sizeof(L));
        MxGemmArgs &a = L.args;
        a.M = (int)M;
        a.N = (int)N;
        a.nk64 = nk64;
        a.num_kb = num_kb;
        a.tiles_m = (int)((M + 255) / 256);
        a.tiles_n = (int)((N + 255) / 256);
        a.num_tiles = a.tiles_m * a.tiles_n;
        a.group_m = 8;
        a.act = (int)act;
        a.alpha = alpha;
        a.bias = bias;
        a.C = C;
        a.status = c.dev.status;
        a.wait_ns = c.dev.wait_ns;
        const int ce = elem_bytes(cd);
        a.c_tma = N * ce % 16 == 0 ? 1 : 0;
        L.out = out_kind(cd);
        L.grid = 2 * (int)std::min<int64_t>(a.num_tiles, c.max_pairs);
        if (!mx_encode(&L.tmA, &L.tmSA, ac, as, M, K, 128, 1) || !mx_encode(&L.tmB, &L.tmSB, bc, bs, N, K, 128, 2))
            return MMACT_ERR_CUDA;
        if (a.c_tma) {
            const uint64_t dC[2] = {(uint64_t)N, (uint64_t)M}, sC[1] = {(uint64_t)N * ce};
            const uint32_t bC[2] = {(uint32_t)(128 / ce), 32};
            if (!encode_tensor_map(&L.tmC, cd, 2, C, dC, sC, bC, true)) return MMACT_ERR_CUDA;
        }
        return MMACT_OK;
    }
    MxRowsLaunch &L = plan.R;
    std::memset(&L, 0, sizeof(L));
    MxRowsArgs &a = L.args;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.nk64 = nk64;
    a.num_kb = num_kb;
    a.tiles_n = (int)((N + 127) / 128);
    const int sms = c.dev.sm_count;
    // the narrowest tile that takes every row (a narrower one than 128 has to be the only one)
    int bt = 16;
    while (bt < 128 && bt < M) bt *= 2;
    const int64_t tiles = a.tiles_n * ((M + bt - 1) / bt);
    if (tiles * 8 > MAX_DIM) return MMACT_ERR_UNSUPPORTED;
    // CTAs to a tile: as long as that leaves no cluster waiting for SMs and each CTA two K blocks
    int split = 1, log2 = 0;
    while (split < 8 && tiles * split * 2 <= sms && tiles <= c.max_clusters[log2 + 1] && num_kb >= split * 2) split *= 2, ++log2;
    a.kb_per = (num_kb + split - 1) / split;
    while (split > 1 && (split - 1) * a.kb_per >= num_kb) split /= 2, a.kb_per = (num_kb + split - 1) / split;
    a.stages = std::min(MX_ROWS_STAGES(bt), a.kb_per);
    a.split = split;
    a.act = (int)act;
    a.alpha = alpha;
    a.bias = bias;
    a.C = C;
    a.status = c.dev.status;
    a.wait_ns = c.dev.wait_ns;
    L.out = out_kind(cd);
    L.bt = bt;
    L.grid = (int)(tiles * split);
    L.x_type = -1;
    plan.quantize = x != nullptr && M > MX_FUSED_ROWS;
    if (!mx_encode(&L.tmW, &L.tmSW, bc, bs, N, K, 128, 1)) return MMACT_ERR_CUDA;
    if (x != nullptr && !plan.quantize) {
        a.x = x;
        L.x_type = out_kind(x_type);
        return MMACT_OK;
    }
    return mx_encode(&L.tmT, &L.tmST, ac, as, M, K, (uint32_t)bt, 1) ? MMACT_OK : MMACT_ERR_CUDA;
}

cudaError_t mx_gemm_launch(const MxPlan &plan, cudaStream_t stream)
{
    return plan.pair ? launch_gemm_mxfp4_pair(plan.P, stream) : launch_gemm_mxfp4_rows(plan.R, stream);
}

cudaError_t quantize_launch(const void *x, void *codes, void *scales, int64_t rows, int64_t K, mmact_dtype xd,
                            int transposed, cudaStream_t stream)
{
    return launch_quantize_mxfp4(x, out_kind(xd), static_cast<uint8_t *>(codes), static_cast<uint8_t *>(scales), rows, K,
                                 transposed != 0, stream);
}

constexpr int64_t MOE_K_PAD = 256;   // whole stages of either form of the weights

// Where the parts of mmact_moe's workspace begin.
struct MoeWorkspace {
    int64_t logits, x, x_scales, h, h_scales, part, bytes;
};

// The same for both forms of the weights: x padded (2 bytes a value) or its terms
// (4 bytes a value and a quarter), h in three parts (6 bytes) or its terms.
MoeWorkspace moe_workspace(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top)
{
    MoeWorkspace w;
    const int64_t Hp = round_up(H, MOE_K_PAD), Ip = round_up(I, MOE_K_PAD);
    int64_t at = 256;                                          // two counters
    auto take = [&at](int64_t bytes) {
        const int64_t here = at;
        at += round_up(bytes, 256);
        return here;
    };
    w.logits = take(T * E * 4);
    w.x = take(T * Hp * 4);
    w.x_scales = take(T * Hp / 4);
    w.h = take(T * top * Ip * 6);
    w.h_scales = take(T * top * Ip / 4);
    w.part = take(T * top * H * 4);
    w.bytes = at;
    return w;
}

// Boxes of `box_rows` rows x 128 bytes of the experts' weights (the rows of all
// experts as one matrix; MXFP4 codes as 16-bit words).
bool moe_encode(CUtensorMap *map, const void *w, int64_t rows, int64_t K, bool mx, int box_rows)
{
    const uint64_t row_bytes = (uint64_t)(mx ? mx_blocks(K) * 16 : K * 2);
    const uint64_t d[2] = {row_bytes / 2, (uint64_t)rows}, st[1] = {row_bytes};
    const uint32_t box[2] = {64, (uint32_t)box_rows};
    return encode_tensor_map(map, MMACT_BF16, 2, w, d, st, box, true);
}

constexpr int64_t MOE_MAX_TOKENS = 64, MOE_MAX_TOP = 16, MOE_MAX_EXPERTS = 512;

mmact_status moe_sizes(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top)
{
    if (T < 0 || H < 0 || I < 0 || E < 0 || top < 0 || H > MAX_DIM || I > MAX_DIM) return MMACT_ERR_INVALID_ARG;
    if (T > MOE_MAX_TOKENS || E > MOE_MAX_EXPERTS || top < 1 || top > MOE_MAX_TOP || top > E || H < 8 || I < 8 ||
        H % 8 != 0 || I % 8 != 0)
        return MMACT_ERR_UNSUPPORTED;
    // rows of the experts' matrices, and H and I up to whole stages, are counted in 32 bits
    if (E * 2 * I > MAX_DIM - MOE_K_PAD || E * H > MAX_DIM - MOE_K_PAD) return MMACT_ERR_UNSUPPORTED;
    return MMACT_OK;
}

// Half the rows of a tile of 16-bit weights: the one with which the busiest SM has
// the least to do, counted in rows x K.  Smaller tiles pay where they save a round of
// the SMs or bring all of them to work (cold caches): 16 tokens, 2 of 16 experts of 4096 x 1792,
// 116 us with tiles of 128 rows, 107 with 112; one token, 2 of 8 experts of the same, 43.6
// and 39.2 us with 64 rows.  Where they do not they cost: 32 tokens, 6 of 64 experts of
// 2048 x 1408, 186 us with 128 rows, 199 with 64 (a ring stage takes as long as one of 72
// rows at least).  The number of chosen experts is not known here: it is taken as what
// random choices give.
int moe_half_rows(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top, bool gated, int sms)
{
    const int64_t chosen = std::llround((double)E * (1.0 - std::pow(1.0 - (double)top / (double)E, (double)T)));
    int best = 64;
    double least = 0;
    for (int half = 64; half >= 32; half -= 8) {
        const int64_t step = gated ? half : 2 * half, up = chosen * ((I + step - 1) / step);
        const int64_t down = chosen * ((H + 2 * half - 1) / (2 * half));
        const double cost = (double)std::max(2 * half, 72) *
                            ((double)((up + sms - 1) / sms) * (double)H + (double)((down + sms - 1) / sms) * (double)I);
        if (half == 64 || cost < 0.97 * least) least = cost, best = half;
    }
    return best;
}

}  // namespace
}  // namespace mmact

using namespace mmact;

MMACT_EXPORT mmact_status mmact_mxfp4_size(int64_t rows, int64_t K, int64_t *codes_bytes, int64_t *scales_bytes)
{
    if (!mx_dims(rows, K) || codes_bytes == nullptr || scales_bytes == nullptr) return MMACT_ERR_INVALID_ARG;
    *codes_bytes = mx_codes_bytes(rows, K);
    *scales_bytes = mx_scales_bytes(rows, K);
    return MMACT_OK;
}

MMACT_EXPORT mmact_status mmact_quantize_mxfp4(const void *x, void *codes, void *scales, int64_t rows, int64_t K,
                                               mmact_dtype x_dtype, int transposed, void *stream)
{
    if (!mx_dims(rows, K) || !valid_float(x_dtype)) return MMACT_ERR_INVALID_ARG;
    if (rows == 0 || K == 0) return MMACT_OK;
    if (x == nullptr || codes == nullptr || scales == nullptr) return MMACT_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return MMACT_ERR_UNSUPPORTED;
    return enqueued(quantize_launch(x, codes, scales, rows, K, x_dtype, transposed, static_cast<cudaStream_t>(stream)));
}

MMACT_EXPORT mmact_status mmact_dequantize_mxfp4(const void *codes, const void *scales, void *y, int64_t rows, int64_t K,
                                                 mmact_dtype y_dtype, void *stream)
{
    if (!mx_dims(rows, K) || !valid_float(y_dtype)) return MMACT_ERR_INVALID_ARG;
    if (rows == 0 || K == 0) return MMACT_OK;
    if (codes == nullptr || scales == nullptr || y == nullptr) return MMACT_ERR_INVALID_ARG;
    if (!aligned16(codes) || !aligned16(scales) || !aligned16(y)) return MMACT_ERR_UNSUPPORTED;
    DeviceContext dev;
    const mmact_status st = device_context(&dev);
    if (st != MMACT_OK) return st;
    return enqueued(launch_dequantize_mxfp4(static_cast<const uint8_t *>(codes), static_cast<const uint8_t *>(scales), y,
                                            out_kind(y_dtype), rows, K, dev.sm_count, static_cast<cudaStream_t>(stream)));
}

MMACT_EXPORT mmact_status mmact_gemm_mxfp4(const void *a_codes, const void *a_scales, const void *b_codes,
                                           const void *b_scales, const float *bias, void *C, int64_t M, int64_t N,
                                           int64_t K, mmact_dtype c_dtype, mmact_act act, float alpha, void *stream)
{
    mmact_status s = mx_gemm_check(a_codes, a_scales, b_codes, b_scales, bias, C, M, N, K, c_dtype, act);
    if (s != MMACT_OK) return s;
    if (M == 0 || N == 0) return MMACT_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (K == 0) return enqueued(launch_mx_bias_act(bias, C, M, N, out_kind(c_dtype), (int)act, alpha, st));
    MxPlan L;
    s = mx_gemm_plan(L, a_codes, a_scales, b_codes, b_scales, bias, C, M, N, K, c_dtype, act, alpha);
    return s == MMACT_OK ? enqueued(mx_gemm_launch(L, st)) : s;
}

MMACT_EXPORT mmact_status mmact_set_gemm_mxfp4_kernel(int mode)
{
    if (mode < 0 || mode > 2) return MMACT_ERR_INVALID_ARG;
    g_mx_kernel.store(mode);
    return MMACT_OK;
}

MMACT_EXPORT mmact_status mmact_linear_mxfp4_workspace_bytes(int64_t M, int64_t K, int64_t *bytes)
{
    if (!mx_dims(M, K) || bytes == nullptr) return MMACT_ERR_INVALID_ARG;
    *bytes = round_up(mx_codes_bytes(M, K), 512) + mx_scales_bytes(M, K);
    return MMACT_OK;
}

MMACT_EXPORT mmact_status mmact_linear_mxfp4(const void *x, const void *w_codes, const void *w_scales, const float *bias,
                                             void *C, int64_t M, int64_t N, int64_t K, mmact_dtype x_dtype,
                                             mmact_dtype c_dtype, mmact_act act, float alpha, void *workspace,
                                             void *stream)
{
    if (!mx_dims(M, K) || !valid_float(x_dtype)) return MMACT_ERR_INVALID_ARG;
    if ((x == nullptr || workspace == nullptr) && M * K != 0) return MMACT_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(workspace)) return MMACT_ERR_UNSUPPORTED;
    uint8_t *codes = static_cast<uint8_t *>(workspace);
    uint8_t *scales = M * K != 0 ? codes + round_up(mx_codes_bytes(M, K), 512) : codes;
    mmact_status s = mx_gemm_check(codes, scales, w_codes, w_scales, bias, C, M, N, K, c_dtype, act);
    if (s != MMACT_OK) return s;
    if (M == 0 || N == 0) return MMACT_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (K == 0) return enqueued(launch_mx_bias_act(bias, C, M, N, out_kind(c_dtype), (int)act, alpha, st));
    MxPlan L;
    if ((s = mx_gemm_plan(L, codes, scales, w_codes, w_scales, bias, C, M, N, K, c_dtype, act, alpha, x, x_dtype)) !=
        MMACT_OK)
        return s;
    if (L.quantize && (s = enqueued(quantize_launch(x, codes, scales, M, K, x_dtype, 0, st))) != MMACT_OK) return s;
    return enqueued(mx_gemm_launch(L, st));
}

MMACT_EXPORT mmact_status mmact_moe_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top,
                                                    int64_t *bytes)
{
    if (bytes == nullptr) return MMACT_ERR_INVALID_ARG;
    const mmact_status s = moe_sizes(T, H, I, E, top);
    if (s != MMACT_OK) return s;
    *bytes = moe_workspace(T, H, I, E, top).bytes;
    return MMACT_OK;
}

MMACT_EXPORT mmact_status mmact_moe(const void *x, const void *router, const float *router_bias, const void *w1,
                                    const void *w1_scales, const float *b1, const void *w2, const void *w2_scales,
                                    const float *b2, void *y, int32_t *experts, float *probs, int64_t T, int64_t H,
                                    int64_t I, int64_t E, int64_t top, mmact_dtype x_dtype, mmact_dtype w_dtype,
                                    mmact_act act, float alpha, int gated, int normalize, void *workspace, void *stream)
{
    if (!valid_16(x_dtype) || !valid_act(act)) return MMACT_ERR_INVALID_ARG;
    if (w_dtype < MMACT_F16 || w_dtype > MMACT_MXFP4) return MMACT_ERR_INVALID_ARG;
    mmact_status s = moe_sizes(T, H, I, E, top);
    if (s != MMACT_OK) return s;
    const bool mx = w_dtype == MMACT_MXFP4;
    if (!mx && w_dtype != x_dtype) return MMACT_ERR_UNSUPPORTED;
    if (T == 0) return MMACT_OK;
    if (x == nullptr || router == nullptr || w1 == nullptr || w2 == nullptr || y == nullptr || experts == nullptr ||
        probs == nullptr || workspace == nullptr || (mx && (w1_scales == nullptr || w2_scales == nullptr)))
        return MMACT_ERR_INVALID_ARG;
    if ((router_bias != nullptr && !aligned4(router_bias)) || (b1 != nullptr && !aligned4(b1)) ||
        (b2 != nullptr && !aligned4(b2)) || !aligned4(experts) || !aligned4(probs))
        return MMACT_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(router) || !aligned16(w1) || !aligned16(w2) || !aligned16(y) ||
        !aligned16(workspace) || (mx && (!aligned16(w1_scales) || !aligned16(w2_scales))))
        return MMACT_ERR_UNSUPPORTED;
    MxContext c;
    if ((s = mx_context(&c)) != MMACT_OK) return s;
    MoeLaunch L;
    std::memset(&L, 0, sizeof(L));
    MoeArgs &a = L.args;
    a.T = (int)T;
    a.H = (int)H;
    a.I = (int)I;
    a.E = (int)E;
    a.top = (int)top;
    a.gated = gated != 0;
    a.normalize = normalize != 0;
    a.R1 = (int)(a.gated ? 2 * I : I);
    a.Hp = (int)round_up(H, MOE_K_PAD);
    a.Ip = (int)round_up(I, MOE_K_PAD);
    a.act = (int)act;
    a.alpha = alpha;
    a.x = x;
    a.router = router;
    a.w1 = w1;
    a.w2 = w2;
    a.s1 = w1_scales;
    a.s2 = w2_scales;
    a.router_bias = router_bias;
    a.b1 = b1;
    a.b2 = b2;
    a.y = y;
    a.experts = experts;
    a.probs = probs;
    const MoeWorkspace w = moe_workspace(T, H, I, E, top);
    char *ws = static_cast<char *>(workspace);
    a.counters = reinterpret_cast<unsigned int *>(ws);
    a.logits = reinterpret_cast<float *>(ws + w.logits);
    if (mx) {
        a.x_codes = reinterpret_cast<uint8_t *>(ws + w.x);
        a.x_scales = reinterpret_cast<uint8_t *>(ws + w.x_scales);
        a.h_codes = reinterpret_cast<uint8_t *>(ws + w.h);
        a.h_scales = reinterpret_cast<uint8_t *>(ws + w.h_scales);
    } else {
        a.x_pad = reinterpret_cast<uint16_t *>(ws + w.x);
        a.h = reinterpret_cast<uint16_t *>(ws + w.h);
    }
    a.part = reinterpret_cast<float *>(ws + w.part);
    a.status = c.dev.status;
    a.wait_ns = c.dev.wait_ns;
    L.x_out = out_kind(x_dtype);
    a.half_rows = mx ? 64 : moe_half_rows(T, H, I, E, top, gated != 0, c.dev.sm_count);
    L.grid = c.dev.sm_count;
    if (!moe_encode(&L.tm1, w1, E * a.R1, H, mx, a.half_rows) || !moe_encode(&L.tm2, w2, E * H, I, mx, a.half_rows))
        return MMACT_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return enqueued(mx ? launch_moe_mxfp4(L, st) : launch_moe(L, st));
}
