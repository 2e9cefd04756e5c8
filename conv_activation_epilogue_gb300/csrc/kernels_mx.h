// kernels_mx.h -- host-side view of the MXFP4 and mixture-of-experts kernels.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mmact.h"
#include "mx_layout.h"

namespace mmact {

cudaError_t launch_quantize_mxfp4(const void *x, int type, uint8_t *codes, uint8_t *scales, int64_t rows, int64_t K,
                                  bool trans, cudaStream_t s);
cudaError_t launch_dequantize_mxfp4(const uint8_t *codes, const uint8_t *scales, void *y, int type, int64_t rows,
                                    int64_t K, int sms, cudaStream_t s);

// Product of two MXFP4 matrices with the fused epilogue.
struct MxGemmArgs {
    int M, N;
    int nk64;            // K steps of 64 (one instruction each) that hold values
    int tiles_m, tiles_n, num_tiles, num_kb;   // num_kb: K blocks of 256 (one ring stage each)
    int group_m;
    int act;
    float alpha;
    const float *bias;   // [N] or null
    void *C;
    int c_tma;           // 1: output tiles by TMA store, 0: element stores (row pitch not a multiple of 16 bytes)
    unsigned int *status;
    unsigned long long wait_ns;
};

struct MxGemmLaunch {
    CUtensorMap tmA, tmB, tmSA, tmSB, tmC;   // codes as 16-bit words, scale tiles as 32-bit words
    MxGemmArgs args;
    int out;
    int grid;
};

cudaError_t setup_mxfp4_pair_kernels(int *max_pairs);   // max_pairs: CTA pairs resident at once
cudaError_t launch_gemm_mxfp4_pair(const MxGemmLaunch &L, cudaStream_t stream);

// The same product with few rows or tiles: W = B's rows on the MMA's 128 lanes,
// T = A's rows on its columns, the K blocks of a tile shared by a cluster.
struct MxRowsArgs {
    int M, N, K;
    const void *x;       // A not yet quantised [M, K], or null
    int nk64, num_kb;    // as above
    int tiles_n;         // tiles of 128 rows of B
    int split, kb_per;   // CTAs of a tile's cluster, K blocks of each
    int stages;          // of the ring
    int act;
    float alpha;
    const float *bias;
    void *C;
    unsigned int *status;
    unsigned long long wait_ns;
};

struct MxRowsLaunch {
    CUtensorMap tmW, tmT, tmSW, tmST;
    MxRowsArgs args;
    int out;
    int bt;              // rows of A in a tile: 16, 32, 64 or 128
    int x_type;          // OUT_* of args.x; < 0: A is tmT, tmST
    int grid;
};

// max_clusters[i]: clusters of 2^i CTAs resident at once, one CTA to an SM
cudaError_t setup_mxfp4_rows_kernels(int (&max_clusters)[4]);
cudaError_t launch_gemm_mxfp4_rows(const MxRowsLaunch &L, cudaStream_t stream);

// A mixture-of-experts layer for a few tokens.
struct MoeArgs {
    int T, H, I, E, top;         // tokens, model width, experts' width, experts, experts per token
    int R1;                      // rows of one expert's w1: 2 I when gated, else I
    int half_rows;               // rows of half a tile of weights: a multiple of 8, 64 at most
    int Hp, Ip;                  // H and I rounded up to whole ring stages (row pitches of the workspace's arrays)
    int gated, normalize, act;
    float alpha;
    const void *x, *router;      // [T, H], [E, H]
    const void *w1, *w2;         // [E, R1, H], [E, H, I] (MXFP4: codes of [E * R1, H], [E * H, I])
    const void *s1, *s2;         // MXFP4: scale tiles of the same
    const float *router_bias, *b1, *b2;   // [E], [E, R1], [E, H], or null
    void *y;                     // [T, H]
    int *experts;                // [T, top]
    float *probs;                // [T, top]
    // workspace
    unsigned int *counters;      // two grid barriers
    float *logits;               // [T, E]
    uint16_t *x_pad;             // 16-bit weights: x [T, Hp], zeros past H
    uint16_t *h;                 // 16-bit weights: h as three bf16 parts, [T * top][Ip / 128][3][128]
    uint8_t *x_codes, *x_scales; // MXFP4: x and h as sums of eight MXFP4 terms: a KB of codes and 64
    uint8_t *h_codes, *h_scales; //   scales for each token (slot) and 256 K
    float *part;                 // [T * top, H]
    unsigned int *status;
    unsigned long long wait_ns;
};

struct MoeLaunch {
    CUtensorMap tm1, tm2;   // w1, w2: boxes of half_rows rows x 128 bytes
    MoeArgs args;
    int x_out;           // OUT_* of x, the router and y
    int grid;            // CTAs of the experts kernel: one for each SM at most
};

cudaError_t setup_moe_kernels();
cudaError_t launch_moe(const MoeLaunch &L, cudaStream_t stream);          // 16-bit weights
cudaError_t setup_moe_mxfp4_kernels();
cudaError_t launch_moe_mxfp4(const MoeLaunch &L, cudaStream_t stream);    // half_rows 64

// out [rows, cols] = act(bias): a product over an empty K.
cudaError_t launch_mx_bias_act(const float *bias, void *out, int64_t rows, int64_t cols, int out_kind, int act,
                               float alpha, cudaStream_t stream);

}  // namespace mmact
