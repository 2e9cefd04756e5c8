// kernels_fp8.h -- host-side view of the 8-bit floating-point kernels.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "mmact.h"

namespace mmact {

// x [rows, K] (trans: [K, rows]) of type OUT_* -> codes, scales; square: blocks of 128 x 128.
cudaError_t launch_quantize_fp8(const void *x, int type, uint8_t *codes, uint8_t *scales, int64_t rows, int64_t K, int f8,
                                bool square, bool trans, cudaStream_t s);
cudaError_t launch_dequantize_fp8(const uint8_t *codes, const uint8_t *scales, void *y, int type, int64_t rows, int64_t K,
                                  int f8, int sms, cudaStream_t s);

// out [cols] = column sums of x [rows, cols].  part: [ceil(rows / 128)][cols] fp32
cudaError_t launch_column_sums(const void *x, int type, float *part, float *out, int64_t rows, int64_t cols, cudaStream_t s);

// Product of two 8-bit matrices with the fused epilogue.
struct F8GemmArgs {
    int M, N;
    int nk32;            // K steps of 32 (one instruction each) that hold values
    int tiles_m, tiles_n, num_tiles, num_kb;   // num_kb: K blocks of 128 (one ring stage each)
    int group_m;
    int act;
    float alpha;
    const float *bias;   // [N] or null
    void *C;
    int c_tma;           // 1: output tiles by TMA store, 0: element stores (row pitch not a multiple of 16 bytes)
    uint32_t idesc;      // operand formats, 256 x 256
    unsigned int *status;
    unsigned long long wait_ns;
};

struct F8GemmLaunch {
    CUtensorMap tmA, tmB, tmSA, tmSB, tmC;   // codes as 16-bit words, scale tiles as 32-bit words
    F8GemmArgs args;
    int out;
    int grid;
};

cudaError_t setup_fp8_pair_kernels(int *max_pairs);   // max_pairs: CTA pairs resident at once
cudaError_t launch_gemm_fp8_pair(const F8GemmLaunch &L, cudaStream_t stream);

// The same product with few rows or tiles: W = B's rows on the MMA's 128 lanes,
// T = A's rows on its columns, the K blocks of a tile shared by a cluster.
struct F8RowsArgs {
    int M, N, K;
    const void *x;       // A not yet quantised [M, K], or null
    int nk32, num_kb;    // as above
    int tiles_n;         // tiles of 128 rows of B
    int split, kb_per;   // CTAs of a tile's cluster, K blocks of each
    int stages;          // of the ring
    int act;
    float alpha;
    const float *bias;
    void *C;
    uint32_t idesc;      // operand formats, 128 x bt
    unsigned int *status;
    unsigned long long wait_ns;
};

struct F8RowsLaunch {
    CUtensorMap tmW, tmT, tmSW, tmST;
    F8RowsArgs args;
    int out;
    int bt;              // rows of A in a tile: 16, 32, 64 or 128
    int x_type;          // OUT_* of args.x; < 0: A is tmT, tmST
    int grid;
};

// max_clusters[i]: clusters of 2^i CTAs resident at once, one CTA to an SM
cudaError_t setup_fp8_rows_kernels(int (&max_clusters)[4]);
cudaError_t launch_gemm_fp8_rows(const F8RowsLaunch &L, cudaStream_t stream);

}  // namespace mmact
