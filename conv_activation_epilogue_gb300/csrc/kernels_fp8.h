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

// What the backward pass of a linear layer makes of dy [M, N] and x [M, K]; null outputs
// are not wanted.
struct F8Grads {
    const void *dy, *x;
    int64_t M, N, K;
    uint8_t *row_codes, *row_scales;     // dy [M, N], blocks along N
    uint8_t *col_codes, *col_scales;     // dy turned round [N, M], blocks along M
    uint8_t *xt_codes, *xt_scales;       // x turned round [K, M], E4M3
    float *part;                         // column sums of 128 rows [ceil(M / 128)][N]
    int64_t dy_tiles;                    // set by the launch
};
cudaError_t launch_quantize_fp8_grads(F8Grads g, int type, int f8, cudaStream_t s);

// out [cols] = sums over all row blocks of part
cudaError_t launch_column_sums(const float *part, float *out, int64_t rows, int64_t cols, cudaStream_t s);

// Product of two 8-bit matrices with the fused epilogue.
struct F8Problem {
    CUtensorMap tmA, tmB, tmSA, tmSB, tmC;   // codes as 16-bit words, scale tiles as 32-bit words
    int M, N;
    int nk32;            // K steps of 32 (one instruction each) that hold values
    int tiles_m, tiles_n, num_tiles, num_kb;   // num_kb: K blocks of 128 (one ring stage each)
    int chunk_kb;        // of these summed in one accumulator: a multiple of 4
    int group_m;
    int act, out;        // out: OUT_* of C
    float alpha;
    const float *bias;   // [N] or null
    void *C;
    int c_tma;           // 1: output tiles by TMA store, 0: element stores (row pitch not a multiple of 16 bytes)
    uint32_t idesc;      // operand formats, 256 x 256
};

// One product, or two that do not depend on each other and share the CTA pairs.
struct F8GemmArgs {
    F8Problem prob[2];
    int tiles[2];        // of each (0: no second product)
    int lead;            // tiles of the second in the time of one of the first
    unsigned int *status;
    unsigned long long wait_ns;
};

cudaError_t setup_fp8_pair_kernels(int *max_pairs);   // max_pairs: CTA pairs resident at once
cudaError_t launch_gemm_fp8_pair(const F8GemmArgs &a, int pairs, cudaStream_t stream);

// The same product with few rows or tiles: W = B's rows on the MMA's 128 lanes,
// T = A's rows on its columns, the K blocks of a tile shared by a cluster.
struct F8RowsProblem {
    int M, N, K;
    int nk32, num_kb;    // as above
    int tiles_n;         // tiles of 128 rows of B
    int num_tiles;
    int kb_per;          // K blocks of a CTA of the tile's cluster
    int chunk_kb;        // of these summed in one accumulator
    int act, out;
    float alpha;
    uint32_t idesc;      // operand formats, 128 x bt
    const float *bias;
    const void *x;       // A not yet quantised [M, K], or null
    void *C;
};

struct F8RowsMaps {
    CUtensorMap tmW, tmT, tmSW, tmST;
};

// One product, or two that do not depend on each other.  What every thread reads is
// together at the front: the first reads of a kernel's arguments miss.
struct F8RowsArgs {
    int split;           // CTAs of a tile's cluster
    int stages;          // of the ring
    unsigned int *status;
    unsigned long long wait_ns;
    F8RowsProblem prob[2];
    F8RowsMaps maps[2];
};

struct F8RowsLaunch {
    F8RowsArgs args;
    int bt;              // rows of A in a tile: 16, 32, 64 or 128
    int x_type;          // OUT_* of the first product's x; < 0: its A is tmT, tmST
    bool chunks;         // some CTA has more K blocks than an accumulator takes
    int grid;
};

// max_clusters[i]: clusters of 2^i CTAs resident at once, one CTA to an SM
cudaError_t setup_fp8_rows_kernels(int (&max_clusters)[4]);
cudaError_t launch_gemm_fp8_rows(const F8RowsLaunch &L, cudaStream_t stream);

}  // namespace mmact
