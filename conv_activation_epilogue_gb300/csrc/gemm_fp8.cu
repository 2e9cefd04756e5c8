// gemm_fp8.cu -- C = act(A x B^T + bias) of two matrices in 8-bit floating point with a
// scale for each block of 128 (fp8.cuh), A [M, K] and B [N, K], for large outputs:
// 256 x 256 tiles on CTA pairs, tcgen05.mma.cta_group::2.kind::mxf8f6f4.
//
// A ring stage is 128 K of the CTA's 128 rows of A and 128 rows of B (16 KB each, by TMA
// with the 128-byte swizzle).  A scale tile holds the scales of 512 K: every fourth
// stage brings the tiles of its own A rows and of all B rows, the MMA issuer copies them
// into tensor memory (tcgen05.cp) ahead of the stage's MMAs, and the instructions of the
// four stages pick their byte.
//
// Tensor memory: two 256-column accumulators that overlap by 32 columns (0..255 and
// 224..479), then two slots of 12 columns of scales.  Copies and MMAs of one issuer run
// in order, so a slot is free again when its next copy comes.  The epilogue of a tile
// takes the shared columns first and lets the next tile's MMAs start as soon as they are
// in registers, before it works on them.
//
// The tensor core cuts off what an addition to the accumulator has below its last bit
// (always towards zero: sums of 8192 positive products came out 3.9e-6 too small).  Far
// below a 16-bit output's rounding; for fp32 outputs a tile's K is summed in chunks of
// 2048, each in a fresh accumulator, and the epilogue's warps add the chunks up in
// registers, rounded.  A weight's gradient over 8192 tokens of different sizes is then 9e-7
// off (2-norm; with chunks of 4096 2.0e-6, of 1024 4e-7), and the backward pass that
// it belongs to takes 232 us (224 and 253; 8192^3 alone, into fp32, 367: 340 and 447).
//
// Two products that do not depend on each other (a linear layer's two gradients) can share
// one launch: the pairs go on from the tiles of the one to the tiles of the other, instead
// of waiting twice for the slowest.
//
//   warp 0      (both CTAs) TMA producer; copies complete on the even CTA's barriers
//   warp 1      TMEM allocation; in the even CTA the scale copies and the MMAs
//   warps 2..9  (both CTAs) epilogue of the CTA's 128 rows, two warps for each 32
//
// Bound by the tensor pipe and, called for longer, the power cap.  Measured with calls back
// to back, LeakyReLU, bf16 out: 8192 x 8192 x 8192 306 to 313 us (3.5 to 3.6 PFLOP/s; a stage takes 336
// ns, and about a microsecond passes between tiles; after seconds of it 356 to 364),
// 4096 x 4096 x 4096 45.3 us, 9728 x 8192 x 512 51 us.
//
// Every wait is bounded, and both CTAs pass a final cluster barrier before TMEM
// is released.
#include "common.cuh"
#include "fp8.cuh"
#include "kernels_fp8.h"
#include "mx_epilogue.cuh"
#include "mx_layout.h"

namespace mmact {

struct F8PairCfg {
    static constexpr int A_BYTES = 128 * 128, B_BYTES = 128 * 128;       // 128 K of 128 rows
    static constexpr int S_BYTES = 3 * 512;                              // A: 512 bytes, B: 1 KB
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + S_BYTES;
    static constexpr int EPI_WARPS = 8, EPI_BYTES = EPI_WARPS * 4096;
    static constexpr int STAGES = 5;
    static constexpr int THREADS = 64 + 32 * EPI_WARPS;
    static constexpr uint32_t ACC_STRIDE = 224, SCALE_COL = 480, SLOT_COLS = 12, TMEM_COLS = 512;
    static constexpr int OFF_A = 0;
    static constexpr int OFF_B = OFF_A + STAGES * A_BYTES;
    static constexpr int OFF_EPI = OFF_B + STAGES * B_BYTES;
    static constexpr int OFF_S = OFF_EPI + EPI_BYTES;
    static constexpr int OFF_BAR = OFF_S + STAGES * S_BYTES;
    static constexpr int OFF_MISC = OFF_BAR + (2 * STAGES + 4) * 8;
    static constexpr int SMEM_BYTES = OFF_MISC + 16;
    static_assert(SMEM_BYTES <= CTA_SMEM && SMEM_BYTES >= tmem_min_smem((int)TMEM_COLS), "shared memory budget");
    static_assert(SCALE_COL + 2 * SLOT_COLS <= TMEM_COLS && SCALE_COL >= ACC_STRIDE + 256, "tensor memory budget");
};

// Tile t of a product -> (M block, N block) of 256 x 256, grouped M-first.
__device__ __forceinline__ void f8_tile(int t, const F8Problem &p, int &mb, int &nb)
{
    const int per_group = p.group_m * p.tiles_n;
    const int g = t / per_group;
    const int m_first = g * p.group_m;
    const int gm = min(p.tiles_m - m_first, p.group_m);
    const int r = t - g * per_group;
    mb = m_first + r % gm;
    nb = r / gm;
}

// A pair's i-th tile: of the first product in rounds of all pairs, then of the second.
// In the first's last round some pairs have no tile; they begin with the second, `lead`
// rounds of their own.  False when there is none.
__device__ __forceinline__ bool f8_schedule(int i, int pair, int npairs, const F8GemmArgs &p, int &which, int &t)
{
    const int rest = p.tiles[0] % npairs, own = p.tiles[0] / npairs + (pair < rest ? 1 : 0);
    which = 0;
    t = pair + i * npairs;
    if (i < own) return true;
    which = 1;
    i -= own;
    const int early = rest != 0 ? npairs - rest : 0, ahead = early * p.lead;
    if (early != 0 && pair >= rest && i < p.lead) t = i * early + pair - rest;
    else t = ahead + (i - (early != 0 && pair >= rest ? p.lead : 0)) * npairs + pair;
    return t < p.tiles[1];
}

// The epilogue of one tile: this warp's 32 rows, every other unit of columns.
template <int OUT>
__device__ __forceinline__ void f8_epilogue(const F8Problem &p, int mb, int nb, uint32_t rank, bool upper, int part, uint32_t tbase,
                                            uint32_t buf, int lane, int row0, uint32_t tempty, uint32_t tempty_leader)
{
    constexpr int COLS = OUT == OUT_F32 ? 32 : 64;
    constexpr int NU = 256 / COLS;                            // units of a tile
    const uint64_t pol_c = ptx::createpolicy_evict_first();   // C is not read back here
    // the shared columns are the last of the lower accumulator and the first of the upper one
    const int first = upper ? 0 : NU - 1;
#pragma unroll 1
    for (int i = part; i < NU; i += 2) {
        const int u = (first + i) & (NU - 1);
        const int col0 = nb * 256 + u * COLS;
        if (lane == 0) ptx::bulk_wait_read<0>();
        __syncwarp();
        mx_epi_unit<OUT>(p.act, tbase + u * COLS, p.bias != nullptr ? p.bias + col0 : nullptr, p.N - col0, p.alpha, buf, lane, [&] {
            // The warp's first unit: the shared columns are the first unit of the warps that have them, and every
            // warp is past the tile before.
            if (i != part) return;
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (rank == 0) ptx::mbar_arrive(tempty);
                else ptx::mbar_arrive_cluster(tempty_leader);
            }
        });
        if (p.c_tma) {
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && row0 < p.M && col0 < p.N) {
                ptx::tma_store_2d_hint(&p.tmC, buf, col0, row0, pol_c);
                ptx::bulk_commit();
            }
        } else {
            __syncwarp();
            mx_store_elements<OUT>(p.C, buf, row0, col0, p.M, p.N, lane);
            __syncwarp();
        }
    }
}

// The epilogue of one tile in several chunks of K, fp32 output: the warp's 32 rows and
// every other 32 columns (units u = 2 k + part).  `chunk` counts the accumulators used
// so far.  False when a wait ran out.
__device__ __forceinline__ bool f8_epilogue_chunks(const F8Problem &p, const Pipe &pp, uint32_t &chunk, int chunks, int nb, uint32_t rank,
                                                   int part, uint32_t tmem, uint32_t buf, int lane, int row0,
                                                   uint32_t tempty_leader)
{
    const uint64_t pol_c = ptx::createpolicy_evict_first();
    float sum[4][32];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < 32; ++j) sum[k][j] = 0.0f;
#pragma unroll 1
    for (int c = 0; c < chunks; ++c, ++chunk) {
        if (!warp_epi_wait(pp, pp.tfull0 + 8 * (chunk & 1u), (chunk >> 1) & 1u)) return false;
        ptx::tc_fence_after();
        const uint32_t base = tmem + (chunk & 1u) * F8PairCfg::ACC_STRIDE + part * 32;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // the shared columns are the first or the last unit
            const int k = i < 2 ? 0 : (i < 4 ? 3 : i / 2 - 1), h = (i & 1) * 16;
            uint32_t r[16];
            ptx::tmem_ld16(base + 64 * k + h, r);
            if (i == 3) {
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (rank == 0) ptx::mbar_arrive(pp.tempty0);
                    else ptx::mbar_arrive_cluster(tempty_leader);
                }
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) sum[k][h + j] += __uint_as_float(r[j]);
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int col0 = nb * 256 + 64 * k + 32 * part;
        if (lane == 0) ptx::bulk_wait_read<0>();
        __syncwarp();
        if (p.bias != nullptr)
#pragma unroll
            for (int j = 0; j < 32; ++j) sum[k][j] += col0 + j < p.N ? p.bias[col0 + j] : 0.0f;
        act_mx_all(p.act, sum[k], p.alpha);
#pragma unroll
        for (int c = 0; c < 8; ++c)
            ptx::st_shared_v4(buf + (uint32_t)lane * 128u + (((uint32_t)c ^ (uint32_t)(lane & 7)) << 4), __float_as_uint(sum[k][4 * c]),
                              __float_as_uint(sum[k][4 * c + 1]), __float_as_uint(sum[k][4 * c + 2]), __float_as_uint(sum[k][4 * c + 3]));
        if (p.c_tma) {
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && row0 < p.M && col0 < p.N) {
                ptx::tma_store_2d_hint(&p.tmC, buf, col0, row0, pol_c);
                ptx::bulk_commit();
            }
        } else {
            __syncwarp();
            mx_store_elements<OUT_F32>(p.C, buf, row0, col0, p.M, p.N, lane);
            __syncwarp();
        }
    }
    return true;
}

// CHUNKS: some product sums its K in several accumulators (its sums take the epilogue's
// registers, 9728 x 8192 x 512 in bf16 55 us with it, 51 without).
template <bool CHUNKS>
__global__ void __launch_bounds__(F8PairCfg::THREADS, 1) gemm_fp8_pair_kernel(const __grid_constant__ F8GemmArgs p)
{
    using Cfg = F8PairCfg;
    constexpr int STAGES = Cfg::STAGES;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t base = ptx::smem_addr(smem);
    const uint32_t rank = ptx::cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = (int)(blockIdx.x >> 1), npairs = (int)(gridDim.x >> 1);

    ptx::griddep_launch_dependents();
    const bool aligned = (base & 1023u) == 0;
    if (!aligned && threadIdx.x == 0) atomicOr(p.status, ST_SMEM_ALIGN);

    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + Cfg::OFF_MISC);
    Pipe pp;
    pp.full0 = base + Cfg::OFF_BAR;
    pp.empty0 = pp.full0 + 8 * STAGES;
    pp.tfull0 = pp.empty0 + 8 * STAGES;       // two, one for each accumulator
    pp.tempty0 = pp.tfull0 + 16;              // one: the shared columns of the last tile are drained
    pp.drain = pp.tempty0 + 8;
    pp.abort = misc + 1;
    pp.status = p.status;
    pp.wait_ns = p.wait_ns;
    if (aligned) {
        if (threadIdx.x == 0) {
            ptx::prefetch_tensormap(&p.prob[0].tmA);
            ptx::prefetch_tensormap(&p.prob[0].tmB);
            for (int s = 0; s < STAGES; ++s) {
                ptx::mbar_init(pp.full0 + 8 * s, 1);
                ptx::mbar_init(pp.empty0 + 8 * s, 1);
            }
            ptx::mbar_init(pp.tfull0, 1);
            ptx::mbar_init(pp.tfull0 + 8, 1);
            ptx::mbar_init(pp.tempty0, 2 * Cfg::EPI_WARPS);
            ptx::mbar_init(pp.drain, 1);
            misc[1] = 0;
            ptx::fence_mbar_init();
        }
        if (warp == 1) {
            ptx::tmem_alloc_pair(base + Cfg::OFF_MISC, Cfg::TMEM_COLS);
            ptx::tmem_relinquish_pair();
        }
    }
    ptx::tc_fence_before();
    ptx::cta_sync();
    ptx::tc_fence_after();
    ptx::cluster_sync();
    pp.tmem = misc[0];
    // the pair's MMAs address both CTAs' tensor memory by the even CTA's columns
    const bool usable = aligned && ptx::ld_cluster_u32(ptx::mapa(base + Cfg::OFF_MISC, rank ^ 1u)) == pp.tmem;
    if (aligned && !usable && threadIdx.x == 0) atomicOr(p.status, ST_PAIR_TMEM);
    ptx::griddep_wait();
    const uint32_t sA = base + Cfg::OFF_A, sB = base + Cfg::OFF_B, sS = base + Cfg::OFF_S;
    ptx::cluster_sync();

    if (usable && warp == 0) {
        if (lane == 0) {
            uint32_t stage = 0, phase = 0;
            bool ok = true;
            for (int i = 0, w, t; ok && f8_schedule(i, pair, npairs, p, w, t); ++i) {
                const F8Problem &q = p.prob[w];
                int mb, nb;
                f8_tile(t, q, mb, nb);
                for (int kb = 0; kb < q.num_kb; ++kb) {
                    if (!pipe_wait(pp, pp.empty0 + 8 * stage, phase ^ 1u)) { ok = false; break; }
                    const uint32_t fb = pp.full0 + 8 * stage;
                    const bool scales = (kb & 3) == 0;
                    if (leader) ptx::mbar_arrive_expect_tx(fb, 2u * (scales ? Cfg::STAGE_BYTES : Cfg::A_BYTES + Cfg::B_BYTES));
                    const uint32_t to = ptx::mapa(fb, 0);
                    ptx::tma_load_2d_pair(sA + stage * Cfg::A_BYTES, &q.tmA, to, kb * 64, mb * 256 + (int)rank * 128);
                    ptx::tma_load_2d_pair(sB + stage * Cfg::B_BYTES, &q.tmB, to, kb * 64, nb * 256 + (int)rank * 128);
                    if (scales) {
                        ptx::tma_load_2d_pair(sS + stage * Cfg::S_BYTES, &q.tmSA, to, (kb >> 2) * 128, mb * 2 + (int)rank);
                        ptx::tma_load_2d_pair(sS + stage * Cfg::S_BYTES + 512u, &q.tmSB, to, (kb >> 2) * 128, nb * 2);
                    }
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            if (!ok) pipe_fail(pp);
        }
    } else if (usable && warp == 1) {
        if (leader) {                                         // the whole warp: see mma_mxf4
            const uint64_t a0 = ptx::smem_desc(sA, 16u, 1024u, ptx::SWIZZLE_128B), b0 = ptx::smem_desc(sB, 16u, 1024u, ptx::SWIZZLE_128B);
            const uint64_t s0 = ptx::smem_desc(sS, 16u, 128u, ptx::SWIZZLE_NONE);
            uint32_t stage = 0, phase = 0, tile = 0, slot = 0;
            bool ok = true;
            uint32_t chunk = 0;                                // accumulators used so far
            for (int w, t; ok && f8_schedule((int)tile, pair, npairs, p, w, t); ++tile) {
                const F8Problem &q = p.prob[w];
                const uint32_t idesc = q.idesc;
                const int num_kb = q.num_kb, nk32 = q.nk32, chunk_kb = q.chunk_kb;
                for (int kb = 0, left = 0; kb < num_kb; ++kb, --left) {
                    const uint32_t d = pp.tmem + (chunk & 1u) * Cfg::ACC_STRIDE;
                    const bool begin = left == 0;
                    if (begin) {
                        left = min(chunk_kb, num_kb - kb);
                        // the shared columns of the previous accumulator are read, and all of the one before it
                        if (chunk != 0 && !mx_warp_wait(pp, pp.tempty0, (chunk - 1) & 1u)) { ok = false; break; }
                        ptx::tc_fence_after();
                    }
                    if (!mx_warp_wait(pp, pp.full0 + 8 * stage, phase)) { ok = false; break; }
                    ptx::tc_fence_after();
                    const bool scales = (kb & 3) == 0;
                    if (scales) slot ^= 1u;
                    ptx::mma_f8_stage_pair(d, a0 + stage * (Cfg::A_BYTES >> 4), b0 + stage * (Cfg::B_BYTES >> 4),
                                           s0 + stage * (Cfg::S_BYTES >> 4), pp.tmem + Cfg::SCALE_COL + slot * Cfg::SLOT_COLS,
                                           idesc | ptx::f8_scale_id(kb), min(4, nk32 - 4 * kb), begin ? 0u : 1u, scales ? 1u : 0u);
                    ptx::commit_elected_pair(pp.empty0 + 8 * stage, 3);
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                    if (left == 1) ptx::commit_elected_pair(pp.tfull0 + 8 * (chunk++ & 1u), 3);
                }
            }
            if (!ok && lane == 0) pipe_fail(pp);
            ptx::commit_elected_pair(pp.drain, 1);
            ptx::mbar_wait_bounded(pp.drain, 0, DRAIN_NS, nullptr);
        }
    } else if (usable) {
        const int q = warp & 3, part = (warp - 2) >> 2;
        const uint32_t buf = base + Cfg::OFF_EPI + (uint32_t)(warp - 2) * 4096u;
        const uint32_t tempty_leader = ptx::mapa(pp.tempty0, 0);
        uint32_t tile = 0, chunk = 0;
        for (int w, t; f8_schedule((int)tile, pair, npairs, p, w, t); ++tile) {
            const F8Problem &o = p.prob[w];
            int mb, nb;
            f8_tile(t, o, mb, nb);
            const uint32_t lanes = pp.tmem + ((uint32_t)(q * 32) << 16);
            const int row0 = mb * 256 + (int)rank * 128 + q * 32;
            if constexpr (CHUNKS) {
                if (o.num_kb > o.chunk_kb) {
                    const int chunks = (o.num_kb + o.chunk_kb - 1) / o.chunk_kb;
                    if (!f8_epilogue_chunks(o, pp, chunk, chunks, nb, rank, part, lanes, buf, lane, row0, tempty_leader)) {
                        pipe_fail(pp);
                        break;
                    }
                    continue;
                }
            }
            if (!warp_epi_wait(pp, pp.tfull0 + 8 * (chunk & 1u), (chunk >> 1) & 1u)) { pipe_fail(pp); break; }
            ptx::tc_fence_after();
            const bool upper = (chunk & 1u) != 0;
            const uint32_t tbase = lanes + (upper ? Cfg::ACC_STRIDE : 0u);
            ++chunk;
            if (o.out == OUT_F32) f8_epilogue<OUT_F32>(o, mb, nb, rank, upper, part, tbase, buf, lane, row0, pp.tempty0, tempty_leader);
            else if (o.out == OUT_BF16) f8_epilogue<OUT_BF16>(o, mb, nb, rank, upper, part, tbase, buf, lane, row0, pp.tempty0, tempty_leader);
            else f8_epilogue<OUT_F16>(o, mb, nb, rank, upper, part, tbase, buf, lane, row0, pp.tempty0, tempty_leader);
        }
        if (lane == 0) ptx::bulk_wait<0>();
        __syncwarp();
    }

    // No commit, copy or arrival is still addressed to either CTA after this.
    ptx::tc_fence_before();
    ptx::cluster_sync();
    ptx::cta_sync();
    __syncwarp();
    if (aligned && warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(pp.tmem, Cfg::TMEM_COLS);
    }
}

static void pair_config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute (&attr)[2], int grid, cudaStream_t stream)
{
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(F8PairCfg::THREADS);
    cfg.dynamicSmemBytes = F8PairCfg::SMEM_BYTES;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
}

cudaError_t setup_fp8_pair_kernels(int *max_pairs)
{
    const auto smem = cudaFuncAttributeMaxDynamicSharedMemorySize;
    cudaError_t e = cudaFuncSetAttribute(gemm_fp8_pair_kernel<false>, smem, F8PairCfg::SMEM_BYTES);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(gemm_fp8_pair_kernel<true>, smem, F8PairCfg::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    pair_config(cfg, attr, 2 * 128, nullptr);
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(max_pairs, gemm_fp8_pair_kernel<true>, &cfg);
}

cudaError_t launch_gemm_fp8_pair(const F8GemmArgs &a, int pairs, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    pair_config(cfg, attr, 2 * pairs, stream);
    const bool chunks = a.prob[0].num_kb > a.prob[0].chunk_kb || (a.tiles[1] != 0 && a.prob[1].num_kb > a.prob[1].chunk_kb);
    return cudaLaunchKernelEx(&cfg, chunks ? gemm_fp8_pair_kernel<true> : gemm_fp8_pair_kernel<false>, a);
}

}  // namespace mmact
