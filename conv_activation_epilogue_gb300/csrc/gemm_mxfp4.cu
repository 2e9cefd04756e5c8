// gemm_mxfp4.cu -- C = act(A x B^T + bias) of two matrices in the 4-bit
// microscaled format (mxfp4.cuh), A [M, K] and B [N, K], for large outputs:
// 256 x 256 tiles on CTA pairs, tcgen05.mma.cta_group::2.kind::mxf4.
//
// The arithmetic runs four times as fast as in 16 bits and the operands are a
// quarter of the size, so the balance of a tile is that of the 16-bit pair
// kernel: a ring stage is 256 K (128-byte rows of codes) of the CTA's 128 rows of
// A and 128 rows of B, 16 KB each, by TMA with the 128-byte swizzle, plus 3 KB of
// scale tiles (its own A rows', all 256 B rows').  The MMA issuer copies the
// scale tiles into tensor memory (tcgen05.cp) ahead of the stage's MMAs.
//
// Tensor memory: the two 256-column accumulators overlap by 128 columns (0..255
// and 128..383), which leaves 24 columns of scales for each ring stage (a stage's
// columns are free when the stage is, so the issuer never waits for them; with
// two slots for five stages it did, 590 cycles a stage where the MMAs take 532).
// The epilogue of a tile takes the shared columns first, one half of its warps
// each half of them, and lets the next tile's MMAs start as soon as they are in
// registers, before it works on them.
//
//   warp 0      (both CTAs) TMA producer; copies complete on the even CTA's barriers
//   warp 1      TMEM allocation; in the even CTA the scale copies and the MMAs
//   warps 2..9  (both CTAs) epilogue of the CTA's 128 rows, two warps for each 32
//
// Bound by the tensor pipe.  Measured with calls back to back, LeakyReLU: 8192 x 8192 x 8192
// 157 us without a bias, 161 with one (7.0 and 6.8 PFLOP/s; the pipe is active 72 % of the time, a
// tile's 32 stages take 295 ns each and about 1.7 us pass between tiles), 4096 x 4096 x 4096 28.4 us.
// Heavier activations show, since the next tile's MMAs only wait for half of the
// columns: 8192^3 with GELU 190 us, SiLU 175; 4096 x 4096 x 1024 with LeakyReLU 15, GELU 26, SiLU 41.
//
// Every wait is bounded, and both CTAs pass a final cluster barrier before TMEM
// is released.
#include "common.cuh"
#include "kernels_mx.h"
#include "mxfp4.cuh"

namespace mmact {

struct MxPairCfg {
    static constexpr int A_BYTES = 128 * 128, B_BYTES = 128 * 128;       // 256 K of 128 rows
    static constexpr int S_BYTES = 3 * 1024;                             // A: 1 KB, B: 2 KB
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + S_BYTES;
    static constexpr int EPI_WARPS = 8, EPI_BYTES = EPI_WARPS * 4096;
    static constexpr int STAGES = 5;
    static constexpr int THREADS = 64 + 32 * EPI_WARPS;
    static constexpr uint32_t ACC_STRIDE = 128, SCALE_COL = 384, SLOT_COLS = 24, TMEM_COLS = 512;
    static constexpr int OFF_A = 0;
    static constexpr int OFF_B = OFF_A + STAGES * A_BYTES;
    static constexpr int OFF_EPI = OFF_B + STAGES * B_BYTES;
    static constexpr int OFF_S = OFF_EPI + EPI_BYTES;
    static constexpr int OFF_BAR = OFF_S + STAGES * S_BYTES;
    static constexpr int OFF_MISC = OFF_BAR + (2 * STAGES + 4) * 8;
    static constexpr int SMEM_BYTES = OFF_MISC + 16;
    static_assert(SMEM_BYTES <= CTA_SMEM && SMEM_BYTES >= tmem_min_smem((int)TMEM_COLS), "shared memory budget");
    static_assert(SCALE_COL + STAGES * SLOT_COLS <= TMEM_COLS, "tensor memory budget");
};

// Pair tile t -> (M block, N block) of 256 x 256, grouped M-first.
__device__ __forceinline__ void mx_tile(int t, const MxGemmArgs &p, int &mb, int &nb)
{
    const int per_group = p.group_m * p.tiles_n;
    const int g = t / per_group;
    const int m_first = g * p.group_m;
    const int gm = min(p.tiles_m - m_first, p.group_m);
    const int r = t - g * per_group;
    mb = m_first + r % gm;
    nb = r / gm;
}

// One epilogue unit: this warp's 32 rows x one 128-byte row segment (32 fp32 or
// 64 16-bit columns): accumulators from TMEM, + bias, activation, conversion,
// into a 32 x 128 B buffer in the 128-byte swizzled order of a TMA store.
// `loaded` is called when the accumulators are in registers.
template <int OUT, int ACT, typename Loaded>
__device__ __forceinline__ void mx_epi_unit(uint32_t taddr, const float *bias, int nvalid, float alpha, uint32_t buf,
                                            int lane, Loaded loaded)
{
    constexpr int HALVES = OUT == OUT_F32 ? 1 : 2;           // 32 columns at a time
    uint32_t r[HALVES][32];
#pragma unroll
    for (int h = 0; h < HALVES; ++h) ptx::tmem_ld32(taddr + 32 * h, r[h]);
#pragma unroll
    for (int h = 0; h < HALVES; ++h) ptx::tmem_ld_wait(r[h]);
    loaded();
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
        float b[32] = {};
        const float *src = bias + 32 * h;
        if (bias != nullptr) {
            if (nvalid >= 32 * (h + 1) && (reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(src + j);
                    b[j] = f.x, b[j + 1] = f.y, b[j + 2] = f.z, b[j + 3] = f.w;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (32 * h + j < nvalid) b[j] = src[j];
            }
        }
        const uint32_t row = buf + (uint32_t)lane * 128u, sw = (uint32_t)(lane & 7);
        constexpr int PER = OUT == OUT_F32 ? 4 : 8;           // values per 16 bytes
#pragma unroll
        for (int c = 0; c < 32 / PER; ++c) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (OUT == OUT_F32) {
                    const int j = 4 * c + e;
                    w[e] = __float_as_uint(act_mx<ACT>(__uint_as_float(r[h][j]) + b[j], alpha));
                } else {
                    const int j = 8 * c + 2 * e;
                    w[e] = pack2<OUT>(act_mx<ACT>(__uint_as_float(r[h][j]) + b[j], alpha),
                                      act_mx<ACT>(__uint_as_float(r[h][j + 1]) + b[j + 1], alpha));
                }
            }
            ptx::st_shared_v4(row + (((uint32_t)(c + h * (32 / PER)) ^ sw) << 4), w[0], w[1], w[2], w[3]);
        }
    }
}

template <int OUT, typename Loaded>
__device__ __forceinline__ void mx_epi_unit(int act, uint32_t taddr, const float *bias, int nvalid, float alpha,
                                            uint32_t buf, int lane,
                                            Loaded loaded)
{
    switch (act) {
    case ACT_RELU: mx_epi_unit<OUT, ACT_RELU>(taddr, bias, nvalid, alpha, buf, lane, loaded); break;
    case ACT_LEAKY: mx_epi_unit<OUT, ACT_LEAKY>(taddr, bias, nvalid, alpha, buf, lane, loaded); break;
    case ACT_TANH: mx_epi_unit<OUT, ACT_TANH>(taddr, bias, nvalid, alpha, buf, lane, loaded); break;
    case ACT_SIGMOID: mx_epi_unit<OUT, ACT_SIGMOID>(taddr, bias, nvalid, alpha, buf, lane, loaded); break;
    case ACT_GELU: mx_epi_unit<OUT, ACT_GELU>(taddr, bias, nvalid, alpha, buf, lane, loaded); break;
    case ACT_SILU: mx_epi_unit<OUT, ACT_SILU>(taddr, bias, nvalid, alpha, buf, lane, loaded); break;
    default: mx_epi_unit<OUT, ACT_NONE>(taddr, bias, nvalid, alpha, buf, lane, loaded); break;
    }
}

// Element stores of a staged unit (32 rows of 128 bytes in the swizzled order)
// for outputs whose row pitch TMA cannot address.
template <int OUT>
__device__ __forceinline__ void mx_store_elements(void *C, uint32_t buf, int row0, int col0, int M, int N, int lane)
{
    constexpr int ESZ = OUT == OUT_F32 ? 4 : 2, COLS = 128 / ESZ;
    for (int r = 0; r < 32 && row0 + r < M; ++r)
#pragma unroll
        for (int c = lane; c < COLS; c += 32) {
            if (col0 + c >= N) continue;
            const uint32_t b = (uint32_t)c * ESZ;
            const uint32_t at = buf + r * 128u + (((b >> 4) ^ (r & 7)) << 4) + (b & 15u);
            const int64_t i = (int64_t)(row0 + r) * N + col0 + c;
            if constexpr (OUT == OUT_F32) {
                uint32_t v;
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
                static_cast<uint32_t *>(C)[i] = v;
            } else {
                uint16_t v;
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
                static_cast<uint16_t *>(C)[i] = v;
            }
        }
}

template <int OUT>
__global__ void __launch_bounds__(MxPairCfg::THREADS, 1)
    gemm_mxfp4_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                           const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                           const __grid_constant__ CUtensorMap tmC, const MxGemmArgs p)
{
    using Cfg = MxPairCfg;
    constexpr int STAGES = Cfg::STAGES;
    constexpr int COLS = OUT == OUT_F32 ? 32 : 64;
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
            ptx::prefetch_tensormap(&tmA);
            ptx::prefetch_tensormap(&tmB);
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
            for (int t = pair; t < p.num_tiles && ok; t += npairs) {
                int mb, nb;
                mx_tile(t, p, mb, nb);
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!pipe_wait(pp, pp.empty0 + 8 * stage, phase ^ 1u)) { ok = false; break; }
                    const uint32_t fb = pp.full0 + 8 * stage;
                    if (leader) ptx::mbar_arrive_expect_tx(fb, 2u * Cfg::STAGE_BYTES);
                    const uint32_t to = ptx::mapa(fb, 0);
                    ptx::tma_load_2d_pair(sA + stage * Cfg::A_BYTES, &tmA, to, kb * 64, mb * 256 + (int)rank * 128);
                    ptx::tma_load_2d_pair(sB + stage * Cfg::B_BYTES, &tmB, to, kb * 64, nb * 256 + (int)rank * 128);
                    ptx::tma_load_2d_pair(sS + stage * Cfg::S_BYTES, &tmSA, to, kb * 256, mb * 2 + (int)rank);
                    ptx::tma_load_2d_pair(sS + stage * Cfg::S_BYTES + 1024u, &tmSB, to, kb * 256, nb * 2);
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            if (!ok) pipe_fail(pp);
        }
    } else if (usable && warp == 1) {
        if (leader) {                                         // the whole warp: see mma_mxf4
            const uint32_t id0 = ptx::idesc_mxf4(256, 256, 0, 0), id2 = ptx::idesc_mxf4(256, 256, 2, 2);
            uint32_t stage = 0, phase = 0, tile = 0;
            bool ok = true;
            for (int t = pair; t < p.num_tiles && ok; t += npairs, ++tile) {
                // the shared columns of the previous tile's accumulator are read, and all of the one before it
                if (tile != 0 && !mx_warp_wait(pp, pp.tempty0, (tile - 1) & 1u)) { ok = false; break; }
                ptx::tc_fence_after();
                const uint32_t d = pp.tmem + (tile & 1u) * Cfg::ACC_STRIDE;
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!mx_warp_wait(pp, pp.full0 + 8 * stage, phase)) { ok = false; break; }
                    ptx::tc_fence_after();
                    const uint32_t a0 = sA + stage * Cfg::A_BYTES, b0 = sB + stage * Cfg::B_BYTES;
                    const uint32_t s0 = sS + stage * Cfg::S_BYTES;
                    const uint32_t ts = pp.tmem + Cfg::SCALE_COL + stage * Cfg::SLOT_COLS;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {                 // B: two times eight columns, then A: two times four
                        ptx::tmem_cp_scales_pair(ts + 8 * j, ptx::smem_desc(s0 + 1024u + 512u * j, 16u, 128u, ptx::SWIZZLE_NONE));
                        ptx::tmem_cp_scales_pair(ts + 8 * j + 4,
                                                 ptx::smem_desc(s0 + 2048u + 512u * j, 16u, 128u, ptx::SWIZZLE_NONE));
                        ptx::tmem_cp_scales_pair(ts + 16 + 4 * j, ptx::smem_desc(s0 + 512u * j, 16u, 128u, ptx::SWIZZLE_NONE));
                    }
                    const int n = min(4, p.nk64 - 4 * kb);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < n)
                            ptx::mma_mxf4_pair(d, ptx::smem_desc(a0 + 32u * k, 16u, 1024u, ptx::SWIZZLE_128B),
                                               ptx::smem_desc(b0 + 32u * k, 16u, 1024u, ptx::SWIZZLE_128B),
                                               k & 1 ? id2 : id0, ts + 16 + 4 * (k >> 1), ts + 8 * (k >> 1),
                                               (kb | k) != 0 ? 1u : 0u);
                    ptx::commit_elected_pair(pp.empty0 + 8 * stage, 3);
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                ptx::commit_elected_pair(pp.tfull0 + 8 * (tile & 1u), 3);
            }
            if (!ok && lane == 0) pipe_fail(pp);
            ptx::commit_elected_pair(pp.drain, 1);
            ptx::mbar_wait_bounded(pp.drain, 0, DRAIN_NS, nullptr);
        }
    } else if (usable) {
        const int q = warp & 3, part = (warp - 2) >> 2;
        const uint32_t buf = base + Cfg::OFF_EPI + (uint32_t)(warp - 2) * 4096u;
        const uint32_t tempty_leader = ptx::mapa(pp.tempty0, 0);
        const uint64_t pol_c = ptx::createpolicy_evict_first();   // C is not read back here
        constexpr int NU = 256 / COLS, SHARED = 128 / COLS;       // units of a tile; of its shared columns
        uint32_t tile = 0;
        for (int t = pair; t < p.num_tiles; t += npairs, ++tile) {
            int mb, nb;
            mx_tile(t, p, mb, nb);
            if (!warp_epi_wait(pp, pp.tfull0 + 8 * (tile & 1u), (tile >> 1) & 1u)) { pipe_fail(pp); break; }
            ptx::tc_fence_after();
            const uint32_t tbase = pp.tmem + ((uint32_t)(q * 32) << 16) + (tile & 1u) * Cfg::ACC_STRIDE;
            const int row0 = mb * 256 + (int)rank * 128 + q * 32;
            // the shared columns are the last of the lower accumulator and the first of the upper one
            const int first = (tile & 1u) == 0 ? NU - SHARED : 0;
#pragma unroll 1
            for (int i = part; i < NU; i += 2) {
                const int u = (first + i) & (NU - 1);
                const int col0 = nb * 256 + u * COLS;
                if (lane == 0) ptx::bulk_wait_read<0>();
                __syncwarp();
                mx_epi_unit<OUT>(p.act, tbase + u * COLS, p.bias != nullptr ? p.bias + col0 : nullptr, p.N - col0,
                                 p.alpha, buf, lane, [&] {
                                     // this warp's last unit of the shared columns
                                     if (i < SHARED - 2 || i >= SHARED) return;
                                     ptx::tc_fence_before();
                                     __syncwarp();
                                     if (lane == 0) {
                                         if (leader) ptx::mbar_arrive(pp.tempty0);
                                         else ptx::mbar_arrive_cluster(tempty_leader);
                                     }
                                 });
                if (p.c_tma) {
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && row0 < p.M && col0 < p.N) {
                        ptx::tma_store_2d_hint(&tmC, buf, col0, row0, pol_c);
                        ptx::bulk_commit();
                    }
                } else {
                    __syncwarp();
                    mx_store_elements<OUT>(p.C, buf, row0, col0, p.M, p.N, lane);
                    __syncwarp();
                }
            }
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
    cfg.blockDim = dim3(MxPairCfg::THREADS);
    cfg.dynamicSmemBytes = MxPairCfg::SMEM_BYTES;
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

template <int OUT>
static cudaError_t launch_mx_pair_t(const MxGemmLaunch &L, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    pair_config(cfg, attr, L.grid, stream);
    return cudaLaunchKernelEx(&cfg, gemm_mxfp4_pair_kernel<OUT>, L.tmA, L.tmB, L.tmSA, L.tmSB, L.tmC, L.args);
}

cudaError_t setup_mxfp4_pair_kernels(int *max_pairs)
{
    const auto attr_of = cudaFuncAttributeMaxDynamicSharedMemorySize;
    cudaError_t e = cudaFuncSetAttribute(gemm_mxfp4_pair_kernel<OUT_BF16>, attr_of, MxPairCfg::SMEM_BYTES);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(gemm_mxfp4_pair_kernel<OUT_F16>, attr_of, MxPairCfg::SMEM_BYTES);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(gemm_mxfp4_pair_kernel<OUT_F32>, attr_of, MxPairCfg::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    pair_config(cfg, attr, 2 * 128, nullptr);
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(max_pairs, gemm_mxfp4_pair_kernel<OUT_BF16>, &cfg);
}

cudaError_t launch_gemm_mxfp4_pair(const MxGemmLaunch &L, cudaStream_t stream)
{
    if (L.out == OUT_BF16) return launch_mx_pair_t<OUT_BF16>(L, stream);
    if (L.out == OUT_F16) return launch_mx_pair_t<OUT_F16>(L, stream);
    return launch_mx_pair_t<OUT_F32>(L, stream);
}

}  // namespace mmact
