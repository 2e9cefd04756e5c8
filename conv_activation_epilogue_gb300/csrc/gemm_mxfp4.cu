// gemm_mxfp4.cu -- C = act(A x B^T + bias) of two matrices in the 4-bit
// microscaled format (mxfp4.cuh): A [M, K], B [N, K], tcgen05.mma.kind::mxf4.
//
// Persistent kernel, one CTA per SM, 128 x 128 output tiles.  A ring stage is
// 256 K: the codes of 128 rows of A and of B (128-byte rows, TMA with the
// 128-byte swizzle) and their scale tiles (two tiles of 512 bytes each, TMA).
// The MMA issuer copies the scale tiles to tensor memory (tcgen05.cp) into
// columns that belong to the ring stage, so that a copy never overtakes an
// MMA that still reads the columns: the stage itself is only refilled when
// that MMA has finished.
//
//   warp 0      TMA producer
//   warp 1      TMEM allocation, scale copies and MMAs
//   warps 2..5  epilogue
#include "common.cuh"
#include "kernels_mx.h"
#include "mxfp4.cuh"

namespace mmact {

struct MxCfg {
    static constexpr int BM = 128, BN = 128, BK = 256;
    static constexpr int A_BYTES = BM * BK / 2, B_BYTES = BN * BK / 2;      // 16 KB each
    static constexpr int S_BYTES = 1024;                                    // scales of one operand and stage
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + 2 * S_BYTES;
    static constexpr int EPI_BYTES = 4 * 2 * 4096;
    static constexpr int STAGES = 5;
    static constexpr uint32_t ACC_STRIDE = BN, SCALE_COL = 2 * BN, TMEM_COLS = 512;
    static constexpr int OFF_A = 0;
    static constexpr int OFF_B = OFF_A + STAGES * A_BYTES;
    static constexpr int OFF_EPI = OFF_B + STAGES * B_BYTES;
    static constexpr int OFF_S = OFF_EPI + EPI_BYTES;
    static constexpr int OFF_BAR = OFF_S + STAGES * 2 * S_BYTES;
    static constexpr int OFF_MISC = OFF_BAR + (2 * STAGES + 5) * 8;
    static constexpr int SMEM_BYTES = OFF_MISC + 16;
    static_assert(SMEM_BYTES <= 232448, "shared memory budget");
    static_assert(SCALE_COL + STAGES * 16 <= TMEM_COLS, "tensor memory budget");
};

// Tile t -> (M block, N block), grouped M-first.
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
template <int OUT, int ACT>
__device__ __forceinline__ void mx_epi_unit(uint32_t taddr, const float *bias, int nvalid, float alpha, uint32_t buf,
                                            int lane)
{
    constexpr int HALVES = OUT == OUT_F32 ? 1 : 2;           // 32 columns at a time
    uint32_t r[HALVES][32];
#pragma unroll
    for (int h = 0; h < HALVES; ++h) ptx::tmem_ld32(taddr + 32 * h, r[h]);
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
        float b[32];
        const float *src = bias + 32 * h;
        if (bias != nullptr && nvalid >= 32 * (h + 1) && (reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const float4 f = __ldg(reinterpret_cast<const float4 *>(src + j));
                b[j] = f.x, b[j + 1] = f.y, b[j + 2] = f.z, b[j + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) b[j] = bias != nullptr && 32 * h + j < nvalid ? __ldg(src + j) : 0.0f;
        }
        __syncwarp();                                         // converged before the warp-collective wait
        ptx::tmem_ld_wait(r[h]);
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

template <int OUT>
__device__ __forceinline__ void mx_epi_unit(int act, uint32_t taddr, const float *bias, int nvalid, float alpha,
                                            uint32_t buf, int lane)
{
    switch (act) {
    case ACT_RELU: mx_epi_unit<OUT, ACT_RELU>(taddr, bias, nvalid, alpha, buf, lane); break;
    case ACT_LEAKY: mx_epi_unit<OUT, ACT_LEAKY>(taddr, bias, nvalid, alpha, buf, lane); break;
    case ACT_TANH: mx_epi_unit<OUT, ACT_TANH>(taddr, bias, nvalid, alpha, buf, lane); break;
    case ACT_SIGMOID: mx_epi_unit<OUT, ACT_SIGMOID>(taddr, bias, nvalid, alpha, buf, lane); break;
    case ACT_GELU: mx_epi_unit<OUT, ACT_GELU>(taddr, bias, nvalid, alpha, buf, lane); break;
    case ACT_SILU: mx_epi_unit<OUT, ACT_SILU>(taddr, bias, nvalid, alpha, buf, lane); break;
    default: mx_epi_unit<OUT, ACT_NONE>(taddr, bias, nvalid, alpha, buf, lane); break;
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
__global__ void __launch_bounds__(192, 1)
    gemm_mxfp4_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                      const __grid_constant__ CUtensorMap tmC, const MxGemmArgs p)
{
    using Cfg = MxCfg;
    constexpr int STAGES = Cfg::STAGES;
    constexpr int COLS = OUT == OUT_F32 ? 32 : 64;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = ptx::smem_addr(smem);

    ptx::griddep_launch_dependents();
    const bool aligned = (base & 1023u) == 0;
    if (!aligned && threadIdx.x == 0) atomicOr(p.status, ST_SMEM_ALIGN);

    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + Cfg::OFF_MISC);
    Pipe pp;
    pp.full0 = base + Cfg::OFF_BAR;
    pp.empty0 = pp.full0 + 8 * STAGES;
    pp.tfull0 = pp.empty0 + 8 * STAGES;
    pp.tempty0 = pp.tfull0 + 16;
    pp.drain = pp.tempty0 + 16;
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
            for (int a = 0; a < 2; ++a) {
                ptx::mbar_init(pp.tfull0 + 8 * a, 1);
                ptx::mbar_init(pp.tempty0 + 8 * a, 4);
            }
            ptx::mbar_init(pp.drain, 1);
            misc[1] = 0;
            ptx::fence_mbar_init();
        }
        if (warp == 1) {
            ptx::tmem_alloc(base + Cfg::OFF_MISC, Cfg::TMEM_COLS);
            ptx::tmem_relinquish();
        }
    }
    ptx::tc_fence_before();
    ptx::cta_sync();
    ptx::tc_fence_after();
    pp.tmem = misc[0];
    ptx::griddep_wait();

    const uint32_t sA = base + Cfg::OFF_A, sB = base + Cfg::OFF_B, sS = base + Cfg::OFF_S;
    if (aligned && warp == 0) {
        if (lane == 0) {
            uint32_t stage = 0, phase = 0, issued = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < p.num_tiles && ok; t += gridDim.x) {
                int mb, nb;
                mx_tile(t, p, mb, nb);
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!pipe_wait(pp, pp.empty0 + 8 * stage, phase ^ 1u)) { ok = false; break; }
                    const uint32_t fb = pp.full0 + 8 * stage;
                    ptx::mbar_arrive_expect_tx(fb, (uint32_t)Cfg::STAGE_BYTES);
                    ptx::tma_load_2d(sA + stage * Cfg::A_BYTES, &tmA, fb, kb * 64, mb * 128);
                    ptx::tma_load_2d(sB + stage * Cfg::B_BYTES, &tmB, fb, kb * 64, nb * 128);
                    ptx::tma_load_2d(sS + stage * 2048u, &tmSA, fb, kb * 256, mb);
                    ptx::tma_load_2d(sS + stage * 2048u + 1024u, &tmSB, fb, kb * 256, nb);
                    ++issued;
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            if (!ok) pipe_fail(pp);
            // Every copy has landed before the CTA exits (the MMA issuer may have given up
            // before it consumed them): the last STAGES uses, oldest first.
            const uint32_t n = issued < (uint32_t)STAGES ? issued : (uint32_t)STAGES;
            for (uint32_t u = issued - n; u < issued; ++u)
                ptx::mbar_wait_bounded(pp.full0 + 8 * (u % STAGES), (u / STAGES) & 1u, DRAIN_NS, nullptr);
        }
    } else if (aligned && warp == 1) {
        if (lane == 0) {
            const uint32_t id0 = ptx::idesc_mxf4(128, Cfg::BN, 0, 0), id2 = ptx::idesc_mxf4(128, Cfg::BN, 2, 2);
            uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < p.num_tiles && ok; t += gridDim.x) {
                if (!pipe_wait(pp, pp.tempty0 + 8 * acc, acc_phase ^ 1u)) { ok = false; break; }
                ptx::tc_fence_after();
                const uint32_t d = pp.tmem + acc * Cfg::ACC_STRIDE;
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!pipe_wait(pp, pp.full0 + 8 * stage, phase)) { ok = false; break; }
                    ptx::tc_fence_after();
                    const uint32_t a0 = sA + stage * Cfg::A_BYTES, b0 = sB + stage * Cfg::B_BYTES;
                    const uint32_t s0 = sS + stage * 2048u, ts = pp.tmem + Cfg::SCALE_COL + stage * 16u;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        ptx::tmem_cp_scales(ts + 4 * j, ptx::smem_desc(s0 + 512u * j, 16u, 128u, ptx::SWIZZLE_NONE));
                        ptx::tmem_cp_scales(ts + 8 + 4 * j,
                                            ptx::smem_desc(s0 + 1024u + 512u * j, 16u, 128u, ptx::SWIZZLE_NONE));
                    }
                    const int n = min(4, p.nk64 - 4 * kb);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < n)
                            ptx::mma_mxf4(d, ptx::smem_desc(a0 + 32u * k, 16u, 1024u, ptx::SWIZZLE_128B),
                                          ptx::smem_desc(b0 + 32u * k, 16u, 1024u, ptx::SWIZZLE_128B),
                                          k & 1 ? id2 : id0, ts + 4 * (k >> 1), ts + 8 + 4 * (k >> 1),
                                          (kb | k) != 0 ? 1u : 0u);
                    ptx::mma_commit(pp.empty0 + 8 * stage);
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                ptx::mma_commit(pp.tfull0 + 8 * acc);
                acc ^= 1u;
                if (acc == 0) acc_phase ^= 1u;
            }
            if (!ok) pipe_fail(pp);
            ptx::mma_commit(pp.drain);
            ptx::mbar_wait_bounded(pp.drain, 0, DRAIN_NS, nullptr);
        }
    } else if (aligned) {
        const int q = warp & 3;
        const uint32_t my_buf = base + Cfg::OFF_EPI + (uint32_t)q * 8192u;
        uint32_t acc = 0, acc_phase = 0, units = 0;
        for (int t = blockIdx.x; t < p.num_tiles; t += gridDim.x) {
            int mb, nb;
            mx_tile(t, p, mb, nb);
            if (!warp_epi_wait(pp, pp.tfull0 + 8 * acc, acc_phase)) { pipe_fail(pp); break; }
            ptx::tc_fence_after();
            const uint32_t tbase = pp.tmem + ((uint32_t)(q * 32) << 16) + acc * Cfg::ACC_STRIDE;
            const int row0 = mb * 128 + q * 32;
#pragma unroll 1
            for (int u = 0; u < Cfg::BN / COLS; ++u) {
                const uint32_t buf = my_buf + (units++ & 1u) * 4096u;
                const int col0 = nb * Cfg::BN + u * COLS;
                if (lane == 0) ptx::bulk_wait_read<1>();
                __syncwarp();
                mx_epi_unit<OUT>(p.act, tbase + u * COLS, p.bias != nullptr ? p.bias + col0 : nullptr, p.N - col0,
                                 p.alpha, buf, lane);
                if (p.c_tma) {
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && row0 < p.M && col0 < p.N) {
                        ptx::tma_store_2d(&tmC, buf, col0, row0);
                        ptx::bulk_commit();
                    }
                } else {
                    __syncwarp();
                    mx_store_elements<OUT>(p.C, buf, row0, col0, p.M, p.N, lane);
                    __syncwarp();
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(pp.tempty0 + 8 * acc);
            acc ^= 1u;
            if (acc == 0) acc_phase ^= 1u;
        }
        if (lane == 0) ptx::bulk_wait<0>();
        __syncwarp();
    }
    ptx::tc_fence_before();
    ptx::cta_sync();
    __syncwarp();
    if (aligned && warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(pp.tmem, Cfg::TMEM_COLS);
    }
}

template <int OUT>
static cudaError_t launch_mx_t(const MxGemmLaunch &L, cudaStream_t stream)
{
    return launch_k(gemm_mxfp4_kernel<OUT>, dim3((unsigned)L.grid), dim3(192), MxCfg::SMEM_BYTES, stream, L.tmA, L.tmB,
                    L.tmSA, L.tmSB, L.tmC, L.args);
}

cudaError_t setup_mxfp4_kernels()
{
    cudaError_t e = cudaFuncSetAttribute(gemm_mxfp4_kernel<OUT_BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         MxCfg::SMEM_BYTES);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(gemm_mxfp4_kernel<OUT_F16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 MxCfg::SMEM_BYTES);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(gemm_mxfp4_kernel<OUT_F32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 MxCfg::SMEM_BYTES);
    return e;
}

cudaError_t launch_gemm_mxfp4(const MxGemmLaunch &L, cudaStream_t stream)
{
    if (L.out == OUT_BF16) return launch_mx_t<OUT_BF16>(L, stream);
    if (L.out == OUT_F16) return launch_mx_t<OUT_F16>(L, stream);
    return launch_mx_t<OUT_F32>(L, stream);
}

}  // namespace mmact
