// gemm_mxfp4_rows.cu -- C = act(A x B^T + bias) of MXFP4 matrices when the output
// has few rows or few tiles: the weights B are the work, and every SM has to be
// reading them.
//
// The operands change sides: an output tile is 128 rows of B (the MMA's 128
// accumulator lanes) by BT rows of A (16 to 128, its columns), so that a product
// with one row of A loads 128-row boxes of weights and 2 KB of everything else.
// The K loop of a tile is shared by a cluster of S CTAs, each over a consecutive
// range of K; their fp32 partial tiles meet in shared memory, each CTA adding up
// a slice of BT / S columns over the cluster in rank order (so results repeat),
// then bias, activation and the stores: consecutive lanes hold consecutive
// columns of C.
//
// The scales of A's rows are read from the first column of a scale tile on: a
// tile narrower than 128 rows is always the only one, because the MMA takes no
// scale address that is not a multiple of four columns.
//
//   warp 0      TMA producer: a ring of stages of 256 K (codes with the 128-byte
//               swizzle, scale tiles).  While the kernel before this one in the
//               stream still runs (it may be writing A's codes) the CTA already
//               asks for its first 16 weight boxes in L2.
//   warp 1      TMEM allocation, scale copies into columns of the ring stage, MMAs
//   warps 2..5  partial tile, reduction, epilogue
//   warps 6..9  when A arrives as x in 16 or 32 bits, up to 8 rows: they quantise
//               its stages into the ring, where the codes would have been copied,
//               which saves a kernel of its own (1 row, 8192 x 8192 weights: 8.9
//               against 10.9 us with one; 8 rows 10.1 and 11.3, 16 rows 14.5 and 11.3)
//
// Measured with calls back to back: 1 x 8192 x 8192 (35.7 MB) 8.4 us, 128 x 8192 x 8192 13.0 us
// (every SM reads the token tiles from L2, 117 MB in all), 77 x 4001 x 2056 7.7 us.  About
// 5.4 us of each are fixed: start, first loads, the cluster's sum, stores.
#include <type_traits>

#include "common.cuh"
#include "kernels_mx.h"
#include "mx_layout.h"
#include "mxfp4.cuh"

namespace mmact {

// C[m0 + j][n] = act(z[j] + bias) for this lane's n and the rows that exist:
// element stores, a warp covering 32 consecutive n.
template <int OUT, int CH>
__device__ __forceinline__ void rows_store(const MxRowsArgs &p, int m0, int n, float (&z)[CH], float bias)
{
#pragma unroll
    for (int j = 0; j < CH; ++j) z[j] += bias;
    act_mx_all(p.act, z, p.alpha);
    if (n >= p.N) return;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        if (m0 + j >= p.M) break;
        const int64_t at = (int64_t)(m0 + j) * p.N + n;
        if constexpr (OUT == OUT_F32) static_cast<float *>(p.C)[at] = z[j];
        else if constexpr (OUT == OUT_BF16) static_cast<__nv_bfloat16 *>(p.C)[at] = __float2bfloat16_rn(z[j]);
        else static_cast<__half *>(p.C)[at] = __float2half_rn(z[j]);
    }
}

// Sum of CH columns of the cluster's partial tiles at this thread's lane, in rank
// order: all loads of a rank in flight together.
template <int CH>
__device__ __forceinline__ void cluster_columns(uint32_t at, int split, float (&z)[CH])
{
#pragma unroll
    for (int j = 0; j < CH; ++j) z[j] = 0.0f;
#pragma unroll 2
    for (int s = 0; s < split; ++s) {
        const uint32_t from = ptx::mapa(at, (uint32_t)s);
        float v[CH];
#pragma unroll
        for (int j = 0; j < CH; ++j) v[j] = ptx::ld_cluster_f32(from + j * 512u);
#pragma unroll
        for (int j = 0; j < CH; ++j) z[j] += v[j];
    }
}

// The rows of x as codes and scales in every stage of the ring (what stands in
// place of rows that do not exist only reaches columns that are not stored).  A
// stage to a warp, so that four stages' loads are in flight; a block of 32 values
// to a lane, two at a time.
template <int XT, int BT>
__device__ __forceinline__ void quantize_stages(const MxRowsArgs &p, const Pipe &pp, uint32_t sT, uint32_t sS, int kb0, int kb1)
{
    using Cfg = MxRowsCfg<BT>;
    const int w = (int)(threadIdx.x >> 5) - 6, lane = threadIdx.x & 31, blk = lane & 7;
    const bool vec = (int64_t)p.K * (XT == IN_F32 ? 4 : 2) % 16 == 0;
    for (int kb = kb0 + w, i = w; kb < kb1; kb += 4, i += 4) {
        const uint32_t stage = (uint32_t)(i % p.stages), phase = (uint32_t)(i / p.stages) & 1u;
        const int k0 = kb * 256 + blk * 32, n = min(32, p.K - k0);
#pragma unroll 1
        for (int r0 = 0; r0 < p.M; r0 += 8) {
            Raw8<XT> r[2][4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int row = r0 + 4 * u + (lane >> 3);
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int j = 0; j < Raw8<XT>::WORDS; ++j) r[u][q].w[j] = 0;
                if (row < p.M && n > 0) {
                    const int64_t at = (int64_t)row * p.K + k0;
                    if (vec)
#pragma unroll
                        for (int q = 0; q < 4; ++q) load8<XT, true>(p.x, at + 8 * q, n - 8 * q, r[u][q]);
                    else load32_any<XT>(p.x, at, n, (int64_t)p.M * p.K, r[u]);
                }
            }
            // A slot goes to another warp in its next use.  This warp saw the slot of four stages ago free, so that with
            // four stages or more all but the last use of this one are over, and the parity names that use.
            static_assert(Cfg::MAX_STAGES >= 4, "a ring of fewer stages than MAX_STAGES never wraps");
            if (r0 == 0 && !mx_warp_wait(pp, pp.empty0 + 8 * stage, phase ^ 1u)) {
                if (lane == 0) pipe_fail(pp);
                return;
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint32_t row = (uint32_t)(r0 + 4 * u + (lane >> 3));
                if (row >= (uint32_t)p.M) continue;
                uint32_t amax = 0, c[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int j = 0; j < Raw8<XT>::WORDS; ++j) amax = raw_max<XT>(amax, r[u][q].w[j]);
                if constexpr (XT != IN_F32) amax = bits_of<XT>(max(amax & 0xffffu, amax >> 16));
                const uint32_t b = mx_scale_byte(amax);
                const float inv = mx_inv_scale(b == 255u ? 0u : b);
#pragma unroll
                for (int q = 0; q < 4; ++q) c[q] = b == 255u ? 0u : raw_encode<XT>(r[u][q].w, inv);
                ptx::st_shared_v4(sT + stage * Cfg::T_BYTES + row * 128u + (((uint32_t)blk ^ (row & 7u)) << 4), c[0], c[1], c[2],
                                  c[3]);
                // at most 32 rows: the first of a scale tile's four groups
                const uint32_t at = sS + stage * Cfg::S_BYTES + 1024u + (uint32_t)(blk >> 2) * 512u + row * 16u + (uint32_t)(blk & 3);
                asm volatile("st.shared.u8 [%0], %1;" ::"r"(at), "r"(b) : "memory");
            }
            __syncwarp();
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(pp.full0 + 8 * stage);
    }
}

constexpr int XT_NONE = -1;          // A comes as codes and scales

template <int XT>
constexpr int ROWS_THREADS = XT == XT_NONE ? 192 : 320;

template <int OUT, int BT, int XT>
__global__ void __launch_bounds__(ROWS_THREADS<XT>, 1)
    gemm_mxfp4_rows_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmT,
                           const __grid_constant__ CUtensorMap tmSW, const __grid_constant__ CUtensorMap tmST,
                           const MxRowsArgs p)
{
    using Cfg = MxRowsCfg<BT>;
    const int stages = p.stages;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t base = ptx::smem_addr(smem);
    const int rank = p.split > 1 ? (int)ptx::cluster_ctarank() : 0;
    const int tile = blockIdx.x / p.split;
    const int nb = tile % p.tiles_n, tb = tile / p.tiles_n;
    const int kb0 = rank * p.kb_per, kb1 = min(p.num_kb, kb0 + p.kb_per);

    const bool aligned = (base & 1023u) == 0;
    if (!aligned && threadIdx.x == 0) atomicOr(p.status, ST_SMEM_ALIGN);
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + Cfg::OFF_MISC);
    Pipe pp;
    pp.full0 = base + Cfg::OFF_BAR;
    pp.empty0 = pp.full0 + 8 * Cfg::MAX_STAGES;
    pp.tfull0 = pp.empty0 + 8 * Cfg::MAX_STAGES;
    pp.drain = pp.tfull0 + 8;
    pp.tempty0 = 0;
    pp.abort = misc + 1;
    pp.status = p.status;
    pp.wait_ns = p.wait_ns;
    if (aligned) {
        if (threadIdx.x == 0) {
            ptx::prefetch_tensormap(&tmW);
            if constexpr (XT == XT_NONE) ptx::prefetch_tensormap(&tmT);
            for (int s = 0; s < stages; ++s) {
                ptx::mbar_init(pp.full0 + 8 * s, XT == XT_NONE ? 1 : 2);   // + a quantising warp
                ptx::mbar_init(pp.empty0 + 8 * s, 1);
            }
            ptx::mbar_init(pp.tfull0, 1);
            ptx::mbar_init(pp.drain, 1);
            misc[1] = 0;
            ptx::fence_mbar_init();
            for (int kb = kb0; kb < min(kb1, kb0 + 16); ++kb) {
                ptx::tma_prefetch_2d(&tmW, kb * 64, nb * 128);
                ptx::tma_prefetch_2d(&tmSW, kb * 256, nb);
            }
        }
    }
    ptx::cta_sync();
    ptx::griddep_wait();
    // Tensor memory is taken when the kernels before this one are done, and the next
    // one may start when every CTA of this one has it: a CTA that holds tensor memory
    // never waits for one of its stream that still needs it.  Nor for one of another
    // stream: CTAs that share an SM all find their columns (see MxRowsCfg).
    if (warp >= 1 && warp < 6) {
        if (warp == 1 && aligned) {
            ptx::tmem_alloc(base + Cfg::OFF_MISC, Cfg::TMEM_COLS);
            ptx::tmem_relinquish();
        }
        __syncwarp();
        ptx::tc_fence_before();
        asm volatile("barrier.sync 2, 160;" ::: "memory");
        ptx::tc_fence_after();
        pp.tmem = misc[0];
    }
    ptx::griddep_launch_dependents();

    const uint32_t sW = base + Cfg::OFF_RING, sT = sW + stages * Cfg::W_BYTES, sS = sT + stages * Cfg::T_BYTES;
    if (aligned && warp == 0) {
        if (lane == 0) {
            bool ok = true;
            int issued = 0;
            uint32_t stage = 0, phase = 0;
            for (int kb = kb0; kb < kb1; ++kb, ++issued) {
                if (!pipe_wait(pp, pp.empty0 + 8 * stage, phase ^ 1u)) { ok = false; break; }
                const uint32_t fb = pp.full0 + 8 * stage;
                ptx::mbar_arrive_expect_tx(fb, (uint32_t)(XT == XT_NONE ? Cfg::STAGE_BYTES : Cfg::W_BYTES + 1024));
                ptx::tma_load_2d(sW + stage * Cfg::W_BYTES, &tmW, fb, kb * 64, nb * 128);
                ptx::tma_load_2d(sS + stage * Cfg::S_BYTES, &tmSW, fb, kb * 256, nb);
                if constexpr (XT == XT_NONE) {
                    ptx::tma_load_2d(sT + stage * Cfg::T_BYTES, &tmT, fb, kb * 64, tb * BT);
                    ptx::tma_load_2d(sS + stage * Cfg::S_BYTES + 1024u, &tmST, fb, kb * 256, tb);
                }
                if (++stage == (uint32_t)stages) { stage = 0; phase ^= 1u; }
            }
            if (!ok) pipe_fail(pp);
            // every copy has landed before the ring's memory is used again or the CTA exits
            for (int u = max(0, issued - stages); u < issued; ++u)
                ptx::mbar_wait_bounded(pp.full0 + 8 * (u % stages), (u / stages) & 1, DRAIN_NS, nullptr);
        }
    } else if (aligned && warp == 1) {
        {                                                     // the whole warp: see mma_mxf4
            const uint32_t id0 = ptx::idesc_mxf4(128, BT, 0, 0), id2 = ptx::idesc_mxf4(128, BT, 2, 2);
            const uint64_t w0 = ptx::smem_desc(sW, 16u, 1024u, ptx::SWIZZLE_128B), t0 = ptx::smem_desc(sT, 16u, 1024u, ptx::SWIZZLE_128B);
            const uint64_t s0 = ptx::smem_desc(sS, 16u, 128u, ptx::SWIZZLE_NONE);
            bool ok = true;
            uint32_t stage = 0, phase = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!mx_warp_wait(pp, pp.full0 + 8 * stage, phase)) { ok = false; break; }
                ptx::tc_fence_after();
                ptx::mma_mxf4_stage(pp.tmem, w0 + stage * (Cfg::W_BYTES >> 4), t0 + stage * (Cfg::T_BYTES >> 4),
                                    s0 + stage * (Cfg::S_BYTES >> 4), pp.tmem + Cfg::SCALE_COL + stage * 16u, id0, id2,
                                    min(4, p.nk64 - 4 * kb), kb > kb0 ? 1u : 0u);
                ptx::commit_elected(pp.empty0 + 8 * stage);
                if (++stage == (uint32_t)stages) { stage = 0; phase ^= 1u; }
            }
            if (ok) ptx::commit_elected(pp.tfull0);
            else if (lane == 0) pipe_fail(pp);
            ptx::commit_elected(pp.drain);
            ptx::mbar_wait_bounded(pp.drain, 0, DRAIN_NS, nullptr);
        }
    }
    if constexpr (XT != XT_NONE) {
        if (aligned && warp >= 6) quantize_stages<XT, BT>(p, pp, sT, sS, kb0, kb1);
    }
    __syncwarp();
    // The epilogue warps take part in cluster barriers with the others below, so
    // the partial tile is read out in one place for every warp's control flow.
    const int q = warp & 3, n = nb * 128 + q * 32 + lane;
    const bool epi = warp >= 2 && warp < 6;
    const float bias = epi && p.bias != nullptr && n < p.N ? p.bias[n] : 0.0f;
    bool good = aligned;
    if (epi && aligned) {
        if (!warp_epi_wait(pp, pp.tfull0, 0)) {
            pipe_fail(pp);
            good = false;
        }
        ptx::tc_fence_after();
    }
    const uint32_t taddr = pp.tmem + ((uint32_t)(q * 32) << 16);
    if (p.split == 1) {
        if (epi && good) {
#pragma unroll 1
            for (int c = 0; c < BT; c += 16) {
                if (tb * BT + c >= p.M) break;
                uint32_t r[16];
                float z[16];
                ptx::tmem_ld16(taddr + c, r);
#pragma unroll
                for (int j = 0; j < 16; ++j) z[j] = __uint_as_float(r[j]);
                rows_store<OUT>(p, tb * BT + c, n, z, bias);
                __syncwarp();
            }
        }
    } else {
        // partial tile [column][lane] over the ring, whose copies and MMAs are done
        float *part = reinterpret_cast<float *>(smem + Cfg::OFF_RING);
        if (epi && good) {
#pragma unroll 1
            for (int c = 0; c < BT; c += 16) {
                uint32_t r[16];
                ptx::tmem_ld16(taddr + c, r);
#pragma unroll
                for (int j = 0; j < 16; ++j) part[(c + j) * 128 + q * 32 + lane] = __uint_as_float(r[j]);
            }
        }
        ptx::cluster_sync();
        if (epi && good) {
            // this CTA's slice of the columns that exist: 16 at a time, or the 2 to 8 it has
            const int rows = min(BT, p.M - tb * BT), even = ((rows + p.split - 1) / p.split + 15) & ~15;
            const int cols = min(BT / p.split, even), c0 = rank * cols;
            const uint32_t at = base + Cfg::OFF_RING + (uint32_t)(c0 * 128 + q * 32 + lane) * 4u;
            auto slice = [&](auto ch) {
                constexpr int CH = decltype(ch)::value;
                for (int c = 0; c < cols && tb * BT + c0 + c < p.M; c += CH) {
                    float z[CH];
                    cluster_columns<CH>(at + c * 512u, p.split, z);
                    rows_store<OUT>(p, tb * BT + c0 + c, n, z, bias);
                }
            };
            if (cols >= 16) slice(std::integral_constant<int, 16>());
            else if (cols == 8) slice(std::integral_constant<int, 8>());
            else if (cols == 4) slice(std::integral_constant<int, 4>());
            else slice(std::integral_constant<int, 2>());
        }
        ptx::cluster_sync();                                  // no CTA exits while its partial tile is read
    }
    ptx::tc_fence_before();
    ptx::cta_sync();
    __syncwarp();
    if (aligned && warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(pp.tmem, Cfg::TMEM_COLS);
    }
}

template <int OUT, int BT, int XT>
static cudaError_t launch_rows_t(const MxRowsLaunch &L, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)L.grid);
    cfg.blockDim = dim3(ROWS_THREADS<XT>);
    cfg.dynamicSmemBytes = (size_t)MxRowsCfg<BT>::smem_bytes(L.args.stages, L.args.split);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)L.args.split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = L.args.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, gemm_mxfp4_rows_kernel<OUT, BT, XT>, L.tmW, L.tmT, L.tmSW, L.tmST, L.args);
}

template <int OUT, int BT>
static cudaError_t launch_rows_x(const MxRowsLaunch &L, cudaStream_t stream)
{
    if (L.x_type == IN_BF16) return launch_rows_t<OUT, BT, IN_BF16>(L, stream);
    if (L.x_type == IN_F16) return launch_rows_t<OUT, BT, IN_F16>(L, stream);
    if (L.x_type == IN_F32) return launch_rows_t<OUT, BT, IN_F32>(L, stream);
    return launch_rows_t<OUT, BT, XT_NONE>(L, stream);
}

template <int OUT>
static cudaError_t launch_rows_o(const MxRowsLaunch &L, cudaStream_t stream)
{
    switch (L.bt) {
    case 16: return launch_rows_x<OUT, 16>(L, stream);
    case 32: return launch_rows_t<OUT, 32, XT_NONE>(L, stream);
    case 64: return launch_rows_t<OUT, 64, XT_NONE>(L, stream);
    default: return launch_rows_t<OUT, 128, XT_NONE>(L, stream);
    }
}

template <int OUT, int BT, int XT>
static cudaError_t setup_rows_t()
{
    return cudaFuncSetAttribute(gemm_mxfp4_rows_kernel<OUT, BT, XT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                MxRowsCfg<BT>::OFF_RING + MxRowsCfg<BT>::MAX_STAGES * MxRowsCfg<BT>::STAGE_BYTES);
}

template <int OUT, int BT>
static cudaError_t setup_rows_x()
{
    cudaError_t e = setup_rows_t<OUT, BT, XT_NONE>();
    if (e == cudaSuccess) e = setup_rows_t<OUT, BT, IN_BF16>();
    if (e == cudaSuccess) e = setup_rows_t<OUT, BT, IN_F16>();
    if (e == cudaSuccess) e = setup_rows_t<OUT, BT, IN_F32>();
    return e;
}

template <int OUT>
static cudaError_t setup_rows_o()
{
    cudaError_t e = setup_rows_x<OUT, 16>();
    if (e == cudaSuccess) e = setup_rows_t<OUT, 32, XT_NONE>();
    if (e == cudaSuccess) e = setup_rows_t<OUT, 64, XT_NONE>();
    if (e == cudaSuccess) e = setup_rows_t<OUT, 128, XT_NONE>();
    return e;
}

// Clusters of `split` CTAs that are resident at once (with a full ring).
template <int BT>
static cudaError_t rows_clusters(int split, int *n)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(split * 64));
    cfg.blockDim = dim3(192);
    cfg.dynamicSmemBytes = MxRowsCfg<BT>::OFF_RING + MxRowsCfg<BT>::MAX_STAGES * MxRowsCfg<BT>::STAGE_BYTES;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(n, gemm_mxfp4_rows_kernel<OUT_BF16, BT, XT_NONE>, &cfg);
}

cudaError_t setup_mxfp4_rows_kernels(int (&max_clusters)[4])
{
    cudaError_t e = setup_rows_o<OUT_BF16>();
    if (e == cudaSuccess) e = setup_rows_o<OUT_F16>();
    if (e == cudaSuccess) e = setup_rows_o<OUT_F32>();
    max_clusters[0] = 1 << 30;
    for (int i = 1; i < 4 && e == cudaSuccess; ++i) e = rows_clusters<128>(1 << i, &max_clusters[i]);
    return e;
}

cudaError_t launch_gemm_mxfp4_rows(const MxRowsLaunch &L, cudaStream_t stream)
{
    if (L.out == OUT_BF16) return launch_rows_o<OUT_BF16>(L, stream);
    if (L.out == OUT_F16) return launch_rows_o<OUT_F16>(L, stream);
    return launch_rows_o<OUT_F32>(L, stream);
}

}  // namespace mmact
