// gemm_fp8_rows.cu -- C = act(A x B^T + bias) of 8-bit matrices (fp8.cuh) when the output
// has few rows or few tiles: the weights B are the work, and every SM has to be
// reading them.
//
// The operands change sides: an output tile is 128 rows of B (the MMA's 128
// accumulator lanes) by BT rows of A (16 to 128, its columns), so that a product
// with one row of A loads 128-row boxes of weights and little else.  The K loop of a
// tile is shared by a cluster of S CTAs, each over a consecutive range of K; their
// fp32 partial tiles meet in shared memory, each CTA adding up a slice of BT / S
// columns over the cluster in rank order (so results repeat), then bias, activation
// and the stores: consecutive lanes hold consecutive columns of C.
//
// The scales of A's rows are read from the first column of a scale tile on: a
// tile narrower than 128 rows is always the only one, because the MMA takes no
// scale address that is not a multiple of four columns.
//
// Two products that do not depend on each other (a linear layer's two gradients) can share
// one launch.
//
// The tensor core cuts off additions to its accumulator (see gemm_fp8.cu): for fp32 outputs an
// accumulator takes 16 K blocks at most, and a CTA with more of them has three accumulators in turn, which
// the epilogue's warps add up, rounded, while the MMAs go on.  (128 x 8192 x 8192 from x in bf16, two chunks to a CTA,
// 23.4 us; 23.3 with all of K in one accumulator; 23.9 with one that the MMAs had to wait for and sums in 128
// registers a thread.  256 x 512 x 131072, eight chunks, 42.4 and 42.1, 42.5.)
//
//   warp 0      TMA producer: a ring of stages of 128 K (codes with the 128-byte
//               swizzle, scale tiles).  (Asking for the first weight boxes in L2 while
//               the kernel before this one still runs gained nothing: 32 x 4096 x 4096
//               8.2 us with it, 7.3 without.)
//   warp 1      TMEM allocation, scale copies into columns of the ring stage, MMAs
//   warps 2..5  partial tile, reduction, epilogue
//   warps 6..9  when A arrives as x in 16 or 32 bits, up to 8 rows: they quantise
//               its stages into the ring, where the codes would have been copied,
//               which saves a kernel of its own
//
// Bound by the weights' bytes and about 5 us of fixed parts (start, first loads, the
// cluster's sum, stores).  Measured with weights from HBM: 1 x 8192 x 8192 with x quantised inside
// 15.5 us, 16 rows 14.4 (67 MB: 4.7 TB/s), 128 rows 18; 32, 64, 128 x 4096 x 4096 7.3,
// 8.5, 9.9 us.
#include <type_traits>

#include "common.cuh"
#include "fp8.cuh"
#include "kernels_fp8.h"
#include "mx_layout.h"
#include "rows_epilogue.cuh"

namespace mmact {

// The rows of x (8 at most) as E4M3 codes and scales in every stage of the ring (what
// stands in place of rows that do not exist only reaches columns that are not stored).
// A stage to a warp, so that four stages' loads are in flight; 32 values to a lane, four
// lanes a row.
template <int XT, int BT>
__device__ __forceinline__ void quantize_f8_stages(const F8RowsProblem &p, const Pipe &pp, int stages, uint32_t sT, uint32_t sS, int kb0, int kb1)
{
    using Cfg = F8RowsCfg<BT>;
    const int w = (int)(threadIdx.x >> 5) - 6, lane = threadIdx.x & 31, row = lane >> 2, q0 = lane & 3;
    const bool vec = (int64_t)p.K * (XT == IN_F32 ? 4 : 2) % 16 == 0;
    for (int kb = kb0 + w, i = w; kb < kb1; kb += 4, i += 4) {
        const uint32_t stage = (uint32_t)(i % stages), phase = (uint32_t)(i / stages) & 1u;
        const int k0 = kb * 128 + q0 * 32, n = min(32, p.K - k0);
        Raw8<XT> r[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < Raw8<XT>::WORDS; ++j) r[q].w[j] = 0;
        if (row < p.M && n > 0) {
            const int64_t at = (int64_t)row * p.K + k0;
            if (vec)
#pragma unroll
                for (int q = 0; q < 4; ++q) load8<XT, true>(p.x, at + 8 * q, n - 8 * q, r[q]);
            else load32_any<XT>(p.x, at, n, (int64_t)p.M * p.K, r);
        }
        uint32_t amax = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < Raw8<XT>::WORDS; ++j) amax = raw_max<XT>(amax, r[q].w[j]);
        if constexpr (XT != IN_F32) amax = max(amax & 0xffffu, amax >> 16);
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        if constexpr (XT != IN_F32) amax = bits_of<XT>(amax);
        const uint32_t b = f8_scale_byte<F8_E4M3>(amax);
        const float inv = mx_inv_scale(b == 255u ? 0u : b);
        // A slot goes to another warp in its next use.  This warp saw the slot of four stages ago free, so that with
        // four stages or more all but the last use of this one are over, and the parity names that use.
        static_assert(Cfg::MAX_STAGES >= 4, "a ring of fewer stages than MAX_STAGES never wraps");
        if (!mx_warp_wait(pp, pp.empty0 + 8 * stage, phase ^ 1u)) {
            if (lane == 0) pipe_fail(pp);
            return;
        }
        if (row < p.M) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint2 u = f8_raw_encode<XT, F8_E4M3>(r[2 * h].w, inv), v = f8_raw_encode<XT, F8_E4M3>(r[2 * h + 1].w, inv);
                const bool bad = b == 255u;
                ptx::st_shared_v4(sT + stage * Cfg::T_BYTES + row * 128u + (((uint32_t)(2 * q0 + h) ^ (uint32_t)row) << 4),
                                  bad ? 0u : u.x, bad ? 0u : u.y, bad ? 0u : v.x, bad ? 0u : v.y);
            }
            // the first of a scale tile's four groups; the byte that the stage's instructions read
            if (q0 == 0) {
                const uint32_t at = sS + stage * Cfg::S_BYTES + 512u + (uint32_t)row * 16u + (uint32_t)(kb & 3);
                asm volatile("st.shared.u8 [%0], %1;" ::"r"(at), "r"(b) : "memory");
            }
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(pp.full0 + 8 * stage);
    }
}

// What the epilogue does with the chunks of a CTA's K blocks as they come: each takes over the sum of
// those before it, rounded, but the last, which is only waited for.  Chunk c is in accumulator c % 3.  The MMAs
// wait for chunk c to be taken over (`tempty0`) before they say that c + 1 is complete and begin c + 2: so neither
// side is ever two phases of a barrier ahead of the other, and chunk c's accumulator is read (with c + 1) before c + 3
// takes it.  False when a wait ran out.
template <int BT>
__device__ __forceinline__ bool rows_chunks(const Pipe &pp, uint32_t taddr, int chunks, int lane)
{
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
        if (!warp_epi_wait(pp, pp.tfull0 + 8 * (c & 1), (uint32_t)(c >> 1) & 1u)) return false;
        ptx::tc_fence_after();
        if (c == chunks - 1) break;
        const uint32_t sum = taddr + (uint32_t)((c + 2) % 3 * BT), here = taddr + (uint32_t)(c % 3 * BT);
#pragma unroll 1
        for (int i = 0; i < BT && c != 0; i += 16) {
            uint32_t a[16], b[16];
            ptx::tmem_ld16(sum + i, a);
            ptx::tmem_ld16(here + i, b);
#pragma unroll
            for (int j = 0; j < 16; ++j) b[j] = __float_as_uint(__uint_as_float(a[j]) + __uint_as_float(b[j]));
            ptx::tmem_st16(here + i, b);
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(pp.tempty0);
    }
    return true;
}

constexpr int X_CODES = -1;          // A comes as codes and scales

template <int XT>
constexpr int F8_ROWS_THREADS = XT == X_CODES ? 192 : 320;

// CHUNKS: some CTA sums its K blocks in several accumulators.
template <int BT, int XT, bool CHUNKS>
__global__ void __launch_bounds__(F8_ROWS_THREADS<XT>, 1) gemm_fp8_rows_kernel(const __grid_constant__ F8RowsArgs args)
{
    using Cfg = F8RowsCfg<BT, CHUNKS>;
    const int stages = args.stages, split = args.split;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t base = ptx::smem_addr(smem);
    const int rank = split > 1 ? (int)ptx::cluster_ctarank() : 0;
    int tile = blockIdx.x / split;
    const bool second = XT == X_CODES && tile >= args.prob[0].num_tiles;
    if (second) tile -= args.prob[0].num_tiles;
    const F8RowsProblem &p = args.prob[second ? 1 : 0];
    const F8RowsMaps &maps = args.maps[second ? 1 : 0];
    const uint32_t idesc = p.idesc;
    const int nk32 = p.nk32;
    const int nb = tile % p.tiles_n, tb = tile / p.tiles_n;
    const int kb0 = rank * p.kb_per, kb1 = min(p.num_kb, kb0 + p.kb_per), chunk_kb = p.chunk_kb;

    const bool aligned = (base & 1023u) == 0;
    if (!aligned && threadIdx.x == 0) atomicOr(args.status, ST_SMEM_ALIGN);
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + Cfg::OFF_MISC);
    Pipe pp;
    pp.full0 = base + Cfg::OFF_BAR;
    pp.empty0 = pp.full0 + 8 * Cfg::MAX_STAGES;
    pp.tfull0 = pp.empty0 + 8 * Cfg::MAX_STAGES;
    pp.drain = pp.tfull0 + 16;                // tfull0: two, of even and odd chunks
    pp.tempty0 = pp.drain + 8;                // a chunk has taken over the sum so far
    pp.abort = misc + 1;
    pp.status = args.status;
    pp.wait_ns = args.wait_ns;
    if (aligned) {
        if (threadIdx.x == 0) {
            ptx::prefetch_tensormap(&maps.tmW);
            if constexpr (XT == X_CODES) ptx::prefetch_tensormap(&maps.tmT);
            for (int s = 0; s < stages; ++s) {
                ptx::mbar_init(pp.full0 + 8 * s, XT == X_CODES ? 1 : 2);   // + a quantising warp
                ptx::mbar_init(pp.empty0 + 8 * s, 1);
            }
            ptx::mbar_init(pp.tfull0, 1);
            ptx::mbar_init(pp.tfull0 + 8, 1);
            ptx::mbar_init(pp.drain, 1);
            ptx::mbar_init(pp.tempty0, 4);
            misc[1] = 0;
            ptx::fence_mbar_init();
        }
    }
    ptx::cta_sync();
    ptx::griddep_wait();
    // Tensor memory is taken when the kernels before this one are done, and the next
    // one may start when every CTA of this one has it: a CTA that holds tensor memory
    // never waits for one of its stream that still needs it.  Nor for one of another
    // stream: CTAs that share an SM all find their columns (see F8RowsCfg).
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
                ptx::mbar_arrive_expect_tx(fb, (uint32_t)(XT == X_CODES ? Cfg::STAGE_BYTES : Cfg::W_BYTES + 512));
                ptx::tma_load_2d(sW + stage * Cfg::W_BYTES, &maps.tmW, fb, kb * 64, nb * 128);
                ptx::tma_load_2d(sS + stage * Cfg::S_BYTES, &maps.tmSW, fb, (kb >> 2) * 128, nb);
                if constexpr (XT == X_CODES) {
                    ptx::tma_load_2d(sT + stage * Cfg::T_BYTES, &maps.tmT, fb, kb * 64, tb * BT);
                    ptx::tma_load_2d(sS + stage * Cfg::S_BYTES + 512u, &maps.tmST, fb, (kb >> 2) * 128, tb);
                }
                if (++stage == (uint32_t)stages) { stage = 0; phase ^= 1u; }
            }
            if (!ok) pipe_fail(pp);
            // every copy has landed before the ring's memory is used again or the CTA exits
            for (int u = max(0, issued - stages); u < issued; ++u)
                ptx::mbar_wait_bounded(pp.full0 + 8 * (u % stages), (u / stages) & 1, DRAIN_NS, nullptr);
        }
    } else if (aligned && warp == 1) {
        {                                                     // the whole warp: see mma_f8_stage
            const uint64_t w0 = ptx::smem_desc(sW, 16u, 1024u, ptx::SWIZZLE_128B), t0 = ptx::smem_desc(sT, 16u, 1024u, ptx::SWIZZLE_128B);
            const uint64_t s0 = ptx::smem_desc(sS, 16u, 128u, ptx::SWIZZLE_NONE);
            bool ok = true;
            uint32_t stage = 0, phase = 0, chunk = 0, d = pp.tmem;
            for (int kb = kb0, left = chunk_kb; kb < kb1; ++kb, --left) {
                bool begin = kb == kb0;
                if constexpr (CHUNKS) {
                    if (left == 0) {
                        // the chunk before this one is taken over: see rows_chunks
                        if (chunk != 0 && !mx_warp_wait(pp, pp.tempty0, (chunk - 1) & 1u)) { ok = false; break; }
                        ptx::commit_elected(pp.tfull0 + 8 * (chunk & 1u));
                        d = pp.tmem + ++chunk % 3 * BT;
                        left = chunk_kb;
                        begin = true;
                    }
                }
                if (!mx_warp_wait(pp, pp.full0 + 8 * stage, phase)) { ok = false; break; }
                ptx::tc_fence_after();
                ptx::mma_f8_stage(d, w0 + stage * (Cfg::W_BYTES >> 4), t0 + stage * (Cfg::T_BYTES >> 4),
                                  s0 + stage * (Cfg::S_BYTES >> 4), s0 + stage * (Cfg::S_BYTES >> 4) + 32u, pp.tmem + Cfg::SCALE_COL + stage * 8u,
                                  idesc | ptx::f8_scale_id(kb), min(4, nk32 - 4 * kb), begin ? 0u : 1u);
                ptx::commit_elected(pp.empty0 + 8 * stage);
                if (++stage == (uint32_t)stages) { stage = 0; phase ^= 1u; }
            }
            if (ok) ptx::commit_elected(pp.tfull0 + 8 * (chunk & 1u));
            else if (lane == 0) pipe_fail(pp);
            ptx::commit_elected(pp.drain);
            ptx::mbar_wait_bounded(pp.drain, 0, DRAIN_NS, nullptr);
        }
    }
    if constexpr (XT != X_CODES) {
        if (aligned && warp >= 6) quantize_f8_stages<XT, BT>(p, pp, stages, sT, sS, kb0, kb1);
    }
    __syncwarp();
    // The epilogue warps take part in cluster barriers with the others below, so
    // the partial tile is read out in one place for every warp's control flow.
    const int q = warp & 3, n = nb * 128 + q * 32 + lane;
    const bool epi = warp >= 2 && warp < 6;
    const float bias = epi && p.bias != nullptr && n < p.N ? p.bias[n] : 0.0f;
    bool good = aligned;
    uint32_t taddr = pp.tmem + ((uint32_t)(q * 32) << 16), before = taddr;
    bool more = false;                                        // the sum of the chunks before the last is at `before`
    if (epi && aligned) {
        if constexpr (CHUNKS) {
            const int chunks = (kb1 - kb0 + chunk_kb - 1) / chunk_kb;
            good = rows_chunks<BT>(pp, taddr, chunks, lane);
            more = chunks > 1;
            if (more) before = taddr + (uint32_t)((chunks - 2) % 3 * BT), taddr += (uint32_t)((chunks - 1) % 3 * BT);
        } else {
            good = warp_epi_wait(pp, pp.tfull0, 0);
        }
        if (!good) pipe_fail(pp);
        ptx::tc_fence_after();
    }
    // 16 columns of this warp's lanes
    auto sums = [&](int c, float (&z)[16]) {
        uint32_t r[16];
        ptx::tmem_ld16(taddr + c, r);
#pragma unroll
        for (int j = 0; j < 16; ++j) z[j] = __uint_as_float(r[j]);
        if constexpr (CHUNKS) {
            if (!more) return;
            ptx::tmem_ld16(before + c, r);
#pragma unroll
            for (int j = 0; j < 16; ++j) z[j] += __uint_as_float(r[j]);
        }
    };
    if (split == 1) {
        if (epi && good) {
#pragma unroll 1
            for (int c = 0; c < BT; c += 16) {
                if (tb * BT + c >= p.M) break;
                float z[16];
                sums(c, z);
                rows_store(p, p.out, tb * BT + c, n, z, bias);
                __syncwarp();
            }
        }
    } else {
        // partial tile [column][lane] over the ring, whose copies and MMAs are done
        float *part = reinterpret_cast<float *>(smem + Cfg::OFF_RING);
        if (epi && good) {
#pragma unroll 1
            for (int c = 0; c < BT; c += 16) {
                float z[16];
                sums(c, z);
#pragma unroll
                for (int j = 0; j < 16; ++j) part[(c + j) * 128 + q * 32 + lane] = z[j];
            }
        }
        ptx::cluster_sync();
        if (epi && good) {
            // this CTA's slice of the columns that exist: 16 at a time, or the 2 to 8 it has
            const int rows = min(BT, p.M - tb * BT), even = ((rows + split - 1) / split + 15) & ~15;
            const int cols = min(BT / split, even), c0 = rank * cols;
            const uint32_t at = base + Cfg::OFF_RING + (uint32_t)(c0 * 128 + q * 32 + lane) * 4u;
            auto slice = [&](auto ch) {
                constexpr int CH = decltype(ch)::value;
                for (int c = 0; c < cols && tb * BT + c0 + c < p.M; c += CH) {
                    float z[CH];
                    cluster_columns<CH>(at + c * 512u, split, z);
                    rows_store(p, p.out, tb * BT + c0 + c, n, z, bias);
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

template <int BT, int XT, bool CHUNKS>
static cudaError_t launch_rows_t(const F8RowsLaunch &L, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)L.grid);
    cfg.blockDim = dim3(F8_ROWS_THREADS<XT>);
    cfg.dynamicSmemBytes = (size_t)F8RowsCfg<BT, CHUNKS>::smem_bytes(L.args.stages, L.args.split);
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
    return cudaLaunchKernelEx(&cfg, gemm_fp8_rows_kernel<BT, XT, CHUNKS>, L.args);
}

template <int BT, int XT>
static cudaError_t launch_rows_t(const F8RowsLaunch &L, cudaStream_t stream)
{
    return L.chunks ? launch_rows_t<BT, XT, true>(L, stream) : launch_rows_t<BT, XT, false>(L, stream);
}

cudaError_t launch_gemm_fp8_rows(const F8RowsLaunch &L, cudaStream_t stream)
{
    if (L.x_type == IN_BF16) return launch_rows_t<16, IN_BF16>(L, stream);
    if (L.x_type == IN_F16) return launch_rows_t<16, IN_F16>(L, stream);
    if (L.x_type == IN_F32) return launch_rows_t<16, IN_F32>(L, stream);
    switch (L.bt) {
    case 16: return launch_rows_t<16, X_CODES>(L, stream);
    case 32: return launch_rows_t<32, X_CODES>(L, stream);
    case 64: return launch_rows_t<64, X_CODES>(L, stream);
    default: return launch_rows_t<128, X_CODES>(L, stream);
    }
}

template <int BT, int XT>
static cudaError_t setup_rows_t()
{
    using Cfg = F8RowsCfg<BT>;
    const auto smem = cudaFuncAttributeMaxDynamicSharedMemorySize;
    constexpr int bytes = Cfg::OFF_RING + Cfg::MAX_STAGES * Cfg::STAGE_BYTES;
    const cudaError_t e = cudaFuncSetAttribute(gemm_fp8_rows_kernel<BT, XT, false>, smem, bytes);
    return e == cudaSuccess ? cudaFuncSetAttribute(gemm_fp8_rows_kernel<BT, XT, true>, smem, bytes) : e;
}

// Clusters of `split` CTAs that are resident at once (with full rings).
static cudaError_t rows_clusters(int split, int *n)
{
    using Cfg = F8RowsCfg<128>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(split * 64));
    cfg.blockDim = dim3(F8_ROWS_THREADS<X_CODES>);
    cfg.dynamicSmemBytes = Cfg::OFF_RING + Cfg::MAX_STAGES * Cfg::STAGE_BYTES;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(n, gemm_fp8_rows_kernel<128, X_CODES, false>, &cfg);
}

cudaError_t setup_fp8_rows_kernels(int (&max_clusters)[4])
{
    cudaError_t e = setup_rows_t<16, X_CODES>();
    if (e == cudaSuccess) e = setup_rows_t<32, X_CODES>();
    if (e == cudaSuccess) e = setup_rows_t<64, X_CODES>();
    if (e == cudaSuccess) e = setup_rows_t<128, X_CODES>();
    if (e == cudaSuccess) e = setup_rows_t<16, IN_BF16>();
    if (e == cudaSuccess) e = setup_rows_t<16, IN_F16>();
    if (e == cudaSuccess) e = setup_rows_t<16, IN_F32>();
    max_clusters[0] = 1 << 30;
    for (int i = 1; i < 4 && e == cudaSuccess; ++i) e = rows_clusters(1 << i, &max_clusters[i]);
    return e;
}

}  // namespace mmact
