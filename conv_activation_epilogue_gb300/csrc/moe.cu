// moe.cu -- a whole mixture-of-experts layer for a few tokens (T <= 64) in two
// kernels.
//
//   router kernel    logits[t][e] = x[t] . router[e] + rb[e]
//   experts kernel   the k experts of each token (largest logits, ties to the
//                    lowest index) and their softmax weights; for every chosen
//                    expert, read once for up to 32 of its tokens:
//                    h = act(g) * u, g and u the two halves of w1[e] x + b1[e]
//                    (or h = act(w1[e] x + b1[e])); a grid barrier;
//                    o = w2[e] h + b2[e]; a grid barrier; y[t] = sum_j p[t][j] o[t, j]
//
// With few tokens every weight is used a handful of times: the time is that of
// reading the chosen experts' weights once, and everything is arranged so that
// the copies never stop.  The experts kernel is persistent, one CTA on each SM,
// taking the items in turn (a tile of weight rows x all of K of one expert; for a
// gated layer half of the rows are gate rows and half the up rows that go with
// them):
//
//   warp 0       producer: TMA boxes of 128 bytes of K of the tile's halves.  It runs
//                ahead over items and over the grid barrier: weights of the down
//                product are on their way while the last h is being finished.
//   warp 9       tokens of the stage (x, or h once the grid barrier is passed), one
//                bulk copy for each token
//   warps 1..8   products: each has 8 + 8 rows of the tile on mma.sync.m16n8k16
//                as the 16-row operand (a gate row and its up row meet in one
//                thread) and eight tokens to its columns, over all of K, so no sums
//                cross warps; bias, activation and stores follow in registers.
//                Which K a lane holds does not matter to a sum over K as long as
//                both operands agree, so fragments are 16-byte loads in memory
//                order.
//
// The intermediate h is held as three bf16 parts of 8 bits each, h = hi + mid + lo
// exactly, and multiplied as all of them: nothing is rounded between the two
// products.  (Two parts, 16 bits of h, take 3 % less of the time of 64 tokens, and put y
// in bf16 1.0e-4 instead of 0.6e-4, in the 2-norm, from what fp32 gives.)  fp16 down
// weights are split into two (hi + lo is exact), which keeps h's fp32 range; of their
// products with the parts, lo x the last part, 2^-24 of the whole, is left out.
//
// Measured (bf16, GB300): 64 tokens, 8 of 64 experts of 4096 x 1792 (2.8 GB of weights)
// 451 to 463 us, 6.2 TB/s.  One token, 8 of 64 experts of 2048 x 1024 (101 MB): 33 us, of
// which the weights take 15; the router kernel is 4, choice and lists 4, the two grid
// barriers with what they leave idle 5.  With more than 16 tokens an expert the down product's three
// parts keep the tensor pipe busy for longer than its weights come in: 64 tokens, 8 of
// 8 experts of 4096 x 1792, 207 us (fp16, five products for each weight: 244), the bytes 53.
#include "moe.cuh"

namespace mmact {

constexpr int MOE_MMA_WARPS = 8;
constexpr int MOE_THREADS = 32 * (2 + MOE_MMA_WARPS);

// ------------------------------------------------------------------ helpers --
// c += a 16 x 16 tile of weights by 16 x 8 of tokens.  The tensor core does not round
// this sum but truncates it: over 256 of these in a row, 4096 K of products of one sign,
// sums were measured 100 (bf16) to 220 (fp16) units of 2^-23 too small, so that more
// of y's bf16 values than with sums rounded to nearest came out a step away.
template <bool BF16>
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1)
{
    if constexpr (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Where the first part of h of a slot at `row` stands; the others follow MOE_STAGE_K
// values apart.
__device__ __forceinline__ int64_t h_at(const MoeArgs &p, int64_t slot, int row)
{
    return slot * p.Ip * MOE_PARTS + (int64_t)(row / MOE_STAGE_K) * (MOE_PARTS * MOE_STAGE_K) + row % MOE_STAGE_K;
}

// h as three bf16 parts: the first 8 bits, the next, the last.  All of them have h's
// sign and none is 0 unless h is (a part that leaves nothing for the next ones is
// taken one step smaller), so that an infinite weight makes the infinity that it makes
// with h itself, and no NaN.  An infinite h is 1 + 1 + infinity: what meets the last part
// are the weights' hi halves, which are 0 only where the weights are.
__device__ __forceinline__ void put_parts(uint16_t *h, float v)
{
    const bool inf = (__float_as_uint(v) & 0x7fffffffu) == 0x7f800000u;
#pragma unroll
    for (int j = 0; j < MOE_PARTS - 1; ++j) {
        uint32_t b = __float_as_uint(v) & 0xffff0000u;
        if (v == __uint_as_float(b) && v != 0.0f) b -= 0x10000u;
        if (inf) b = 0x3f800000u | (b & 0x80000000u);
        h[j * MOE_STAGE_K] = (uint16_t)(b >> 16);
        v -= __uint_as_float(b);
    }
    h[(MOE_PARTS - 1) * MOE_STAGE_K] = (uint16_t)(__float_as_uint(v) >> 16);
}

// Hi and lo bf16 halves of a pair of fp16 values.  Where a value is infinite, lo is the
// number 256 and not the NaN of inf - inf: no lo is above 128.
__device__ __forceinline__ void split_pair(float a, float b, uint32_t &hi, uint32_t &lo)
{
    hi = pack2<OUT_BF16>(a, b);
    const float2 f = unpack2<OUT_BF16>(hi);
    asm("min.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(pack2<OUT_BF16>(a - f.x, b - f.y)), "r"(0x43804380u));
}

// ------------------------------------------------------------------- router --
// The CTAs past the logits' prepare what the experts kernel reads: its counters, x
// with zeros up to a whole stage, and the same zeros of h.
template <int XT>
__global__ void __launch_bounds__(MOE_ROUTER_THREADS) moe_router_kernel(const MoeArgs p, int token_groups)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    if ((int)blockIdx.x < p.E * token_groups) {
        router_logits<XT>(p, (int)blockIdx.x, token_groups);
        return;
    }
    // MOE_ROUTER_K of one token, 8 values to a thread
    const int chunks = (p.Hp + MOE_ROUTER_K - 1) / MOE_ROUTER_K, at = (int)blockIdx.x - p.E * token_groups, t = at / chunks;
    const int k = (at - t * chunks) * MOE_ROUTER_K + (int)threadIdx.x * 8;
    if (at == 0 && threadIdx.x < 2) p.counters[threadIdx.x] = 0;
    if (k < p.Hp)
        *reinterpret_cast<uint4 *>(p.x_pad + (int64_t)t * p.Hp + k) =
            k < p.H ? __ldcg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.x) + (int64_t)t * p.H + k))
                    : make_uint4(0, 0, 0, 0);
    fence_proxy_async_all();                                   // bulk copies read x and the zeros
    if (at != t * chunks) return;
    const int pad = (p.Ip - p.I) / 8;                          // eights of zeros past h's rows
    for (int i = threadIdx.x; i < pad * p.top; i += MOE_ROUTER_THREADS) {
        const int64_t to = h_at(p, (int64_t)t * p.top + i / pad, p.I + i % pad * 8);
#pragma unroll
        for (int j = 0; j < MOE_PARTS; ++j) *reinterpret_cast<uint4 *>(p.h + to + j * MOE_STAGE_K) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_all();
}

// ----------------------------------------------------------------- products --
// A warp's view of an item.
struct MoeItem {
    uint32_t row;                    // shared address of this lane's row in the lower half, from a stage's start
    uint32_t upper;                  // from there to its row in the upper half
};

// Tokens of one piece of K (16 bytes of each row): this lane's 8 values of one
// token of each eight, x or the parts of h.
template <int NT, bool DOWN>
struct MoeTokens {
    static constexpr int PARTS = DOWN ? MOE_PARTS : 1;
    uint4 v[PARTS][NT];
};

template <int NT, bool DOWN>
__device__ __forceinline__ void load_tokens(MoeTokens<NT, DOWN> &x, uint32_t at)
{
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < MoeTokens<NT, DOWN>::PARTS; ++j) x.v[j][n] = ptx::ld_shared_v4(at + n * 8 * MOE_RECORD + j * MOE_PART);
}

// c += 16 rows x eight tokens over one piece: a, b the two rows' four pairs of values,
// v the tokens'.
template <bool BF>
__device__ __forceinline__ void piece_mma(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[4], const uint4 &v)
{
    mma_16816<BF>(c, a[0], b[0], a[1], b[1], v.x, v.y);
    mma_16816<BF>(c, a[2], b[2], a[3], b[3], v.z, v.w);
}

// The rings of one CTA.
struct MoePipe {
    Pipe pp;                         // weights: full0, empty0
    uint32_t tfull0, tempty0;        // tokens
    uint32_t ring, tokens;           // shared addresses
    uint32_t stages, tstages, stage_bytes, token_bytes;
};

// A role's place in a ring.
struct MoePlace {
    uint32_t slot, phase;
    __device__ __forceinline__ void next(uint32_t stages)
    {
        if (++slot == stages) slot = 0, phase ^= 1u;
    }
};

// What a warp multiplies in one stage: units of 32 K, 8 values to a lane of its two
// rows and of its tokens.
template <int NT, bool DOWN>
struct MoeFragments {
    uint4 a[2 * MOE_BOXES], b[2 * MOE_BOXES];
    MoeTokens<NT, DOWN> x[2 * MOE_BOXES];
};

// A warp's walk over the stages of its items.
struct MoeWalk {
    MoePlace w, t;
};

template <int NT, bool DOWN>
__device__ __forceinline__ bool fetch(MoeFragments<NT, DOWN> &f, const MoePipe &m, const MoeItem &it, const MoeWalk &walk, int s)
{
    const int lane = threadIdx.x & 31;
    const uint32_t sw = (uint32_t)(lane >> 2), t4 = (uint32_t)(lane & 3);   // the 128-byte swizzle: chunk ^ (row & 7)
    const uint32_t c0 = (t4 ^ sw) << 4, c1 = ((4u + t4) ^ sw) << 4;
    const uint32_t part = (uint32_t)s % MOE_SPAN<DOWN>;
    const uint32_t row = m.ring + walk.w.slot * m.stage_bytes + it.row;
    const uint32_t tok = m.tokens + walk.t.slot * m.token_bytes + sw * MOE_RECORD + part * (MOE_STAGE_K * 2u) + t4 * 16u;
    if (part == 0 && !mx_warp_wait(m.pp, m.tfull0 + 8 * walk.t.slot, walk.t.phase)) return false;
    if (!mx_warp_wait(m.pp, m.pp.full0 + 8 * walk.w.slot, walk.w.phase)) return false;
#pragma unroll
    for (int u = 0; u < 2 * MOE_BOXES; ++u) {
        const uint32_t at = row + (uint32_t)(u >> 1) * (2u * it.upper) + (u & 1 ? c1 : c0);
        f.a[u] = ptx::ld_shared_v4(at);
        f.b[u] = ptx::ld_shared_v4(at + it.upper);
        load_tokens<NT, DOWN>(f.x[u], tok + u * 64u);
    }
    return true;
}

// A stage's products.  Each piece has a sum of its own on the tensor core, a few
// instructions long, its smallest parts first, which is added to the running sum by an
// fp32 addition.  SPLITW: fp16 weights as two bf16 halves, whose lo halves meet the
// tokens' first two parts only.
template <bool BF, int NT, bool DOWN, bool SPLITW>
__device__ __forceinline__ void multiply(float (&acc)[NT][4], const MoeFragments<NT, DOWN> &f)
{
#pragma unroll
    for (int u = 0; u < 2 * MOE_BOXES; ++u) {
        uint32_t a[4] = {f.a[u].x, f.a[u].y, f.a[u].z, f.a[u].w}, b[4] = {f.b[u].x, f.b[u].y, f.b[u].z, f.b[u].w};
        uint32_t al[4], bl[4];
        if constexpr (SPLITW) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 va = unpack2<OUT_F16>(a[i]), vb = unpack2<OUT_F16>(b[i]);
                split_pair(va.x, va.y, a[i], al[i]);
                split_pair(vb.x, vb.y, b[i], bl[i]);
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float c[4] = {};
#pragma unroll
            for (int j = MoeTokens<NT, DOWN>::PARTS - 1; j >= 0; --j) {
                if constexpr (SPLITW) {
                    if (j < MOE_PARTS - 1) piece_mma<true>(c, al, bl, f.x[u].v[j][n]);
                }
                piece_mma<BF || SPLITW>(c, a, b, f.x[u].v[j][n]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] += c[i];
        }
    }
}

template <bool DOWN>
__device__ __forceinline__ void give_back(const MoePipe &m, MoeWalk &walk, int s, int stages)
{
    const bool last = s % MOE_SPAN<DOWN> == MOE_SPAN<DOWN> - 1 || s == stages - 1;      // of its stage of tokens
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
        ptx::mbar_arrive(m.pp.empty0 + 8 * walk.w.slot);
        if (last) ptx::mbar_arrive(m.tempty0 + 8 * walk.t.slot);
    }
    walk.w.next(m.stages);
    if (last) walk.t.next(m.tstages);
}

// One warp's rows of an item over all of K.
template <bool BF, int NT, bool DOWN, bool SPLITW>
__device__ __forceinline__ bool item_mma(float (&acc)[NT][4], const MoePipe &m, const MoeProduct &pr, const MoeItem &it,
                                         MoeWalk &walk)
{
#pragma unroll 1
    for (int s = 0; s < pr.stages; ++s) {
        MoeFragments<NT, DOWN> f;
        if (!fetch<NT, DOWN>(f, m, it, walk, s)) return false;
        multiply<BF, NT, DOWN, SPLITW>(acc, f);
        give_back<DOWN>(m, walk, s, pr.stages);
    }
    return true;
}

// One item of the up (DOWN = false) or down product by one warp, stores included.
template <int XT, bool DOWN, int NT>
__device__ __forceinline__ bool run_item(const MoeArgs &p, const MoeShared &S, const MoePipe &m, const MoeProduct &pr,
                                         MoeWalk &walk, int ai, int tile)
{
    const int w = (int)(threadIdx.x >> 5) - 1, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int e = S.act[ai], first = S.first[ai], cnt = S.first[ai + 1] - first;
    const int r = tile * pr.step + 8 * w + g;                  // this lane's row in the lower half, within the expert
    const int64_t ra = (int64_t)e * pr.rows + r, rb = ra + pr.half;
    MoeItem it;
    it.row = (uint32_t)(8 * w + g) * 128u;
    it.upper = (uint32_t)p.half_rows * 128u;
    float acc[NT][4] = {};
    if (!item_mma<XT == OUT_BF16, NT, DOWN, DOWN && XT == OUT_F16>(acc, m, pr, it, walk)) return false;

    // acc[n][0..1]: the lower row, tokens n * 8 + 2 t4 and the next; acc[n][2..3]: the upper row
    const bool gated = pr.pairs;
    const int r2 = gated ? r : r + pr.half;
    const bool in1 = r < pr.limit, in2 = !gated && r2 < pr.limit;
    const float *bias = DOWN ? p.b2 : p.b1;
    const float bias1 = bias != nullptr && in1 ? bias[ra] : 0.0f;
    const float bias2 = bias != nullptr && (gated ? in1 : in2) ? bias[rb] : 0.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = n * 8 + 2 * t4 + j;
            if (c >= cnt) continue;
            const int64_t s = S.slot[first + c];
            float v1 = acc[n][j] + bias1, v2 = acc[n][2 + j] + bias2;
            if constexpr (DOWN) {
                if (in1) p.part[s * p.H + r] = v1;
                if (in2) p.part[s * p.H + r2] = v2;
            } else {
                auto put = [&](int row, float v) { put_parts(p.h + h_at(p, s, row), v); };
                v1 = act_mx(p.act, v1, p.alpha);
                if (gated) {
                    if (in1) put(r, v1 * v2);
                } else {
                    if (in1) put(r, v1);
                    if (in2) put(r2, act_mx(p.act, v2, p.alpha));
                }
            }
        }
    return true;
}

template <int XT, bool DOWN>
__device__ __forceinline__ bool mma_phase(const MoeArgs &p, const MoeShared &S, const MoePipe &m, const MoeProduct &pr,
                                          MoeWalk &walk)
{
    const int n = S.nact * pr.tiles;
    for (int i = blockIdx.x; i < n; i += gridDim.x) {
        const int ai = i / pr.tiles, tile = i - ai * pr.tiles, cnt = S.first[ai + 1] - S.first[ai];
        // moe_eights(cnt), spelled out (by its value 64 tokens, 8 of 64 experts of 4096 x 1792 took 461 us instead of 457)
        const bool ok = cnt <= 8    ? run_item<XT, DOWN, 1>(p, S, m, pr, walk, ai, tile)
                        : cnt <= 16 ? run_item<XT, DOWN, 2>(p, S, m, pr, walk, ai, tile)
                                    : run_item<XT, DOWN, 4>(p, S, m, pr, walk, ai, tile);
        if (!ok) return false;
    }
    return true;
}

// ------------------------------------------------------------------- kernel --
__device__ __forceinline__ bool produce(const CUtensorMap *map, const MoeArgs &p, const MoeShared &S, const MoePipe &m,
                                        const MoeProduct &pr, MoePlace &to, uint64_t pol)
{
    const int n = S.nact * pr.tiles;
    const uint32_t box = (uint32_t)p.half_rows * 128u;
    for (int i = blockIdx.x; i < n; i += gridDim.x) {
        const int ai = i / pr.tiles, tile = i - ai * pr.tiles, row = S.act[ai] * pr.rows + tile * pr.step;
        // the upper half of the last tile may have no rows (its products are not stored either)
        const bool both = pr.pairs || tile * pr.step + p.half_rows < pr.limit;
        for (int s = 0; s < pr.stages; ++s, to.next(m.stages)) {
            const uint32_t full = m.pp.full0 + 8 * to.slot, at = m.ring + to.slot * m.stage_bytes;
            if (!mx_warp_wait(m.pp, m.pp.empty0 + 8 * to.slot, to.phase ^ 1u)) return false;
            elected_expect_tx(full, (both ? 2u * box : box) * MOE_BOXES);
#pragma unroll
            for (int b = 0; b < MOE_BOXES; ++b) {              // K past the end arrives as zeros
                elected_load_2d(at + 2u * b * box, map, full, s * MOE_STAGE_K + 64 * b, row, pol);
                if (both) elected_load_2d(at + (2u * b + 1u) * box, map, full, s * MOE_STAGE_K + 64 * b, row + pr.half, pol);
            }
        }
    }
    return true;
}

// The tokens of every item, in the weights' order: lane c copies token c's pieces.
template <bool DOWN>
__device__ __forceinline__ bool produce_tokens(const MoeArgs &p, const MoeShared &S, const MoePipe &m, const MoeProduct &pr,
                                               MoePlace &to)
{
    const int lane = threadIdx.x & 31, n = S.nact * pr.tiles;
    for (int i = blockIdx.x; i < n; i += gridDim.x) {
        const int ai = i / pr.tiles, first = S.first[ai], cnt = S.first[ai + 1] - first;
        const int64_t slot_of = lane < cnt ? S.slot[first + lane] : 0;
        const uint16_t *from = DOWN ? p.h + slot_of * p.Ip * MOE_PARTS : p.x_pad + slot_of / p.top * p.Hp;
        for (int s = 0; s < pr.tstages; ++s, to.next(m.tstages)) {
            const uint32_t full = m.tfull0 + 8 * to.slot;
            const uint32_t at = m.tokens + to.slot * m.token_bytes + (uint32_t)lane * MOE_RECORD;
            if (!mx_warp_wait(m.pp, m.tempty0 + 8 * to.slot, to.phase ^ 1u)) return false;
            elected_expect_tx(full, (uint32_t)cnt * MOE_TOKEN<DOWN>);
            __syncwarp();
            if (lane < cnt) bulk_load(at, from + (int64_t)s * (MOE_TOKEN<DOWN> / 2), MOE_TOKEN<DOWN>, full);
            __syncwarp();
        }
    }
    return true;
}

// Every copy has landed before the CTA exits: the last one of each slot, from the
// oldest on (before the first round, a slot of an earlier phase has no copy and its
// barrier's phase before the first counts as complete).
__device__ __forceinline__ void drain(const Pipe &pp, uint32_t full0, MoePlace to, uint32_t stages)
{
    for (uint32_t i = 0; i < stages; ++i, to.next(stages))
        ptx::mbar_wait_bounded(full0 + 8 * to.slot, to.phase ^ 1u, DRAIN_NS, nullptr);
}

template <int XT>
__global__ void __launch_bounds__(MOE_THREADS, 1)
    moe_experts_kernel(const __grid_constant__ CUtensorMap tm1, const __grid_constant__ CUtensorMap tm2, const MoeArgs p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    const MoeLayout layout(p.T, p.half_rows);
    MoeShared &S = *reinterpret_cast<MoeShared *>(smem + layout.off_shared);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    ptx::griddep_launch_dependents();
    const int active = p.half_rows / 8;                        // product warps that have rows
    MoePipe m;
    m.ring = ptx::smem_addr(smem);
    m.tokens = m.ring + (uint32_t)layout.off_tokens;
    m.stages = (uint32_t)layout.stages;
    m.tstages = (uint32_t)layout.tstages;
    m.stage_bytes = (uint32_t)layout.stage_bytes;
    m.token_bytes = (uint32_t)layout.token_bytes;
    m.pp.full0 = ptx::smem_addr(S.bar);
    m.pp.empty0 = m.pp.full0 + 8 * m.stages;
    m.tfull0 = m.pp.empty0 + 8 * m.stages;
    m.tempty0 = m.tfull0 + 8 * m.tstages;
    m.pp.abort = reinterpret_cast<volatile uint32_t *>(&S.abort_flag);
    m.pp.status = p.status;
    m.pp.wait_ns = p.wait_ns;
    const bool aligned = (m.ring & 1023u) == 0;                // the swizzle counts rows from multiples of 1024 bytes
    if (threadIdx.x == 0) {
        if (!aligned) atomicOr(p.status, ST_SMEM_ALIGN);
        ptx::prefetch_tensormap(&tm1);
        ptx::prefetch_tensormap(&tm2);
        for (uint32_t s = 0; s < m.stages; ++s) {
            ptx::mbar_init(m.pp.full0 + 8 * s, 1);
            ptx::mbar_init(m.pp.empty0 + 8 * s, (uint32_t)active);
        }
        for (uint32_t s = 0; s < m.tstages; ++s) {
            ptx::mbar_init(m.tfull0 + 8 * s, 1);
            ptx::mbar_init(m.tempty0 + 8 * s, (uint32_t)active);
        }
        S.abort_flag = aligned ? 0 : 1;
        ptx::fence_mbar_init();
    }
    ptx::griddep_wait();                                       // the router's logits
    plan_experts<MOE_GROUP, MOE_THREADS>(p, S, reinterpret_cast<uint32_t *>(smem),
                                         reinterpret_cast<uint32_t *>(smem + p.T * p.E * 4));

    const MoeProduct up = up_product(p, MOE_STAGE_K, MOE_TOKEN_K<false>), down = down_product(p, MOE_STAGE_K, MOE_TOKEN_K<true>);
    bool ok = aligned;
    if (warp == 0) {
        MoePlace to = {0, 0};
        const uint64_t pol = ptx::createpolicy_evict_first();  // weights are read once
        ok = ok && produce(&tm1, p, S, m, up, to, pol) && produce(&tm2, p, S, m, down, to, pol);
        if (!ok && lane == 0) pipe_fail(m.pp);
        drain(m.pp, m.pp.full0, to, m.stages);
    } else if (warp == 1 + MOE_MMA_WARPS) {
        MoePlace to = {0, 0};
        fence_proxy_async_all();
        ok = ok && produce_tokens<false>(p, S, m, up, to);
        // every h is written before any is read
        if (ok) ok = __all_sync(0xffffffffu, lane != 0 || grid_wait(m.pp, p.counters)) != 0;
        fence_proxy_async_all();
        ok = ok && produce_tokens<true>(p, S, m, down, to);
        if (!ok && lane == 0) pipe_fail(m.pp);
        drain(m.pp, m.tfull0, to, m.tstages);
    } else {
        MoeWalk walk = {};
        if (ok && warp <= active) ok = mma_phase<XT, false>(p, S, m, up, walk);
        // this CTA's part of h is written
        fence_proxy_async_all();
        __syncwarp();
        asm volatile("barrier.sync 1, %0;" ::"n"(32 * MOE_MMA_WARPS) : "memory");
        if (ok && threadIdx.x == 32) grid_arrive(p.counters);
        __syncwarp();
        if (ok && warp <= active) ok = mma_phase<XT, true>(p, S, m, down, walk);
        if (!ok && lane == 0) pipe_fail(m.pp);
    }
    __syncwarp();
    sum_experts<XT, MOE_THREADS>(p, S, m.pp);
}

template <int XT>
static cudaError_t launch_t(const MoeLaunch &L, cudaStream_t stream)
{
    const MoeArgs &a = L.args;
    const int groups = (a.T + 7) / 8;
    const int ctas = a.E * groups + a.T * ((a.Hp + MOE_ROUTER_K - 1) / MOE_ROUTER_K);
    const cudaError_t e = launch_k(moe_router_kernel<XT>, dim3((unsigned)ctas), dim3(MOE_ROUTER_THREADS), 0, stream, a, groups);
    if (e != cudaSuccess) return e;
    return launch_cooperative(moe_experts_kernel<XT>, L.grid, MOE_THREADS,
                              (size_t)MoeLayout(a.T, a.half_rows).off_shared + sizeof(MoeShared), stream, L.tm1, L.tm2, a);
}

cudaError_t setup_moe_kernels()
{
    const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    const cudaError_t e = cudaFuncSetAttribute(moe_experts_kernel<OUT_BF16>, attr, MOE_RINGS + (int)sizeof(MoeShared));
    return e == cudaSuccess ? cudaFuncSetAttribute(moe_experts_kernel<OUT_F16>, attr, MOE_RINGS + (int)sizeof(MoeShared)) : e;
}

cudaError_t launch_moe(const MoeLaunch &L, cudaStream_t stream)
{
    return L.x_out == OUT_BF16 ? launch_t<OUT_BF16>(L, stream) : launch_t<OUT_F16>(L, stream);
}

}  // namespace mmact
