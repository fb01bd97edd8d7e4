// Grouped products of microscaled 4-bit floating point (MXFP4): e2m1 codes with a power of two as scale for every 32
// values along the contraction, in both operands. Expert e owns the rows [offs[e], offs[e + 1]):
//
//   y[p, n] = sum_b 2^(xs[p, b] + ws[e, n, b]) (sum_{k in block b} x[p, k] w[e, n, k])
//
// The scales are powers of two, so that the tensor cores apply them: tcgen05.mma (kind::mxf4, block_scale) takes 64
// contraction steps of packed codes from shared memory and both operands' scale bytes from tensor memory, and adds
// to fp32 accumulators there. A stage is 256 steps: 128 bytes of codes per row (TMA, 128-byte swizzle) and two words
// of four scale bytes. The weights' words lie in memory in the order that tensor memory wants (tiles of 128 rows x
// 128 steps, 512 bytes: 32 lanes of four words), a bulk copy brings them in; a batch's words lie by row, and two
// warps put them into that order on their way through shared memory. tcgen05.cp moves both to tensor memory, in
// order with the MMAs that follow it.
//
// What bounds it, measured on one GB300 (copy bandwidth 6.7 TB/s, cuBLAS bf16 1919 TFLOP/s):
//   - many rows: shared memory, by this count: a stage of a wide tile (256 x 192 x 256 by a pair of CTAs) writes 31 KB to
//     each SM's and its MMAs read 28 KB back, 470 cycles at 128 bytes each; the MMAs alone take 384 and the six copies of
//     scales 120. (What L2 delivers, 42 bytes a cycle and SM, may count as well: the two were not told apart.)
//     8192 x 8192 x 8192 takes 150 us, 7300 TFLOP/s; 4096 x 4096 x 4096 (352 units on 76 pairs, five rounds) 28.7 us, 4800:
//     18 us of it are five rounds of 16 stages, the rest was not taken apart.
//   - skewed routing: 8192 tokens to 8 of 256 experts of 1024 x 2048 (65536 rows, 0.41 GB) 90 us, 4.6 TB/s: a round of
//     units takes 470 cycles a stage, and 1100 more where the unit before goes through shared memory on its way out;
//     experts' last tiles fill 256 rows by two thirds.
//   - few rows: the weights' one pass through memory. 64 tokens to 222 of 256 experts of 1024 x 2048 (0.25 GB) take 42 us,
//     5.9 TB/s, 3 of them before the first bytes arrive; of 4096 x 4096 (2 GB) 285 us, 6.9 TB/s.
//   - one token: latency. Eight rows, 2048 x 512: 4 us after SwiGLU's 2.5.
#include <cuda_bf16.h>

#include <type_traits>

#include "group_gemm.cuh"

namespace ftmoe {

namespace {

using namespace grp;

constexpr int kThreads4 = 416;   // warps: 0 TMA, 1 MMA, 2-3 scales of x, 4..11 epilogue, 12 units
constexpr int kStep4 = 256;      // contraction steps per stage
constexpr int kTileBytes = 512;  // scale words of 128 rows x 128 steps
// fp32 outputs: sums in parts of this many stages (32 instructions), added in registers, since the tensor cores
// truncate where an fp32 addition rounds.
constexpr int kPart4 = 8;

template <int BN>
struct Ring4 {
    static constexpr int b_bytes = BN * kChunkBytes;
    static constexpr int sf_bytes = 2 * kTileBytes;  // of one operand and stage
    static constexpr int stage = kABytes + b_bytes + 2 * sf_bytes;
    static constexpr int fit = 208 * 1024 / stage;
    static constexpr int stages = fit < 8 ? fit : 8;
    static constexpr int box_rows = BN <= 32 ? 16 : 32;
    static constexpr int group = BN <= 32 ? 4 : 2;   // stages whose scale words a warp loads together
    static constexpr int sf_col = 2 * BN;            // tensor memory: two accumulators, then two stages' scales
    static constexpr int tmem = BN <= 32 ? 128 : 512;
};

struct Group4Params {
    const int *offs;
    int E, P, N, K;
    const uint32_t *xs;   // [ceil(K / 128)][ld_xs]
    int64_t ld_xs;
    const uint8_t *ws;    // [E][ceil(N / 128)][ceil(K / 128)][512]
    void *out;            // [P][ld]
    int64_t ld;
    int split;            // CTAs (one cluster) that share a unit's contraction
    int pairs;            // bf16 out: N even and rows 4-byte aligned
    int vec;              // N and the rows of out are multiples of 16 bytes
    int *status;
    uint64_t wait_ns;
    int skip_producer;
};

// D[tmem] (+)= A[smem] x B[smem]^T over 64 e2m1 steps, with the scale bytes at sfa and sfb (in tensor memory).
template <int CG>
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate)
{
    if constexpr (CG == 1) {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    }
}

// 512 bytes of shared memory, 16 for each of 32 lanes, to four columns of tensor memory, the same in all four
// quarters of the lanes.
template <int CG>
__device__ __forceinline__ void copy_scales(uint32_t to, uint64_t from)
{
    if constexpr (CG == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(to), "l"(from) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(to), "l"(from) : "memory");
}

// Whether phase `parity` of `bar` is complete, without waiting; if so, what other CTAs of the cluster released is seen.
__device__ __forceinline__ bool test_cluster(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Shared-memory descriptor of such 512 bytes: no swizzle, groups of eight 16-byte rows 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t smem_addr)
{
    uint64_t d = 0;
    d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
    d |= (uint64_t)1 << 16;
    d |= (uint64_t)(128 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    return d;
}

// kind::mxf4 instruction descriptor: e2m1 operands (1 at bits 7 and 10), scales that are powers of two (bit 23).
// The bytes of a word that an instruction takes: `pair` 0 the lower two, 1 the upper two (bits 4 and 29).
__device__ __forceinline__ uint32_t idesc_mxf4(int M, int N, int pair)
{
    return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24) |
           ((uint32_t)(2 * pair) << 4) | ((uint32_t)(2 * pair) << 29);
}

// Where a unit's tile lies: found by one warp of the CTA ahead of the others, which take it from a ring in shared memory.
// (The issuing warps found it themselves at first, by a binary search over the experts and a division: 800 cycles with one
// expert and up to 2000 with 256, during which the tensor cores stood still between two units.)
struct Unit4 {
    int e;           // expert, or -1 after the last unit
    int row0;        // first row of the tile
    int lo, hi;      // wide tiles: rows [row0 + lo, row0 + hi) are the expert's; else lo = 0 and hi of them are
    int n0;          // first weight row
    int cols;        // columns of an MMA: rows (wide tiles: weight rows) in whole MMA columns
    int width;       // wide tiles: weight rows
    int unused;
};
static_assert(sizeof(Unit4) == 32, "two 16-byte stores");

constexpr int kUnitSlots = 4;

struct UnitRing {
    Unit4 *slot;
    uint64_t *full, *empty;
    volatile int *abort_flag;
    uint64_t wl;
    int turn = 0;

    __device__ __forceinline__ UnitRing(void *smem, uint64_t *bars, volatile int *flag, uint64_t limit)
        : slot(static_cast<Unit4 *>(smem)), full(bars), empty(bars + kUnitSlots), abort_flag(flag), wl(limit) {}

    // By one thread: `readers` warps take every unit.
    __device__ __forceinline__ void init(int readers)
    {
        for (int i = 0; i < kUnitSlots; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, readers);
        }
    }

    // The finding warp; false: given up.
    __device__ __forceinline__ bool put(const Unit4 &x)
    {
        const int i = turn % kUnitSlots;
        if (!warp_wait(empty + i, ((turn / kUnitSlots) & 1) ^ 1, abort_flag, wl)) return false;
        if ((threadIdx.x & 31) == 0) {
            int4 *to = reinterpret_cast<int4 *>(slot + i);
            to[0] = make_int4(x.e, x.row0, x.lo, x.hi);
            to[1] = make_int4(x.n0, x.cols, x.width, 0);
            mbar_arrive(full + i);
        }
        __syncwarp();
        ++turn;
        return true;
    }

    // The others: the next unit, the same in all lanes. `dead` is set where the wait gave up.
    __device__ __forceinline__ bool get(Unit4 &x, bool &dead)
    {
        const int i = turn % kUnitSlots;
        if (!warp_wait(full + i, (turn / kUnitSlots) & 1, abort_flag, wl)) {
            dead = true;
            return false;
        }
        const int4 *from = reinterpret_cast<const int4 *>(slot + i);
        const int4 a = from[0], b = from[1];
        x.e = uniform(a.x); x.row0 = uniform(a.y); x.lo = uniform(a.z); x.hi = uniform(a.w);
        x.n0 = uniform(b.x); x.cols = uniform(b.y); x.width = uniform(b.z);
        if ((threadIdx.x & 31) == 0) mbar_arrive(empty + i);  // (after the shuffles: every lane has read)
        ++turn;
        return x.e >= 0;
    }
};

}  // namespace

template <int BN, bool F32>
__global__ void __launch_bounds__(kThreads4, 1)
    group_gemm_mxfp4_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                            const __grid_constant__ Group4Params p)
{
    using T = Ring4<BN>;
    constexpr int S = T::stages;
    constexpr int HC = BN / 2;               // columns of one half's epilogue warps
    constexpr int W = HC < 32 ? HC : 32;     // columns per tensor-memory load
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + S * T::stage);
    uint64_t *empty = full + S, *sc_full = empty + S, *acc_full = sc_full + S, *acc_empty = acc_full + 2;
    uint64_t *unit_bars = acc_empty + 2;
    Unit4 *sh_unit = reinterpret_cast<Unit4 *>(unit_bars + 2 * kUnitSlots);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sh_unit + kUnitSlots);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *sh_offs = reinterpret_cast<int *>(tmem_slot + 4), *sh_tiles = sh_offs + p.E + 1;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint64_t wl = p.wait_ns ? p.wait_ns : kWaitNs;
    UnitRing ring(sh_unit, unit_bars, abort_flag, wl);
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
            mbar_init(sc_full + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + i, 1);
            mbar_init(acc_empty + i, 8);  // every epilogue warp
        }
        ring.init(12);  // all warps but the one that finds the units
        *abort_flag = 0;
        fence_mbar_init();
        tc::prefetch_map(&map_w);
        tc::prefetch_map(&map_x);
    }
    if (warp == 1) tmem_alloc<1>(tmem_slot, T::tmem);
    // (only now: the set-up above overlaps the end of the kernel before. The kernel behind this one is not let in early:
    // its CTAs would come to SMs whose L1 is almost all shared memory here, and keep them so. A quantizer of 16384 x
    // 2048 values behind this kernel took 24 us instead of 15.)
    pdl_wait();
    const bool valid = build_tiles<1>(p.offs, p.E, p.P, BN, sh_offs, sh_tiles);
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = valid ? FT_OK : FT_ERR_INVALID_ROUTING;
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = uniform(*tmem_slot);

    const int m_tiles = (p.N + kTileM - 1) / kTileM;
    const int units = uniform(sh_tiles[p.E]) * m_tiles;
    const int split = p.split, part = (int)(blockIdx.x % split);
    const int nstages = (p.K + kStep4 - 1) / kStep4, kt = (p.K + 127) / 128;
    const int b0 = nstages * part / split, nb = nstages * (part + 1) / split;  // this CTA's stages
    const int u0 = blockIdx.x / split, du = gridDim.x / split;
    auto unit_of = [&](int u) {
        const int t = u / m_tiles;
        const Tile x = tile_of(t, expert_of(t, p.E, sh_tiles), BN, 16, sh_offs, sh_tiles);
        Unit4 r = {};
        r.e = x.e;
        r.n0 = (u - t * m_tiles) * kTileM;
        r.row0 = x.row0;
        r.lo = 0;
        r.hi = x.rows;
        r.cols = (x.rows + 15) / 16 * 16;
        return r;
    };
    bool dead = false;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (!p.skip_producer) {
            const bool one = elect_one();
            int s = 0, it = 0;
            uint32_t ph = 1;
            bool ready = false;
            for (Unit4 x; !dead && ring.get(x, dead);) {
                const int boxes = (x.cols + T::box_rows - 1) / T::box_rows;
                const uint8_t *ws = p.ws + ((int64_t)x.e * m_tiles + x.n0 / kTileM) * kt * kTileBytes;
                for (int b = b0; b < nb; ++b, ++it) {
                    if (!ready && !warp_wait(empty + s, ph, abort_flag, wl)) { dead = true; break; }
                    unsigned char *sa = smem + s * T::stage, *sb = sa + kABytes;
                    const uint32_t bar = smem_u32(full + s);
                    const uint32_t sf = min(kt - 2 * b, 2) * kTileBytes;  // (the last stage may have one word a row)
                    if (one) {
                        mbar_arrive_expect_tx(full + s, kABytes + boxes * T::box_rows * kChunkBytes + sf);
                        load_3d<1>(sa, &map_w, b * kChunkBytes, x.n0, x.e, bar);
                        bulk_g2s(sb + T::b_bytes, ws + 2 * b * kTileBytes, sf, full + s);
                        for (int i = 0; i < boxes; ++i)
                            load_2d<1>(sb + i * T::box_rows * kChunkBytes, &map_x, b * kChunkBytes, x.row0 + i * T::box_rows, bar);
                    }
                    if (++s == S) { s = 0; ph ^= 1; }
                    ready = __all_sync(0xFFFFFFFFu, test_cluster(empty + s, ph));
                }
            }
            if (dead && lane == 0) { raise_status(p.status, FT_ERR_TIMEOUT); *abort_flag = 1; }
            if (dead)  // every issued copy lands before the exit
                for (int i = 0; i < S && i < it; ++i) {
                    const int last = it - 1 - i;
                    mbar_wait_timed(full + last % S, (last / S) & 1, nullptr, wl);
                }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        // (The next stage's barriers are looked at before this stage's instructions are issued, and a whole stage's have
        // no conditions: see the wide tiles below.)
        const bool one = elect_one();
        const uint32_t base = smem_u32(smem);
        const uint64_t a0 = tc::sw128_desc(base), bd0 = tc::sw128_desc(base + kABytes), f0 = scale_desc(base + kABytes + T::b_bytes);
        const int whole = p.K / kStep4;  // stages with four instructions
        int s = 0, ac = 0;
        uint32_t ph = 0, sfa = tmem + T::sf_col;
        bool ready = false;
        Unit4 x = {};
        uint32_t idesc[2] = {};
        auto stage = [&](int b, bool end) {
            const int in_part = F32 ? (b - b0) % kPart4 : b - b0;
            const bool first = in_part == 0, last = end || (F32 && in_part == kPart4 - 1);
            if ((first && !warp_wait(acc_empty + (ac & 1), ((ac >> 1) & 1) ^ 1, abort_flag, wl)) ||
                (!ready && (!warp_wait(full + s, ph, abort_flag, wl) || !warp_wait(sc_full + s, ph, abort_flag, wl)))) {
                dead = true;
                return;
            }
            tc::fence_after_sync();
            const uint32_t at = (uint32_t)s * (T::stage / 16);
            const uint64_t ad = a0 + at, bd = bd0 + at, sd = f0 + at;
            const uint32_t d = tmem + (uint32_t)(ac & 1) * BN, sfb = sfa + 8;
            uint64_t *done = empty + s;
            if (++s == S) { s = 0; ph ^= 1; }
            const bool seen = test_cluster(full + s, ph) && test_cluster(sc_full + s, ph);
            if (b < whole) {
                if (one) {
                    copy_scales<1>(sfa, sd);
                    copy_scales<1>(sfb, sd + T::sf_bytes / 16);
                    copy_scales<1>(sfa + 4, sd + kTileBytes / 16);
                    copy_scales<1>(sfb + 4, sd + (T::sf_bytes + kTileBytes) / 16);
                    mma_mxf4<1>(d, ad, bd, idesc[0], sfa, sfb, !first);
#pragma unroll
                    for (int j = 1; j < 4; ++j)
                        mma_mxf4<1>(d, ad + 2 * j, bd + 2 * j, idesc[j & 1], sfa + 4 * (j >> 1), sfb + 4 * (j >> 1), 1);
                    commit<1>(done);
                    if (last) commit<1>(acc_full + (ac & 1));
                }
            } else if (one) {
                const int steps = (p.K - b * kStep4 + 63) / 64;  // instructions that have something to multiply
                copy_scales<1>(sfa, sd);
                copy_scales<1>(sfb, sd + T::sf_bytes / 16);
                if (steps > 2) {
                    copy_scales<1>(sfa + 4, sd + kTileBytes / 16);
                    copy_scales<1>(sfb + 4, sd + (T::sf_bytes + kTileBytes) / 16);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < steps)
                        mma_mxf4<1>(d, ad + 2 * j, bd + 2 * j, idesc[j & 1], sfa + 4 * (j >> 1), sfb + 4 * (j >> 1), !first || j != 0);
                commit<1>(done);
                if (last) commit<1>(acc_full + (ac & 1));
            }
            __syncwarp();
            ready = __all_sync(0xFFFFFFFFu, seen);
            sfa ^= (tmem + T::sf_col) ^ (tmem + T::sf_col + 16);
            if (last) ++ac;
        };
        bool more = ring.get(x, dead);
        while (more && !dead) {
            idesc[0] = idesc_mxf4(kTileM, x.cols, 0);
            idesc[1] = idesc_mxf4(kTileM, x.cols, 1);
            for (int b = b0; b + 1 < nb && !dead; ++b) stage(b, false);
            if (!dead) more = ring.get(x, dead);
            if (!dead) stage(nb - 1, true);
        }
        if (dead && lane == 0) { raise_status(p.status, FT_ERR_TIMEOUT); *abort_flag = 1; }
    } else if (warp < 4) {
        // ------------------------------------------------------------ scales of x
        // The two warps take groups of stages in turn, a group's words loaded together. Column c of the tile goes to
        // word c / 32 of lane c % 32; columns beyond the tile's rows get zeros (their sums are not stored).
        constexpr int G = T::group, C = BN / 32;
        int g = 0, it = 0;  // groups and stages so far, over all units
        for (Unit4 x; !dead && ring.get(x, dead);) {
            const uint32_t *xr = p.xs + x.row0;
            for (int b = b0; b < nb; b += G, ++g) {
                const int len = min(G, nb - b);
                if ((g & 1) == warp - 2) {
                    uint32_t v[G][2][C];
#pragma unroll
                    for (int i = 0; i < G; ++i)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int c = 0; c < C; ++c) {
                                const int at = 2 * (b + i) + k;
                                v[i][k][c] = at < kt && 32 * c + lane < x.hi ? __ldg(xr + at * p.ld_xs + 32 * c + lane) : 0u;
                            }
#pragma unroll
                    for (int i = 0; i < G; ++i) {
                        if (i >= len || dead) break;
                        const int s = (it + i) % S;
                        if (!warp_wait(empty + s, (((it + i) / S) & 1) ^ 1, abort_flag, wl)) { dead = true; break; }
                        unsigned char *to = smem + s * T::stage + kABytes + T::b_bytes + T::sf_bytes + 16 * lane;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            if constexpr (C == 4)
                                *reinterpret_cast<uint4 *>(to + k * kTileBytes) =
                                    make_uint4(v[i][k][0], v[i][k][1], v[i][k][2], v[i][k][3]);
                            else *reinterpret_cast<uint32_t *>(to + k * kTileBytes) = v[i][k][0];
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(sc_full + s);
                    }
                    if (dead) break;
                }
                it += len;
            }
        }
        if (dead && lane == 0) { raise_status(p.status, FT_ERR_TIMEOUT); *abort_flag = 1; }
    } else if (warp < 12) {
        // ------------------------------------------------------------ epilogue
        // thread = TMEM lane = weight row; columns [h * HC, h * HC + HC) of the tile
        const int q = warp & 3, h = (warp - 4) >> 2;
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * q) << 16) + h * HC;
        int ac = 0;
        const int parts = F32 ? (nb - b0 + kPart4 - 1) / kPart4 : 1;
        for (Unit4 x; !dead && ring.get(x, dead);) {
            const int mine = min(max(x.hi - h * HC, 0), HC);  // columns of this half in use
            const int m = x.n0 + 32 * q + lane;
            const int64_t row0 = x.row0 + h * HC;
            auto emit = [&](int c, const float (&v)[W]) {
                if (split > 1) {
                    // (every stage of the ring has been read by the time the last sums are complete)
                    float *red = reinterpret_cast<float *>(smem);
#pragma unroll
                    for (int j = 0; j < W; ++j) red[(h * HC + c + j) * kTileM + 32 * q + lane] = v[j];
                } else if (F32 || p.pairs) {
                    store_rows<F32, W>(v, m, p.N, row0 + c, mine - c, p.out, p.ld);
                } else {
                    store_rows<F32, W, false>(v, m, p.N, row0 + c, mine - c, p.out, p.ld);
                }
            };
            float sum[F32 ? HC : 1];  // the parts' running sums
            for (int t = 0; t < parts; ++t, ++ac) {
                if (!warp_wait(acc_full + (ac & 1), (ac >> 1) & 1, abort_flag, wl)) { dead = true; break; }
                tc::fence_after_sync();
                const uint32_t addr = lane_addr + (uint32_t)(ac & 1) * BN;
#pragma unroll
                for (int c = 0; c < HC; c += W) {
                    if (c >= mine) break;
                    uint32_t v[W];
                    tmem_ld<W>(addr + c, v);
                    tc::wait_ld();
                    if constexpr (F32) {
#pragma unroll
                        for (int j = 0; j < W; ++j) sum[c + j] = t ? sum[c + j] + __uint_as_float(v[j]) : __uint_as_float(v[j]);
                    } else {
                        float f[W];
#pragma unroll
                        for (int j = 0; j < W; ++j) f[j] = __uint_as_float(v[j]);
                        emit(c, f);
                    }
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(acc_empty + (ac & 1));
            }
            if (dead) break;
            if constexpr (F32) {
#pragma unroll
                for (int c = 0; c < HC; c += W) {
                    if (c >= mine) break;
                    float f[W];
#pragma unroll
                    for (int j = 0; j < W; ++j) f[j] = sum[c + j];
                    emit(c, f);
                }
            }
        }
        if (dead && lane == 0) { raise_status(p.status, FT_ERR_TIMEOUT); *abort_flag = 1; }
    } else {
        // ------------------------------------------------------------ units
        Unit4 x = {};
        for (int u = u0; u < units && !dead; u += du) {
            x = unit_of(u);
            dead = !ring.put(x);
        }
        x.e = -1;
        if (!dead) dead = !ring.put(x);
        if (dead && lane == 0) { raise_status(p.status, FT_ERR_TIMEOUT); *abort_flag = 1; }
    }

    // wind down; a cluster leaves together
    tc::fence_before_sync();
    __syncthreads();
    if (split > 1) {  // one unit per cluster: add its CTAs' sums, always in the same order
        cluster_sync();
        if (u0 < units) {
            const Unit4 x = unit_of(u0);
            add_parts<F32>(reinterpret_cast<const float *>(smem), x.hi, x.n0, p.N, x.row0, p.out, p.ld, split, part);
        }
        cluster_sync();
    }
    tc::fence_after_sync();
    if (warp == 1) tmem_dealloc<1>(tmem, T::tmem);
}

// ---------------------------------------------------------------- many rows per expert
//
// The rows along the M axis (thread = lane = row) and the weight rows along N, by pairs of CTAs: 256 rows x 192
// columns, each CTA its own 128 rows and half of the shared weight tile (both CTAs' scales of the weights are whole).
// Everything comes by TMA, the scales too, so that no warp stands between memory and the tensor cores. For that
// the rows' scale words must lie in shared memory in tensor memory's order as they come: lane r of 32 takes four
// neighbouring words, of rows 4 r .. 4 r + 3, for the MMA's rows r, 32 + r, 64 + r and 96 + r. So row 4 r + j of the tile is
// the MMA's row 32 j + r: one box fetches the codes in that order from x seen as [4][P / 4] rows (the tile that holds
// the last P % 4 rows takes four boxes of every fourth row instead), and a tile begins at a multiple of four rows, at
// most three before its expert's first one (neither those nor the rows behind the expert's last are stored). Tensor memory holds two accumulators of 192 columns and two stages' scales; 256
// columns would fill it with the accumulators alone.

namespace {

struct RingP {
    static constexpr int BN = 192, half = BN / 2;
    static constexpr int b_bytes = half * kChunkBytes;
    static constexpr int a_sf = 2 * kTileBytes, b_sf = 4 * kTileBytes;  // [steps of 128], [tile][steps of 128]
    static constexpr int stage = kABytes + b_bytes + a_sf + b_sf;
    static constexpr int stages = 6;
    static constexpr int groups = BN / 64;           // epilogue: four warps for each 64 columns
    static constexpr int warps = 4 * groups;
    static constexpr int threads = 128 + 32 * warps;
    static constexpr int out = warps * 16 * 128;     // 16 rows x 128 bytes per warp, on their way out
    static constexpr int sf_col = 2 * BN, sf_cols = 24;
    static_assert(stage % 1024 == 0 && sf_col + 2 * sf_cols <= 512, "layout");
};

}  // namespace

template <bool F32>
__global__ void __launch_bounds__(RingP::threads, 1)
    group_gemm_mxfp4_wide_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                                 const __grid_constant__ CUtensorMap map_x_end, const __grid_constant__ CUtensorMap map_ws,
                                 const __grid_constant__ CUtensorMap map_xs, const __grid_constant__ Group4Params p)
{
    using T = RingP;
    constexpr int S = T::stages, BN = T::BN;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char *sh_out = smem + S * T::stage;
    uint64_t *full = reinterpret_cast<uint64_t *>(sh_out + T::out);
    uint64_t *empty = full + S, *acc_full = empty + S, *acc_empty = acc_full + 2;
    uint64_t *unit_bars = acc_empty + 2;
    Unit4 *sh_unit = reinterpret_cast<Unit4 *>(unit_bars + 2 * kUnitSlots);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sh_unit + kUnitSlots);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *sh_offs = reinterpret_cast<int *>(tmem_slot + 4), *sh_tiles = sh_offs + p.E + 1;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const bool leader = rank == 0;
    const uint64_t wl = p.wait_ns ? p.wait_ns : kWaitNs;
    UnitRing ring(sh_unit, unit_bars, abort_flag, wl);
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + i, 1);
            mbar_init(acc_empty + i, 2 * T::warps);  // the epilogue warps of both CTAs
        }
        ring.init(T::warps + 1 + (int)leader);  // the producer and the epilogue, in the leader the MMA issuer
        *abort_flag = 0;
        fence_mbar_init();
        tc::prefetch_map(&map_w);
        tc::prefetch_map(&map_x);
        tc::prefetch_map(&map_x_end);
        tc::prefetch_map(&map_ws);
        tc::prefetch_map(&map_xs);
    }
    if (warp == 1) tmem_alloc<2>(tmem_slot, 512);
    // (only now: the set-up above overlaps the end of the kernel before. The kernel behind this one is not let in early:
    // its CTAs would come to SMs whose L1 is almost all shared memory here, and keep them so. A quantizer of 65536 x
    // 2048 values behind this kernel took 85 us instead of 57.)
    pdl_wait();
    const bool valid = build_tiles<4>(p.offs, p.E, p.P, 2 * kTileM, sh_offs, sh_tiles);
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = valid ? FT_OK : FT_ERR_INVALID_ROUTING;
    tc::fence_before_sync();
    cluster_sync();
    tc::fence_after_sync();
    const uint32_t tmem = uniform(*tmem_slot);

    // columns are dealt out in 64s: as many to every tile, or one more
    const int n_tiles = (p.N + BN - 1) / BN, n64 = (p.N + 63) / 64;
    const int units = uniform(sh_tiles[p.E]) * n_tiles;
    const int nb = (p.K + kStep4 - 1) / kStep4, nt128 = (p.N + 127) / 128;
    const int u0 = blockIdx.x / 2, du = gridDim.x / 2;
    auto unit_of = [&](int u) {
        const int t = u / n_tiles, j = u - t * n_tiles;
        const AlignedTile x = find_aligned_tile<4>(t, p.E, 2 * kTileM, sh_offs, sh_tiles);
        Unit4 r = {};
        r.e = x.e;
        r.row0 = x.row0;
        r.lo = x.lo;
        r.hi = x.hi;
        r.n0 = n64 * j / n_tiles * 64;
        r.width = min(n64 * (j + 1) / n_tiles * 64, p.N) - r.n0;
        r.cols = (r.width + 31) / 32 * 32;
        return r;
    };
    bool dead = false;

    if (warp < 4) {
        if (warp == 0 && !p.skip_producer) {
            // -------------------------------------------------------- producer
            const bool one = elect_one();
            const uint32_t full0 = map_rank(full, 0);
            int s = 0, it = 0;
            uint32_t ph = 1;
            bool ready = false;
            for (Unit4 x; !dead && ring.get(x, dead);) {
                const int mine = x.hi - (int)rank * kTileM;  // rows of this CTA, if positive
                const uint32_t bytes = 2 * (T::b_bytes + T::b_sf) + (x.hi > kTileM ? 2 : 1) * (kABytes + T::a_sf);
                const int ws_tile = x.e * nt128 + x.n0 / 128, row = x.row0 + (int)rank * kTileM, n0 = x.n0 + (int)rank * (x.cols / 2);
                const bool whole = row + kTileM <= p.P / 4 * 4 || p.P % 4 == 0;
                for (int b = 0; b < nb; ++b, ++it) {
                    if (!ready && !warp_wait(empty + s, ph, abort_flag, wl)) { dead = true; break; }
                    unsigned char *sa = smem + s * T::stage, *sb = sa + kABytes, *sf = sb + T::b_bytes;
                    const uint32_t bar = full0 + 8 * s;
                    if (one) {
                        if (leader) mbar_arrive_expect_tx(full + s, bytes);
                        load_3d<2>(sb, &map_w, b * kChunkBytes, n0, x.e, bar);
                        if (mine > 0) {
                            if (whole) load_3d<2>(sa, &map_x, b * kChunkBytes, row / 4, 0, bar);
                            else
                                for (int j = 0; j < 4; ++j) load_2d<2>(sa + j * 32 * kChunkBytes, &map_x_end, b * kChunkBytes, row + j, bar);
                            load_2d<2>(sf, &map_xs, row, 2 * b, bar);
                        }
                        load_3d<2>(sf + T::a_sf, &map_ws, 0, 2 * b, ws_tile, bar);
                    }
                    if (++s == S) { s = 0; ph ^= 1; }
                    ready = __all_sync(0xFFFFFFFFu, test_cluster(empty + s, ph));
                }
            }
            // The last stages' MMAs also arrive in the other CTA: neither leaves before all have.
            for (int i = 0; i < S && !dead; ++i) {
                if (!warp_wait(empty + s, ph, abort_flag, wl)) dead = true;
                if (++s == S) { s = 0; ph ^= 1; }
            }
            if (dead && lane == 0) { raise_status(p.status, FT_ERR_TIMEOUT); *abort_flag = 1; }
            if (dead && leader)  // every issued copy lands before the exit
                for (int i = 0; i < S && i < it; ++i) {
                    const int last = it - 1 - i;
                    mbar_wait_timed(full + last % S, (last / S) & 1, nullptr, wl);
                }
        } else if (warp == 1 && leader) {
            // -------------------------------------------------------- MMA issuer
            // A stage takes the tensor cores 500 cycles, and this loop must not take longer: the next stage's barrier is
            // looked at before this stage's instructions are issued, and a whole stage's have no conditions.
            const bool one = elect_one();
            const uint32_t base = smem_u32(smem);
            const uint64_t a0 = tc::sw128_desc(base), b0 = tc::sw128_desc(base + kABytes);
            const uint64_t f0 = scale_desc(base + kABytes + T::b_bytes);  // the rows' scales, then the weights'
            const int whole = p.K / kStep4;                               // stages with four instructions
            int s = 0, ac = 0;
            uint32_t ph = 0, sf = tmem + T::sf_col;
            bool ready = false;
            Unit4 x = {};
            uint32_t idesc[2] = {}, col0 = 0;
            bool two = false;
            auto enter = [&]() {
                idesc[0] = idesc_mxf4(2 * kTileM, x.cols, 0);
                idesc[1] = idesc_mxf4(2 * kTileM, x.cols, 1);
                two = x.n0 % 128 + x.cols > 128;
                col0 = 4 + x.n0 % 128 / 32;  // of the unit's first weight row in its tile's scales
            };
            auto stage = [&](int b, bool end) {
                const int in_part = F32 ? b % kPart4 : b;
                const bool first = in_part == 0, last = end || (F32 && in_part == kPart4 - 1);
                if ((first && !warp_wait(acc_empty + (ac & 1), ((ac >> 1) & 1) ^ 1, abort_flag, wl)) ||
                    (!ready && !warp_wait(full + s, ph, abort_flag, wl))) {
                    dead = true;
                    return;
                }
                tc::fence_after_sync();
                const uint32_t at = (uint32_t)s * (T::stage / 16);
                const uint64_t ad = a0 + at, bd = b0 + at, xs = f0 + at, ws = xs + T::a_sf / 16;
                const uint32_t d = tmem + (uint32_t)(ac & 1) * BN;
                uint64_t *done = empty + s;
                if (++s == S) { s = 0; ph ^= 1; }
                const bool seen = test_cluster(full + s, ph);
                // columns: four of the rows' scales, eight of the weights', for each 128 steps
                if (b < whole) {
                    if (one) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            copy_scales<2>(sf + 12 * k, xs + k * (kTileBytes / 16));
                            copy_scales<2>(sf + 12 * k + 4, ws + k * (kTileBytes / 16));
                            if (two) copy_scales<2>(sf + 12 * k + 8, ws + (2 + k) * (kTileBytes / 16));
                        }
                        mma_mxf4<2>(d, ad, bd, idesc[0], sf, sf + col0, !first);
#pragma unroll
                        for (int j = 1; j < 4; ++j)
                            mma_mxf4<2>(d, ad + 2 * j, bd + 2 * j, idesc[j & 1], sf + 12 * (j >> 1), sf + 12 * (j >> 1) + col0, 1);
                        commit<2>(done);
                        if (last) commit<2>(acc_full + (ac & 1));
                    }
                } else if (one) {
                    const int steps = (p.K - b * kStep4 + 63) / 64;  // instructions that have something to multiply
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (2 * k < steps) {
                            copy_scales<2>(sf + 12 * k, xs + k * (kTileBytes / 16));
                            copy_scales<2>(sf + 12 * k + 4, ws + k * (kTileBytes / 16));
                            if (two) copy_scales<2>(sf + 12 * k + 8, ws + (2 + k) * (kTileBytes / 16));
                        }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < steps)
                            mma_mxf4<2>(d, ad + 2 * j, bd + 2 * j, idesc[j & 1], sf + 12 * (j >> 1), sf + 12 * (j >> 1) + col0,
                                        !first || j != 0);
                    commit<2>(done);
                    if (last) commit<2>(acc_full + (ac & 1));
                }
                __syncwarp();
                ready = __all_sync(0xFFFFFFFFu, seen);
                sf ^= (tmem + T::sf_col) ^ (tmem + T::sf_col + T::sf_cols);
                if (last) ++ac;
            };
            bool more = ring.get(x, dead);
            while (more && !dead) {
                enter();
                for (int b = 0; b + 1 < nb && !dead; ++b) stage(b, false);
                // (before the last stage, so that there is nothing to look up between two units)
                if (!dead) more = ring.get(x, dead);
                if (!dead) stage(nb - 1, true);
            }
            if (dead && lane == 0) { raise_status(p.status, FT_ERR_TIMEOUT); *abort_flag = 1; }
        } else if (warp == 2) {
            // -------------------------------------------------------- units
            Unit4 x = {};
            for (int u = u0; u < units && !dead; u += du) {
                x = unit_of(u);
                dead = !ring.put(x);
            }
            x.e = -1;
            if (!dead) dead = !ring.put(x);
            if (dead && lane == 0) { raise_status(p.status, FT_ERR_TIMEOUT); *abort_flag = 1; }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        // the warp takes 64 columns of the rows 4 l + q (lane l of its quarter q)
        const int q = warp & 3, g = (warp - 4) >> 2;
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * q) << 16) + 64 * g;
        const uint32_t empty_bar = map_rank(acc_empty, 0);
        unsigned char *tile = sh_out + (warp - 4) * 16 * 128;
        const int parts = F32 ? (nb + kPart4 - 1) / kPart4 : 1;
        int ac = 0;
        for (Unit4 x; !dead && ring.get(x, dead);) {
            float sum[64];
            for (int t = 0; t < parts; ++t, ++ac) {
                if (!warp_wait(acc_full + (ac & 1), (ac >> 1) & 1, abort_flag, wl)) { dead = true; break; }
                tc::fence_after_sync();
                const uint32_t addr = lane_addr + (uint32_t)(ac & 1) * BN;
#pragma unroll
                for (int c = 0; c < 64; c += 32) {
                    uint32_t v[32];
                    tc::ld32(addr + c, v);
                    tc::wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) sum[c + i] = F32 && t ? sum[c + i] + __uint_as_float(v[i]) : __uint_as_float(v[i]);
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) arrive_cluster_relaxed(empty_bar + 8 * (ac & 1));
            }
            if (dead) break;
            // 128 bytes of each row at a time through shared memory (16-byte pieces swizzled by the row, free of bank
            // conflicts), so that a store instruction writes whole lines of four rows; rows that are not made of
            // 16-byte pieces leave a row at a time, an element a lane
            constexpr int per = F32 ? 32 : 64;
            const int n0 = x.n0 + 64 * g, mine = min(max(x.width - 64 * g, 0), 64);
            const int first = (int)rank * kTileM + q;  // of the warp's rows, four apart
            const int64_t at = (int64_t)x.row0 * p.ld + n0;
            const int l8 = lane & 7, r4 = lane >> 3;
#pragma unroll
            for (int c = 0; c < 64; c += per) {
                if (c >= mine) break;
                uint4 o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if constexpr (F32) {
                        const float *f = sum + c + 4 * i;
                        o[i] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
                    } else {
                        const float *f = sum + 8 * i;
                        o[i] = make_uint4(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]), bf16x2(f[4], f[5]), bf16x2(f[6], f[7]));
                    }
                }
                const int col = c + l8 * (per / 8);
#pragma unroll
                for (int h = 0; h < 2; ++h) {  // 16 rows at a time
                    __syncwarp();
                    if (lane >> 4 == h) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<uint4 *>(tile + (lane & 15) * 128 + ((i ^ l8) << 4)) = o[i];
                    }
                    __syncwarp();
                    if (p.vec) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = 4 * i + r4, row = first + 4 * (16 * h + r);
                            const uint4 w = *reinterpret_cast<const uint4 *>(tile + r * 128 + ((l8 ^ (r & 7)) << 4));
                            if (row >= x.lo && row < x.hi && col < mine)
                                *reinterpret_cast<uint4 *>(static_cast<char *>(p.out) + (at + row * p.ld + col) * (F32 ? 4 : 2)) = w;
                        }
                    } else {
                        using O = std::conditional_t<F32, uint32_t, uint16_t>;
                        constexpr int each = 16 / (int)sizeof(O);
#pragma unroll 4
                        for (int r = 0; r < 16; ++r) {
                            const int row = first + 4 * (16 * h + r);
#pragma unroll
                            for (int i = lane; i < per; i += 32)
                                if (row >= x.lo && row < x.hi && c + i < mine)
                                    static_cast<O *>(p.out)[at + row * p.ld + c + i] =
                                        reinterpret_cast<const O *>(tile + r * 128 + (((i / each) ^ (r & 7)) << 4))[i % each];
                        }
                    }
                }
            }
            __syncwarp();
        }
        if (dead && lane == 0) { raise_status(p.status, FT_ERR_TIMEOUT); *abort_flag = 1; }
    }

    // wind down; a cluster leaves together
    tc::fence_before_sync();
    __syncthreads();
    cluster_sync();
    tc::fence_after_sync();
    if (warp == 1) tmem_dealloc<2>(tmem, 512);
}

namespace {

template <int BN, bool F32>
cudaError_t launch4(const CUtensorMap &w, const CUtensorMap &x, Group4Params &p, int32_t *plan, cudaStream_t s)
{
    using T = Ring4<BN>;
    auto kern = group_gemm_mxfp4_kernel<BN, F32>;
    constexpr size_t fixed = 1024 + T::stages * T::stage + 8 * (3 * T::stages + 4 + 2 * kUnitSlots) + kUnitSlots * sizeof(Unit4) + 16;
    constexpr size_t most = fixed + table_bytes(kGroupMaxExperts);
    static_assert(most <= 227 * 1024, "shared memory");
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess) return e;
    const int64_t m_tiles = (p.N + kTileM - 1) / kTileM;
    const int64_t units = m_tiles * (p.P / BN + (p.E < p.P ? p.E : p.P));  // at most
    static ClusterLimit clusters;
    // Few units: the CTAs of a cluster share one unit's contraction, at least two stages each, as
    // long as all clusters run at once.
    p.split = 1;
    while (p.split < 8 && p.K >= 4 * kStep4 * p.split && units <= clusters.get(kern, 2 * p.split, kThreads4, most)) p.split *= 2;
    if (plan) {
        write_plan(plan, 1, BN, p.split, false);
        return cudaSuccess;
    }
    int64_t grid = p.split > 1 ? units : sm_count();
    if (units < grid) grid = units;
    if (grid < 1) grid = 1;
    const cudaError_t le = launch_cluster(kern, dim3((unsigned)grid * p.split), dim3(kThreads4), fixed + table_bytes(p.E), p.split, s, w,
                                          x, p);
    if (le != cudaSuccess) return le;
    count_launches(1);
    return cudaGetLastError();
}

template <bool F32>
cudaError_t launch_wide4(const CUtensorMap &w, const CUtensorMap &x, const CUtensorMap &x_end, const CUtensorMap &ws,
                         const CUtensorMap &xs, const Group4Params &p, cudaStream_t s)
{
    using T = RingP;
    auto kern = group_gemm_mxfp4_wide_kernel<F32>;
    constexpr size_t fixed = 1024 + T::stages * T::stage + T::out + 8 * (2 * T::stages + 4 + 2 * kUnitSlots) + kUnitSlots * sizeof(Unit4) + 16;
    constexpr size_t most = fixed + table_bytes(kGroupMaxExperts);
    static_assert(most <= 227 * 1024, "shared memory");
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)((p.N + T::BN - 1) / T::BN) * (p.P / (2 * kTileM) + 2 * (p.E < p.P ? p.E : p.P));  // at most
    static ClusterLimit clusters;
    int64_t grid = clusters.get(kern, 2, T::threads, most);
    if (units < grid) grid = units;
    const cudaError_t le = launch_cluster(kern, dim3((unsigned)grid * 2), dim3(T::threads), fixed + table_bytes(p.E), 2, s, w, x,
                                          x_end, ws, xs, p);
    if (le != cudaSuccess) return le;
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_group_gemm_mxfp4(const GroupGemm4 &g, cudaStream_t s)
{
    Group4Params p = {};
    p.offs = g.offs;
    p.E = g.E;
    p.P = g.P;
    p.N = g.N;
    p.K = g.K;
    p.xs = g.xs;
    p.ld_xs = g.ld_xs;
    p.ws = g.ws;
    p.out = g.out;
    p.ld = g.ld_out;
    p.pairs = g.N % 2 == 0 && g.ld_out % 2 == 0;
    p.vec = g.N % (g.out_f32 ? 4 : 8) == 0 && g.ld_out % (g.out_f32 ? 4 : 8) == 0;
    p.status = g.status;
    injected_stall(&p.wait_ns, &p.skip_producer);
    // The tile, by the rows per expert that has any. Measured on 256 experts of 1024 x 2048 (us, with 32 or 128 rows
    // along N / 256 rows along M): 16 rows 50 / 50 / 57, 32 rows 51 / 52 / 59, 96 rows 92 / 59 / 64, 128 rows 118 / 65 /
    // 67, 160 rows 142 / 78 / 70, 256 rows 217 / 96 / 92. The wide tiles need two and a half rounds of units to be the
    // better ones (one expert, 4096 rows: of 1024 x 4096, 102 units, 13.9 / 15.2; 2048 rows of 4096 x 4096, 198 units,
    // 23.5 / 20.3), and small tiles are as long as they all run at once (one expert of 2048 x 2048: 256 rows 6.4 / 9.0 /
    // 7.7).
    const int64_t touched = g.E < g.P ? g.E : g.P, per = g.P / touched;
    const int64_t small = (int64_t)((g.N + kTileM - 1) / kTileM) * (g.P / 32 + touched);
    const int64_t pairs = (int64_t)((g.N + RingP::BN - 1) / RingP::BN) * (g.P / 256 + touched);
    const int bn = per <= 24 || small <= sm_count() ? 32 : per < 144 || 4 * pairs < 5 * sm_count() ? 128 : 256;
    if (g.plan && bn == 256) {
        write_plan(g.plan, 2, bn, 1, false);
        return cudaSuccess;
    }
    CUtensorMap w, x, x_end, ws, xs;
    const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8, u32 = CU_TENSOR_MAP_DATA_TYPE_UINT32;
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B, none = CU_TENSOR_MAP_SWIZZLE_NONE;
    const uint64_t bytes = g.K / 2, kt = (g.K + 127) / 128, nt = (g.N + 127) / 128;
    bool ok = true;
    if (g.plan) {  // nothing to read
    } else if (bn == 256) {
        ok = make_tensor_map_3d(&w, u8, g.w, bytes, g.N, g.E, bytes, bytes * g.N, kChunkBytes, RingP::half, sw) &&
             make_tensor_map_3d(&x, u8, g.x, bytes, g.P / 4, 4, 4 * g.ld_x, g.ld_x, kChunkBytes, 32, sw, 4) &&
             make_tensor_map_2d(&x_end, u8, g.x, bytes, g.P, g.ld_x, kChunkBytes, 32, sw, 4) &&
             make_tensor_map_3d(&ws, u32, g.ws, 128, kt, g.E * nt, kTileBytes, kTileBytes * kt, 128, 2, none, 2) &&
             make_tensor_map_2d(&xs, u32, g.xs, g.P, kt, 4 * g.ld_xs, 128, 2, none);
    } else {
        ok = make_tensor_map_3d(&w, u8, g.w, bytes, g.N, g.E, bytes, bytes * g.N, kChunkBytes, kTileM, sw) &&
             make_tensor_map_2d(&x, u8, g.x, bytes, g.P, g.ld_x, kChunkBytes, bn == 32 ? Ring4<32>::box_rows : Ring4<128>::box_rows, sw);
    }
    if (!ok) return cudaErrorInvalidValue;
    if (bn == 32) return g.out_f32 ? launch4<32, true>(w, x, p, g.plan, s) : launch4<32, false>(w, x, p, g.plan, s);
    if (bn == 128) return g.out_f32 ? launch4<128, true>(w, x, p, g.plan, s) : launch4<128, false>(w, x, p, g.plan, s);
    return g.out_f32 ? launch_wide4<true>(w, x, x_end, ws, xs, p, s) : launch_wide4<false>(w, x, x_end, ws, xs, p, s);
}

}  // namespace ftmoe
