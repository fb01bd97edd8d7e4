// Grouped products of 8-bit floating point (e4m3) operands with fp32 scales: x in blocks of 128
// along each row, w in blocks of 128 x 128. Expert e owns the rows [offs[e], offs[e + 1]):
//
//   y[p, n] = sum_b xs[b, p] * ws[e, n / 128, b] * (sum_{k in block b} x[p, k] * w[e, n, k])
//
// The inner sum of a block of 128 is one stage of tcgen05.mma (kind::f8f6f4) into a fresh
// tensor-memory buffer; the scales differ from block to block and are no powers of two, so the
// outer sum cannot be left to the tensor cores: eight warps read every block's partial sums and
// add them, times the two scales, to fp32 accumulators in registers (two columns per
// fma.rn.f32x2) while the tensor cores work on the next block.
//
// What bounds it, measured on one GB300:
//   - many rows: the way of each block's partial sums from the tensor cores through registers and
//     back. Dense 4864 x 4096 x 4096 takes 68 us, 2400 TFLOP/s; the MMAs alone took 42.
//   - few rows: the weights' one pass through memory. 64 tokens over 256 experts of 1024 x 2048 (0.47 GB)
//     take 75 us after 2 us for the quantizer, 6.2 TB/s.
//   - one row: latency. 1024 x 2048 takes 4.3 us after the quantizer, the contraction split over
//     clusters of eight CTAs.
#include <cuda_bf16.h>

#include <type_traits>

#include "group_gemm.cuh"

namespace ftmoe {

namespace {

using namespace grp;

constexpr int kThreads8 = 384;  // warps: 0 TMA, 1 MMA, 2-3 scales, 4..11 sums and epilogue
constexpr int kStep8 = 128;     // contraction steps per stage: one scale block

// Tiles of up to BN rows.
template <int BN>
struct Ring8 {
    static constexpr int b_bytes = BN * kChunkBytes;
    static constexpr int stage = kABytes + b_bytes;
    static constexpr int fit = 208 * 1024 / stage;
    static constexpr int stages = fit < 8 ? fit : 8;
    static constexpr int box_rows = BN <= 32 ? 16 : 32;
    static constexpr int acc = BN >= 128 ? 4 : 8;  // partial-sum buffers in tensor memory
    static constexpr int slots = 8;                  // scale slots in shared memory
};

struct Group8Params {
    const int *offs;
    int E, P, N, K;
    const float *xs;      // [ceil(K / 128)][ld_xs]
    int64_t ld_xs;
    const float *ws;      // [E][ceil(N / 128)][ceil(K / 128)]
    void *out;            // [P][ld]
    int64_t ld;
    int split;            // CTAs (one cluster) that share a unit's contraction
    int pairs;            // bf16 out: N even and rows 4-byte aligned
    int vec;              // N and the rows of out are multiples of 16 bytes
    int *status;
    uint64_t wait_ns;
    int skip_producer;
};

template <int CG>
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    if constexpr (CG == 1) {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    }
}

// (a.x, a.y) += (s0, s1) * (v0, v1), each one fp32 fused multiply-add.
__device__ __forceinline__ void fma2(float2 &a, float s0, float s1, uint32_t v0, uint32_t v1)
{
    asm("{\n\t.reg .b64 s, v, c;\n\tmov.b64 s, {%2, %3};\n\tmov.b64 v, {%4, %5};\n\tmov.b64 c, {%0, %1};\n\t"
        "fma.rn.f32x2 c, s, v, c;\n\tmov.b64 {%0, %1}, c;\n\t}"
        : "+f"(a.x), "+f"(a.y)
        : "f"(s0), "f"(s1), "r"(v0), "r"(v1));
}

// kind::f8f6f4 instruction descriptor: e4m3 operands (type fields 0), fp32 D.
__device__ __forceinline__ uint32_t idesc_e4m3(int M, int N)
{
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

struct Unit8 {
    int e, m0, row0, rows, cols;  // cols: rows in whole MMA columns
};

}  // namespace

template <int BN, bool F32>
__global__ void __launch_bounds__(kThreads8, 1)
    group_gemm_fp8_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                          const __grid_constant__ Group8Params p)
{
    using T = Ring8<BN>;
    constexpr int S = T::stages, NA = T::acc, NS = T::slots;
    constexpr int HC = BN / 2;  // columns of one half's warps
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float *sh_scale = reinterpret_cast<float *>(smem + S * T::stage);  // [NS][BN]
    uint64_t *full = reinterpret_cast<uint64_t *>(sh_scale + NS * BN);
    uint64_t *empty = full + S, *acc_full = empty + S, *acc_empty = acc_full + NA, *sc_full = acc_empty + NA,
             *sc_empty = sc_full + NS;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sc_empty + NS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *sh_flag = reinterpret_cast<int *>(tmem_slot + 2);
    int *sh_offs = reinterpret_cast<int *>(tmem_slot + 4), *sh_tiles = sh_offs + p.E + 1;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint64_t wl = p.wait_ns ? p.wait_ns : kWaitNs;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < NA; ++i) {
            mbar_init(acc_full + i, 1);
            mbar_init(acc_empty + i, 8);  // every sum warp
        }
        for (int i = 0; i < NS; ++i) {
            mbar_init(sc_full + i, 1);
            mbar_init(sc_empty + i, 8);
        }
        *abort_flag = 0;
        fence_mbar_init();
        tc::prefetch_map(&map_w);
        tc::prefetch_map(&map_x);
    }
    if (warp == 1) tmem_alloc<1>(tmem_slot, NA * BN);
    pdl_enter();  // (only now: the set-up above overlaps the end of the kernel before)
    const bool valid = build_table(p.offs, p.E, p.P, BN, sh_offs, sh_tiles, sh_flag);
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = valid ? FT_OK : FT_ERR_INVALID_ROUTING;
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = uniform(*tmem_slot);

    const int m_tiles = (p.N + kTileM - 1) / kTileM;
    const int units = uniform(sh_tiles[p.E]) * m_tiles;
    const int split = p.split, part = (int)(blockIdx.x % split);
    const int nblocks = (p.K + kStep8 - 1) / kStep8;
    const int b0 = nblocks * part / split, nb = nblocks * (part + 1) / split;  // this CTA's blocks
    const int u0 = blockIdx.x / split, du = gridDim.x / split;
    auto unit_of = [&](int u) {
        const int t = u / m_tiles;
        const Tile x = find_tile(t, p.E, BN, 16, sh_offs, sh_tiles);
        Unit8 r;
        r.e = x.e;
        r.m0 = (u - t * m_tiles) * kTileM;
        r.row0 = x.row0;
        r.rows = x.rows;
        r.cols = (x.rows + 15) / 16 * 16;
        return r;
    };
    auto uniform_unit = [](Unit8 x) {
        x.e = uniform(x.e); x.m0 = uniform(x.m0); x.row0 = uniform(x.row0); x.rows = uniform(x.rows); x.cols = uniform(x.cols);
        return x;
    };
    bool dead = false;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (!p.skip_producer) {
            const bool one = elect_one();
            int s = 0, it = 0;
            uint32_t ph = 1;
            for (int u = u0; u < units && !dead; u += du) {
                const Unit8 x = uniform_unit(unit_of(u));
                const int boxes = (x.cols + T::box_rows - 1) / T::box_rows;
                const uint32_t bytes = kABytes + boxes * T::box_rows * kChunkBytes;
                for (int b = b0; b < nb; ++b, ++it) {
                    if (!warp_wait(empty + s, ph, abort_flag, wl)) { dead = true; break; }
                    unsigned char *sa = smem + s * T::stage, *sb = sa + kABytes;
                    const uint32_t bar = smem_u32(full + s);
                    if (one) {
                        mbar_arrive_expect_tx(full + s, bytes);
                        load_3d<1>(sa, &map_w, b * kStep8, x.m0, x.e, bar);
                        for (int i = 0; i < boxes; ++i)
                            load_2d<1>(sb + i * T::box_rows * kChunkBytes, &map_x, b * kStep8, x.row0 + i * T::box_rows, bar);
                    }
                    __syncwarp();
                    if (++s == S) { s = 0; ph ^= 1; }
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
        const bool one = elect_one();
        int s = 0, a = 0;
        uint32_t ph = 0, pa = 1;
        for (int u = u0; u < units && !dead; u += du) {
            const Unit8 x = uniform_unit(unit_of(u));
            const uint32_t idesc = idesc_e4m3(kTileM, x.cols);
            for (int b = b0; b < nb; ++b) {
                if (!warp_wait(acc_empty + a, pa, abort_flag, wl) || !warp_wait(full + s, ph, abort_flag, wl)) {
                    dead = true;
                    break;
                }
                tc::fence_after_sync();
                const uint32_t sa = smem_u32(smem + s * T::stage);
                const uint64_t ad = tc::sw128_desc(sa), bd = tc::sw128_desc(sa + kABytes);
                if (one) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) mma_e4m3<1>(tmem + (uint32_t)a * BN, ad + 2 * j, bd + 2 * j, idesc, j != 0);
                    commit<1>(empty + s);
                    commit<1>(acc_full + a);
                }
                __syncwarp();
                if (++s == S) { s = 0; ph ^= 1; }
                if (++a == NA) { a = 0; pa ^= 1; }
            }
        }
        if (dead && lane == 0) { raise_status(p.status, FT_ERR_TIMEOUT); *abort_flag = 1; }
    } else if (warp < 4) {
        // ------------------------------------------------------------ scales
        // The two warps take the blocks in turn: slot c of block it = xs[b, row of c] * ws[e, tile, b]
        // (one rounding), zero beyond the tile's rows.
        const int n_blocks128 = (p.N + 127) / 128;
        int it = 0;  // blocks so far, over all units
        for (int u = u0; u < units && !dead; u += du) {
            const Unit8 x = unit_of(u);
            const int tile_m = min(x.m0 / 128, n_blocks128 - 1);
            const float *w = p.ws + ((int64_t)x.e * n_blocks128 + tile_m) * nblocks;
            const float *xr = p.xs + x.row0;
            for (int b = b0; b < nb; ++b, ++it) {
                if ((it & 1) != warp - 2) continue;
                float v[BN / 32];
                const float wb = __ldg(w + b);
#pragma unroll
                for (int i = 0; i < BN / 32; ++i) {
                    const int c = 32 * i + lane;
                    v[i] = c < x.rows ? __ldg(xr + (int64_t)b * p.ld_xs + c) : 0.f;
                }
                const int slot = it % NS;
                if (!warp_wait(sc_empty + slot, ((it / NS) & 1) ^ 1, abort_flag, wl)) { dead = true; break; }
#pragma unroll
                for (int i = 0; i < BN / 32; ++i) sh_scale[slot * BN + 32 * i + lane] = v[i] * wb;
                __syncwarp();
                if (lane == 0) mbar_arrive(sc_full + slot);
            }
        }
        if (dead && lane == 0) { raise_status(p.status, FT_ERR_TIMEOUT); *abort_flag = 1; }
    } else {
        // ------------------------------------------------------------ sums and epilogue
        // thread = TMEM lane = weight row; columns [h * HC, h * HC + HC) of the tile
        const int q = warp & 3, h = (warp - 4) >> 2;
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * q) << 16) + h * HC;
        int a = 0, it = 0;
        uint32_t pa = 0;
        for (int u = u0; u < units && !dead; u += du) {
            const Unit8 x = unit_of(u);
            float2 sum[HC / 2];
#pragma unroll
            for (int j = 0; j < HC / 2; ++j) sum[j] = make_float2(0.f, 0.f);
            const int mine = min(max(x.rows - h * HC, 0), HC);  // columns of this half in use
            for (int b = b0; b < nb; ++b, ++it) {
                const int slot = it % NS;
                if (!warp_wait(sc_full + slot, (it / NS) & 1, abort_flag, wl) ||
                    !warp_wait(acc_full + a, pa, abort_flag, wl)) {
                    dead = true;
                    break;
                }
                tc::fence_after_sync();
                const float *sc = sh_scale + slot * BN + h * HC;
#pragma unroll
                for (int c = 0; c < HC / 16; ++c) {
                    if (16 * c >= mine) break;
                    uint32_t v[16];
                    tc::ld16(lane_addr + (uint32_t)a * BN + 16 * c, v);
                    tc::wait_ld();
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 f = *reinterpret_cast<const float4 *>(sc + 16 * c + 4 * j);
                        fma2(sum[8 * c + 2 * j], f.x, f.y, v[4 * j], v[4 * j + 1]);
                        fma2(sum[8 * c + 2 * j + 1], f.z, f.w, v[4 * j + 2], v[4 * j + 3]);
                    }
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(acc_empty + a);
                    mbar_arrive(sc_empty + slot);
                }
                if (++a == NA) { a = 0; pa ^= 1; }
            }
            if (dead) break;
            const int m = x.m0 + 32 * q + lane;
            if (split > 1) {
                // (every stage of the ring has been read by the time the last sums are complete)
                float *red = reinterpret_cast<float *>(smem);
#pragma unroll
                for (int j = 0; j < HC; ++j) red[(h * HC + j) * kTileM + 32 * q + lane] = j & 1 ? sum[j / 2].y : sum[j / 2].x;
            } else {
#pragma unroll
                for (int c = 0; c < HC; c += 16) {
                    if (c >= mine) break;
                    float v[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = j & 1 ? sum[(c + j) / 2].y : sum[(c + j) / 2].x;
                    if (F32 || p.pairs) store_rows<F32, 16>(v, m, p.N, x.row0 + h * HC + c, mine - c, p.out, p.ld);
                    else store_rows<F32, 16, false>(v, m, p.N, x.row0 + h * HC + c, mine - c, p.out, p.ld);
                }
            }
            __syncwarp();
        }
        if (dead && lane == 0) { raise_status(p.status, FT_ERR_TIMEOUT); *abort_flag = 1; }
    }

    // wind down; a cluster leaves together
    tc::fence_before_sync();
    __syncthreads();
    if (split > 1) {
        cluster_sync();
        if (u0 < units) {
            const Unit8 x = unit_of(u0);
            add_parts<F32>(reinterpret_cast<const float *>(smem), x.rows, x.m0, p.N, x.row0, p.out, p.ld, split, part);
        }
        cluster_sync();
    }
    tc::fence_after_sync();
    if (warp == 1) tmem_dealloc<1>(tmem, NA * BN);
}

// ---------------------------------------------------------------- many rows per expert
//
// The same product with the rows along the M axis (thread = lane = row) and the weight rows along
// N, by pairs of CTAs: 256 rows x 256 columns, each CTA its own 128 rows and half of the shared
// weight tile. The scale of a block is then one number per thread, loaded ahead, and the
// running sums cost the tensor-memory read and a multiply-add per column; with the rows along N each
// column's scale has to be read from shared memory too. The price is that rows come in tiles of
// 256, paid for by every expert's remainder.
//
// A block's columns are two pieces of 128 with their own MMAs and tensor-memory buffers (two each):
// a buffer's way from the tensor cores through the sums and back takes longer than its MMAs, and
// overlaps three others this way.

namespace {

struct RingW {
    static constexpr int BN = 256, piece = 128;
    static constexpr int stage = kABytes + BN / 2 * kChunkBytes;
    static constexpr int stages = 5;
    static constexpr int box_rows = 32;           // rows of x per TMA box
    static constexpr int warps = 16;              // sum warps: eight per piece, 64 columns each
    static constexpr int threads = 128 + 32 * warps;
    static constexpr int out = warps * 16 * 128;  // 16 rows x 128 bytes per sum warp, on their way out
};

// Wait for this thread's tensor-memory loads into v (the values are tied to the wait, so that
// nothing that uses them moves before it). Eight columns at a time: longer reads hold the tensor
// cores' own traffic to tensor memory up (4864 x 4096 x 4096: 68 us, with 16 columns 71, 32: 98).
__device__ __forceinline__ void wait_ld8(uint32_t (&v)[8])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7])
                 :
                 : "memory");
}

}  // namespace

template <bool F32>
__global__ void __launch_bounds__(RingW::threads, 1)
    group_gemm_fp8_wide_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                               const __grid_constant__ Group8Params p)
{
    using T = RingW;
    constexpr int S = T::stages, BN = T::BN, HC = T::piece / 2;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char *sh_out = smem + S * T::stage;
    uint64_t *full = reinterpret_cast<uint64_t *>(sh_out + T::out);
    uint64_t *empty = full + S, *acc_full = empty + S, *acc_empty = acc_full + 4;  // [piece][buffer]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_empty + 4);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *sh_flag = reinterpret_cast<int *>(tmem_slot + 2);
    int *sh_offs = reinterpret_cast<int *>(tmem_slot + 4), *sh_tiles = sh_offs + p.E + 1;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const bool leader = rank == 0;
    const uint64_t wl = p.wait_ns ? p.wait_ns : kWaitNs;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(acc_full + i, 1);
            mbar_init(acc_empty + i, T::warps);  // the piece's sum warps in both CTAs
        }
        *abort_flag = 0;
        fence_mbar_init();
        tc::prefetch_map(&map_w);
        tc::prefetch_map(&map_x);
    }
    if (warp == 1) tmem_alloc<2>(tmem_slot, 2 * BN);
    pdl_enter();  // (only now: the set-up above overlaps the end of the kernel before)
    const bool valid = build_table(p.offs, p.E, p.P, 2 * kTileM, sh_offs, sh_tiles, sh_flag);
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = valid ? FT_OK : FT_ERR_INVALID_ROUTING;
    tc::fence_before_sync();
    cluster_sync();
    tc::fence_after_sync();
    const uint32_t tmem = uniform(*tmem_slot);

    const int n_tiles = (p.N + BN - 1) / BN;
    const int units = uniform(sh_tiles[p.E]) * n_tiles;
    const int nb = (p.K + kStep8 - 1) / kStep8;
    const int u0 = blockIdx.x / 2, du = gridDim.x / 2;
    struct UnitW {
        int e, row0, rows;  // the unit's rows (of both CTAs)
        int n0;             // its first weight row
    };
    auto unit_of = [&](int u) {
        const int t = u / n_tiles;
        const Tile x = find_tile(t, p.E, 2 * kTileM, kTileM, sh_offs, sh_tiles);
        UnitW r;
        r.e = uniform(x.e);
        r.row0 = uniform(x.row0);
        r.rows = uniform(x.rows);
        r.n0 = uniform((u - t * n_tiles) * BN);
        return r;
    };
    // weight rows of piece j that one CTA loads: half the piece's, in steps of 16
    auto half_of = [&](const UnitW &x, int j) { return (min(max(p.N - x.n0 - T::piece * j, 1), T::piece) + 31) / 32 * 16; };
    bool dead = false;

    if (warp < 4) {
        if (warp == 0 && !p.skip_producer) {
            // -------------------------------------------------------- producer
            const bool one = elect_one();
            int s = 0, it = 0;
            uint32_t ph = 1;
            for (int u = u0; u < units && !dead; u += du) {
                const UnitW x = unit_of(u);
                // boxes of x rows: this CTA's, and both CTAs' (the leader expects them all)
                auto boxes_of = [&](int r) { return (min(max(x.rows - r * kTileM, 0), kTileM) + T::box_rows - 1) / T::box_rows; };
                const int boxes = boxes_of(rank);
                const uint32_t bytes = ((boxes_of(0) + boxes_of(1)) * T::box_rows + 4 * 64) * kChunkBytes;
                const int w0 = x.n0 + (int)rank * half_of(x, 0), w1 = x.n0 + T::piece + (int)rank * half_of(x, 1);
                for (int b = 0; b < nb; ++b, ++it) {
                    if (!warp_wait(empty + s, ph, abort_flag, wl)) { dead = true; break; }
                    unsigned char *sa = smem + s * T::stage, *sb = sa + kABytes;
                    const uint32_t bar = map_rank(full + s, 0);
                    if (one) {
                        if (leader) mbar_arrive_expect_tx(full + s, bytes);
                        for (int i = 0; i < boxes; ++i)
                            load_2d<2>(sa + i * T::box_rows * kChunkBytes, &map_x, b * kStep8,
                                       x.row0 + (int)rank * kTileM + i * T::box_rows, bar);
                        load_3d<2>(sb, &map_w, b * kStep8, w0, x.e, bar);
                        load_3d<2>(sb + 64 * kChunkBytes, &map_w, b * kStep8, w1, x.e, bar);
                    }
                    __syncwarp();
                    if (++s == S) { s = 0; ph ^= 1; }
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
            const bool one = elect_one();
            int s = 0, a = 0;
            uint32_t ph = 0, pa = 1;
            for (int u = u0; u < units && !dead; u += du) {
                const UnitW x = unit_of(u);
                const uint32_t idesc[2] = {idesc_e4m3(2 * kTileM, 2 * half_of(x, 0)), idesc_e4m3(2 * kTileM, 2 * half_of(x, 1))};
                for (int b = 0; b < nb && !dead; ++b) {
                    if (!warp_wait(full + s, ph, abort_flag, wl)) { dead = true; break; }
                    const uint32_t sa = smem_u32(smem + s * T::stage);
                    const uint64_t ad = tc::sw128_desc(sa);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (!warp_wait(acc_empty + 2 * j + a, pa, abort_flag, wl)) { dead = true; break; }
                        tc::fence_after_sync();
                        const uint64_t bd = tc::sw128_desc(sa + kABytes + j * 64 * kChunkBytes);
                        if (one) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                mma_e4m3<2>(tmem + (uint32_t)a * BN + j * T::piece, ad + 2 * i, bd + 2 * i, idesc[j], i != 0);
                            commit<2>(acc_full + 2 * j + a);
                            if (j == 1) commit<2>(empty + s);
                        }
                        __syncwarp();
                    }
                    if (++s == S) { s = 0; ph ^= 1; }
                    a ^= 1;
                    if (a == 0) pa ^= 1;
                }
            }
            if (dead && lane == 0) { raise_status(p.status, FT_ERR_TIMEOUT); *abort_flag = 1; }
        }
    } else {
        // ------------------------------------------------------------ sums and epilogue
        const int q = warp & 3, j = (warp - 4) >> 3, h = ((warp - 4) >> 2) & 1;  // lane quarter, piece, its half
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * q) << 16) + j * T::piece + h * HC;
        const uint32_t empty_bar = map_rank(acc_empty + 2 * j, 0);
        unsigned char *tile = sh_out + (warp - 4) * 16 * 128;
        const int n_blocks128 = (p.N + 127) / 128;
        int a = 0;
        uint32_t pa = 0;
        UnitW x;
        int first, live;           // the warp's first row of the unit, and how many of its rows are the unit's
        const float *xs, *ws;      // this thread's row's and the piece's scales
        float xn[4], wn[4];        // those of this block and the next three (a load takes longer than a block)
        auto enter = [&](int u) {
            x = unit_of(u);
            first = (int)rank * kTileM + 32 * q;
            live = min(max(x.rows - first, 0), 32);
            xs = p.xs + x.row0 + (lane < live ? first + lane : 0);
            ws = p.ws + ((int64_t)x.e * n_blocks128 + min(x.n0 / 128 + j, n_blocks128 - 1)) * nb;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xn[i] = i < nb ? __ldg(xs + i * p.ld_xs) : 0.f;
                wn[i] = i < nb ? __ldg(ws + i) : 0.f;
            }
        };
        if (u0 < units) enter(u0);
        for (int u = u0; u < units && !dead; u += du) {
            float2 sum[HC / 2];
#pragma unroll
            for (int i = 0; i < HC / 2; ++i) sum[i] = make_float2(0.f, 0.f);
            for (int b = 0; b < nb; ++b) {
                const float f = xn[0] * wn[0];
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    xn[i] = xn[i + 1];
                    wn[i] = wn[i + 1];
                }
                if (b + 4 < nb) {
                    xn[3] = __ldg(xs + (b + 4) * p.ld_xs);
                    wn[3] = __ldg(ws + b + 4);
                }
                if (!warp_wait(acc_full + 2 * j + a, pa, abort_flag, wl)) { dead = true; break; }
                tc::fence_after_sync();
                const uint32_t addr = lane_addr + (uint32_t)a * BN;
#pragma unroll
                for (int c = 0; c < HC / 8; ++c) {
                    uint32_t v[8];
                    tc::ld8(addr + 8 * c, v);
                    wait_ld8(v);
                    if (c == HC / 8 - 1) {  // read out: the tensor cores may have the buffer back
                        tc::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) arrive_cluster_relaxed(empty_bar + 8 * a);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) fma2(sum[4 * c + i], f, f, v[2 * i], v[2 * i + 1]);
                }
                a ^= 1;
                if (a == 0) pa ^= 1;
            }
            if (dead) break;
            {
                const int n0 = x.n0 + j * T::piece + h * HC;               // these 64 columns
                const int mine = min(max(p.N - n0, 0), HC);               // how many of them exist
                const int64_t at = (int64_t)(x.row0 + first) * p.ld + n0;  // their first element
                const int rows = live;
                if (u + du < units) enter(u + du);  // the next unit's first scales, while this one is stored
                // 128 bytes of each row at a time through shared memory (16-byte pieces swizzled by
                // the row, free of bank conflicts), so that a store instruction writes whole lines
                // of four rows instead of 16 bytes of 32. Rows that are not made of 16-byte pieces leave
                // a row at a time, an element a lane (8 experts of 867 x 432, 11244 rows, with the
                // quantizer: 25 us; an element of each of 32 rows at a time 132, 864 columns 21)
                constexpr int per = F32 ? 32 : 64;
                const int l8 = lane & 7, r4 = lane >> 3;
#pragma unroll
                for (int c = 0; c < HC; c += per) {
                    if (c >= mine) break;
                    uint4 o[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if constexpr (F32) {
                            const float2 s0 = sum[c / 2 + 2 * i], s1 = sum[c / 2 + 2 * i + 1];
                            o[i] = make_uint4(__float_as_uint(s0.x), __float_as_uint(s0.y), __float_as_uint(s1.x),
                                              __float_as_uint(s1.y));
                        } else {
                            const float2 *t = sum + 4 * i;
                            o[i] = make_uint4(bf16x2(t[0].x, t[0].y), bf16x2(t[1].x, t[1].y), bf16x2(t[2].x, t[2].y),
                                              bf16x2(t[3].x, t[3].y));
                        }
                    }
                    const int col = c + l8 * (per / 8);
#pragma unroll
                    for (int g = 0; g < 2; ++g) {  // 16 rows at a time
                        __syncwarp();
                        if (lane >> 4 == g) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                *reinterpret_cast<uint4 *>(tile + (lane & 15) * 128 + ((i ^ l8) << 4)) = o[i];
                        }
                        __syncwarp();
                        if (p.vec) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int r = 4 * i + r4;
                                const uint4 w = *reinterpret_cast<const uint4 *>(tile + r * 128 + ((l8 ^ (r & 7)) << 4));
                                if (16 * g + r < rows && col < mine)
                                    *reinterpret_cast<uint4 *>(static_cast<char *>(p.out) +
                                                               (at + (16 * g + r) * p.ld + col) * (F32 ? 4 : 2)) = w;
                            }
                        } else {
                            using O = std::conditional_t<F32, uint32_t, uint16_t>;
                            constexpr int each = 16 / (int)sizeof(O);
#pragma unroll 4
                            for (int r = 0; r < 16; ++r)
#pragma unroll
                                for (int i = lane; i < per; i += 32)
                                    if (16 * g + r < rows && c + i < mine)
                                        static_cast<O *>(p.out)[at + (16 * g + r) * p.ld + c + i] =
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
    if (warp == 1) tmem_dealloc<2>(tmem, 2 * BN);
}

namespace {

template <int BN, bool F32>
cudaError_t launch8(const CUtensorMap &w, const CUtensorMap &x, Group8Params &p, int32_t *plan, cudaStream_t s)
{
    using T = Ring8<BN>;
    auto kern = group_gemm_fp8_kernel<BN, F32>;
    constexpr size_t fixed = 1024 + T::stages * T::stage + 4 * T::slots * BN +
                             8 * (2 * T::stages + 2 * T::acc + 2 * T::slots) + 16;
    constexpr size_t most = fixed + table_bytes(kGroupMaxExperts);
    static_assert(most <= 227 * 1024, "shared memory");
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess) return e;
    const int64_t m_tiles = (p.N + kTileM - 1) / kTileM;
    const int64_t units = m_tiles * (p.P / BN + (p.E < p.P ? p.E : p.P));  // at most
    static ClusterLimit clusters;
    // Few units: the CTAs of a cluster share one unit's contraction, at least two blocks each, as
    // long as all clusters run at once.
    p.split = 1;
    while (p.split < 8 && p.K >= 4 * kStep8 * p.split && units <= clusters.get(kern, 2 * p.split, kThreads8, most)) p.split *= 2;
    if (plan) {
        write_plan(plan, 1, BN, p.split, false);
        return cudaSuccess;
    }
    int64_t grid = p.split > 1 ? units : sm_count();
    if (units < grid) grid = units;
    if (grid < 1) grid = 1;
    const cudaError_t le = launch_cluster(kern, dim3((unsigned)grid * p.split), dim3(kThreads8), fixed + table_bytes(p.E), p.split, s, w,
                                          x, p);
    if (le != cudaSuccess) return le;
    count_launches(1);
    return cudaGetLastError();
}

template <bool F32>
cudaError_t launch_wide(const CUtensorMap &w, const CUtensorMap &x, const Group8Params &p, cudaStream_t s)
{
    using T = RingW;
    auto kern = group_gemm_fp8_wide_kernel<F32>;
    constexpr size_t fixed = 1024 + T::stages * T::stage + T::out + 8 * (2 * T::stages + 8) + 16;
    constexpr size_t most = fixed + table_bytes(kGroupMaxExperts);
    static_assert(most <= 227 * 1024, "shared memory");
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)((p.N + T::BN - 1) / T::BN) * (p.P / (2 * kTileM) + (p.E < p.P ? p.E : p.P));  // at most
    static ClusterLimit clusters;
    int64_t grid = clusters.get(kern, 2, T::threads, most);
    if (units < grid) grid = units;
    const cudaError_t le = launch_cluster(kern, dim3((unsigned)grid * 2), dim3(T::threads), fixed + table_bytes(p.E), 2, s, w, x,
                                          p);
    if (le != cudaSuccess) return le;
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_group_gemm_fp8(const GroupGemm8 &g, cudaStream_t s)
{
    Group8Params p = {};
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
    // The tile, by the rows per expert that has any. Measured on 256 experts of 1024 x 2048 (us, with 32
    // or 128 rows along N / 256 rows along M): 12 rows 88 / 87 / 126, 32 rows 114 / 96 / 138, 96 rows
    // 247 / 118 / 154, 128 rows 319 / 159 / 158, 512 rows 1142 / 470 / 396. Where the wide tiles
    // leave most SMs idle, smaller tiles and a shared contraction win: one expert of 2048 x 2048 with
    // 256 rows 8.4 / 8.7 / 12.8.
    const int64_t per = g.P / (g.E < g.P ? g.E : g.P);
    const int64_t pairs = (int64_t)(g.N + 255) / 256 * (g.P / 256 + (g.E < g.P ? g.E : g.P));
    const int bn = per <= 24 ? 32 : per < 128 || g.N <= kTileM || 4 * pairs < sm_count() ? 128 : 256;
    if (g.plan && bn == 256) {
        write_plan(g.plan, 2, bn, 1, false);
        return cudaSuccess;
    }
    CUtensorMap w, x;
    const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    if (g.plan) {  // nothing to read
    } else if (!make_tensor_map_3d(&w, u8, g.w, g.K, g.N, g.E, g.K, (uint64_t)g.K * g.N, kStep8, bn == 256 ? 64 : kTileM,
                            CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_tensor_map_2d(&x, u8, g.x, g.K, g.P, g.ld_x, kStep8, bn == 32 ? Ring8<32>::box_rows : Ring8<128>::box_rows,
                            CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    if (bn == 32) return g.out_f32 ? launch8<32, true>(w, x, p, g.plan, s) : launch8<32, false>(w, x, p, g.plan, s);
    if (bn == 128) return g.out_f32 ? launch8<128, true>(w, x, p, g.plan, s) : launch8<128, false>(w, x, p, g.plan, s);
    return g.out_f32 ? launch_wide<true>(w, x, p, s) : launch_wide<false>(w, x, p, s);
}

}  // namespace ftmoe
