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
#include <cuda_bf16.h>

#include "group_gemm.cuh"

namespace ftmoe {

namespace {

using namespace grp;

constexpr int kThreads4 = 384;   // warps: 0 TMA, 1 MMA, 2-3 scales of x, 4..11 epilogue
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

struct Unit4 {
    int e, m0, row0, rows, cols;  // cols: rows in whole MMA columns
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
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_empty + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *sh_flag = reinterpret_cast<int *>(tmem_slot + 2);
    int *sh_offs = reinterpret_cast<int *>(tmem_slot + 4), *sh_tiles = sh_offs + p.E + 1;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint64_t wl = p.wait_ns ? p.wait_ns : kWaitNs;
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
        *abort_flag = 0;
        fence_mbar_init();
        tc::prefetch_map(&map_w);
        tc::prefetch_map(&map_x);
    }
    if (warp == 1) tmem_alloc<1>(tmem_slot, T::tmem);
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
    const int nstages = (p.K + kStep4 - 1) / kStep4, kt = (p.K + 127) / 128;
    const int b0 = nstages * part / split, nb = nstages * (part + 1) / split;  // this CTA's stages
    const int u0 = blockIdx.x / split, du = gridDim.x / split;
    auto unit_of = [&](int u) {
        const int t = u / m_tiles;
        const Tile x = find_tile(t, p.E, BN, 16, sh_offs, sh_tiles);
        Unit4 r;
        r.e = x.e;
        r.m0 = (u - t * m_tiles) * kTileM;
        r.row0 = x.row0;
        r.rows = x.rows;
        r.cols = (x.rows + 15) / 16 * 16;
        return r;
    };
    auto uniform_unit = [](Unit4 x) {
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
                const Unit4 x = uniform_unit(unit_of(u));
                const int boxes = (x.cols + T::box_rows - 1) / T::box_rows;
                const uint8_t *ws = p.ws + ((int64_t)x.e * m_tiles + x.m0 / kTileM) * kt * kTileBytes;
                for (int b = b0; b < nb; ++b, ++it) {
                    if (!warp_wait(empty + s, ph, abort_flag, wl)) { dead = true; break; }
                    unsigned char *sa = smem + s * T::stage, *sb = sa + kABytes;
                    const uint32_t bar = smem_u32(full + s);
                    const uint32_t sf = min(kt - 2 * b, 2) * kTileBytes;  // (the last stage may have one word a row)
                    if (one) {
                        mbar_arrive_expect_tx(full + s, kABytes + boxes * T::box_rows * kChunkBytes + sf);
                        load_3d<1>(sa, &map_w, b * kChunkBytes, x.m0, x.e, bar);
                        bulk_g2s(sb + T::b_bytes, ws + 2 * b * kTileBytes, sf, full + s);
                        for (int i = 0; i < boxes; ++i)
                            load_2d<1>(sb + i * T::box_rows * kChunkBytes, &map_x, b * kChunkBytes, x.row0 + i * T::box_rows, bar);
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
        int s = 0, ac = 0, it = 0;
        uint32_t ph = 0;
        for (int u = u0; u < units && !dead; u += du) {
            const Unit4 x = uniform_unit(unit_of(u));
            const uint32_t idesc[2] = {idesc_mxf4(kTileM, x.cols, 0), idesc_mxf4(kTileM, x.cols, 1)};
            for (int b = b0; b < nb; ++b, ++it) {
                const int in_part = F32 ? (b - b0) % kPart4 : b - b0;
                const bool first = in_part == 0, last = b + 1 == nb || (F32 && in_part == kPart4 - 1);
                if ((first && !warp_wait(acc_empty + (ac & 1), ((ac >> 1) & 1) ^ 1, abort_flag, wl)) ||
                    !warp_wait(full + s, ph, abort_flag, wl) || !warp_wait(sc_full + s, ph, abort_flag, wl)) {
                    dead = true;
                    break;
                }
                tc::fence_after_sync();
                const uint32_t sa = smem_u32(smem + s * T::stage), sf = sa + kABytes + T::b_bytes;
                const uint64_t ad = tc::sw128_desc(sa), bd = tc::sw128_desc(sa + kABytes), sd = scale_desc(sf);
                const uint32_t d = tmem + (uint32_t)(ac & 1) * BN, sfa = tmem + T::sf_col + (it & 1) * 16, sfb = sfa + 8;
                const int steps = min((p.K - b * kStep4 + 63) / 64, 4);  // instructions that have something to multiply
                if (one) {
                    copy_scales<1>(sfa, sd);
                    copy_scales<1>(sfb, sd + T::sf_bytes / 16);
                    if (steps > 2) {
                        copy_scales<1>(sfa + 4, sd + kTileBytes / 16);
                        copy_scales<1>(sfb + 4, sd + (T::sf_bytes + kTileBytes) / 16);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < steps)
                            mma_mxf4<1>(d, ad + 2 * j, bd + 2 * j, idesc[j & 1], sfa + 4 * (j >> 1), sfb + 4 * (j >> 1),
                                        !first || j != 0);
                    commit<1>(empty + s);
                    if (last) commit<1>(acc_full + (ac & 1));
                }
                __syncwarp();
                if (last) ++ac;
                if (++s == S) { s = 0; ph ^= 1; }
            }
        }
        if (dead && lane == 0) { raise_status(p.status, FT_ERR_TIMEOUT); *abort_flag = 1; }
    } else if (warp < 4) {
        // ------------------------------------------------------------ scales of x
        // The two warps take groups of stages in turn, a group's words loaded together. Column c of the tile goes to
        // word c / 32 of lane c % 32; columns beyond the tile's rows get zeros (their sums are not stored).
        constexpr int G = T::group, C = BN / 32;
        int g = 0, it = 0;  // groups and stages so far, over all units
        for (int u = u0; u < units && !dead; u += du) {
            const Unit4 x = unit_of(u);
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
                                v[i][k][c] = at < kt && 32 * c + lane < x.rows ? __ldg(xr + at * p.ld_xs + 32 * c + lane) : 0u;
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
    } else {
        // ------------------------------------------------------------ epilogue
        // thread = TMEM lane = weight row; columns [h * HC, h * HC + HC) of the tile
        const int q = warp & 3, h = (warp - 4) >> 2;
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * q) << 16) + h * HC;
        int ac = 0;
        const int parts = F32 ? (nb - b0 + kPart4 - 1) / kPart4 : 1;
        for (int u = u0; u < units && !dead; u += du) {
            const Unit4 x = unit_of(u);
            const int mine = min(max(x.rows - h * HC, 0), HC);  // columns of this half in use
            const int m = x.m0 + 32 * q + lane;
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
    }

    // wind down; a cluster leaves together
    tc::fence_before_sync();
    __syncthreads();
    if (split > 1) {  // one unit per cluster: add its CTAs' sums, always in the same order
        cluster_sync();
        if (u0 < units) {
            const Unit4 x = unit_of(u0);
            add_parts<F32>(reinterpret_cast<const float *>(smem), x.rows, x.m0, p.N, x.row0, p.out, p.ld, split, part);
        }
        cluster_sync();
    }
    tc::fence_after_sync();
    if (warp == 1) tmem_dealloc<1>(tmem, T::tmem);
}

namespace {

template <int BN, bool F32>
cudaError_t launch4(const CUtensorMap &w, const CUtensorMap &x, Group4Params &p, int32_t *plan, cudaStream_t s)
{
    using T = Ring4<BN>;
    auto kern = group_gemm_mxfp4_kernel<BN, F32>;
    constexpr size_t fixed = 1024 + T::stages * T::stage + 8 * (3 * T::stages + 4) + 16;
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
    p.status = g.status;
    injected_stall(&p.wait_ns, &p.skip_producer);
    const int64_t per = g.P / (g.E < g.P ? g.E : g.P);
    const int bn = per <= 24 ? 32 : 128;
    CUtensorMap w, x;
    const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const uint64_t bytes = g.K / 2;
    if (g.plan) {  // nothing to read
    } else if (!make_tensor_map_3d(&w, u8, g.w, bytes, g.N, g.E, bytes, bytes * g.N, kChunkBytes, kTileM, CU_TENSOR_MAP_SWIZZLE_128B) ||
               !make_tensor_map_2d(&x, u8, g.x, bytes, g.P, g.ld_x, kChunkBytes, bn == 32 ? Ring4<32>::box_rows : Ring4<128>::box_rows,
                                   CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    if (bn == 32) return g.out_f32 ? launch4<32, true>(w, x, p, g.plan, s) : launch4<32, false>(w, x, p, g.plan, s);
    return g.out_f32 ? launch4<128, true>(w, x, p, g.plan, s) : launch4<128, false>(w, x, p, g.plan, s);
}

}  // namespace ftmoe
