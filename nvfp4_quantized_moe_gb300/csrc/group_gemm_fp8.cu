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
#include <cuda_bf16.h>

#include "group_gemm.cuh"

namespace ftmoe {

namespace {

using namespace grp;

constexpr int kThreads8 = 384;  // warps: 0 TMA, 1 MMA, 2-3 scales, 4..11 sums and epilogue
constexpr int kStep8 = 128;     // contraction steps per stage: one scale block

template <int CG, int BN>
struct Ring8 {
    static constexpr int b_bytes = BN / CG * kChunkBytes;
    static constexpr int stage = kABytes + b_bytes;
    static constexpr int stages = (192 * 1024) / stage < 10 ? (192 * 1024) / stage : 10;
    static constexpr int box_rows = BN <= 32 ? 16 : 32;
    static constexpr int acc = BN >= 256 ? 2 : 8;    // partial-sum buffers in tensor memory
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
    int f32;
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

struct Unit8 {
    int e, m0, row0, rows, half;
};

}  // namespace

template <int CG, int BN>
__global__ void __launch_bounds__(kThreads8, 1)
    group_gemm_fp8_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                          const __grid_constant__ Group8Params p)
{
    using T = Ring8<CG, BN>;
    constexpr int S = T::stages, NA = T::acc, NS = T::slots;
    constexpr int HC = BN / 2;  // columns of one half's warps
    pdl_enter();
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
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0;
    const bool leader = rank == 0;
    const uint64_t wl = p.wait_ns ? p.wait_ns : kWaitNs;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < NA; ++i) {
            mbar_init(acc_full + i, 1);
            mbar_init(acc_empty + i, 8 * CG);
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
    if (warp == 1) tmem_alloc<CG>(tmem_slot, NA * BN);
    const bool valid = build_table(p.offs, p.E, p.P, BN, sh_offs, sh_tiles, sh_flag);
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = valid ? FT_OK : FT_ERR_INVALID_ROUTING;
    tc::fence_before_sync();
    if constexpr (CG == 2) cluster_sync();
    else __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;

    const int m_tiles = (p.N + kTileM * CG - 1) / (kTileM * CG);
    const int units = sh_tiles[p.E] * m_tiles;
    const int nb = (p.K + kStep8 - 1) / kStep8;
    const int u0 = blockIdx.x / CG, du = gridDim.x / CG;
    auto unit_of = [&](int u) {
        const int t = u / m_tiles;
        const Tile x = find_tile(t, p.E, BN, 16 * CG, sh_offs, sh_tiles);
        Unit8 r;
        r.e = x.e;
        r.m0 = ((u - t * m_tiles) * CG + (int)rank) * kTileM;
        r.row0 = x.row0;
        r.rows = x.rows;
        r.half = ((x.rows + CG - 1) / CG + 15) / 16 * 16;
        return r;
    };
    bool dead = false;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0 && !p.skip_producer) {
            int s = 0, it = 0;
            uint32_t ph = 1;
            for (int u = u0; u < units && !dead; u += du) {
                const Unit8 x = unit_of(u);
                const int boxes = (x.half + T::box_rows - 1) / T::box_rows;
                const uint32_t bytes = kABytes + boxes * T::box_rows * kChunkBytes;
                for (int b = 0; b < nb; ++b, ++it) {
                    if (!mbar_wait_timed(empty + s, ph, abort_flag, wl)) { dead = true; break; }
                    unsigned char *sa = smem + s * T::stage, *sb = sa + kABytes;
                    const uint32_t bar = CG == 2 ? map_rank(full + s, 0) : smem_u32(full + s);
                    if (leader) mbar_arrive_expect_tx(full + s, CG * bytes);  // for both CTAs of a pair
                    load_3d<CG>(sa, &map_w, b * kStep8, x.m0, x.e, bar);
                    for (int i = 0; i < boxes; ++i)
                        load_2d<CG>(sb + i * T::box_rows * kChunkBytes, &map_x, b * kStep8,
                                    x.row0 + (int)rank * x.half + i * T::box_rows, bar);
                    if (++s == S) { s = 0; ph ^= 1; }
                }
            }
            if (dead) { raise_status(p.status, FT_ERR_TIMEOUT); *abort_flag = 1; }
            if (dead && leader)  // every issued copy lands before the exit
                for (int i = 0; i < S && i < it; ++i) {
                    const int last = it - 1 - i;
                    mbar_wait_timed(full + last % S, (last / S) & 1, nullptr, wl);
                }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0 && leader) {
            int s = 0, a = 0;
            uint32_t ph = 0, pa = 1;
            for (int u = u0; u < units && !dead; u += du) {
                const Unit8 x = unit_of(u);
                // kind::f8f6f4: e4m3 operands (type fields 0), fp32 sums
                const uint32_t idesc = (1u << 4) | ((uint32_t)(x.half * CG >> 3) << 17) | ((uint32_t)(kTileM * CG >> 4) << 24);
                for (int b = 0; b < nb; ++b) {
                    if (!wait_cluster(acc_empty + a, pa, abort_flag, wl) || !wait_cluster(full + s, ph, abort_flag, wl)) {
                        dead = true;
                        break;
                    }
                    tc::fence_after_sync();
                    const uint32_t a0 = smem_u32(smem + s * T::stage), b0 = a0 + kABytes;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_e4m3<CG>(tmem + (uint32_t)a * BN, tc::sw128_desc(a0 + 32 * j), tc::sw128_desc(b0 + 32 * j), idesc,
                                     j != 0);
                    commit<CG>(empty + s);
                    commit<CG>(acc_full + a);
                    if (++s == S) { s = 0; ph ^= 1; }
                    if (++a == NA) { a = 0; pa ^= 1; }
                }
            }
            if (dead) { raise_status(p.status, FT_ERR_TIMEOUT); *abort_flag = 1; }
        }
    } else if (warp < 4) {
        // ------------------------------------------------------------ scales
        // The two warps take the blocks in turn: slot c of block it = xs[b, row of c] * ws[e, tile, b]
        // (one rounding), zero beyond the tile's rows.
        const int n_blocks128 = (p.N + 127) / 128;
        int it = 0;  // blocks so far, over all units
        for (int u = u0; u < units && !dead; u += du) {
            const Unit8 x = unit_of(u);
            const int tile_m = min(x.m0 / 128, n_blocks128 - 1);
            const float *w = p.ws + ((int64_t)x.e * n_blocks128 + tile_m) * nb;
            const float *xr = p.xs + x.row0;
            for (int b = 0; b < nb; ++b, ++it) {
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
        const uint32_t empty_bar = CG == 2 ? map_rank(acc_empty, 0) : 0;
        int a = 0, it = 0;
        uint32_t pa = 0;
        for (int u = u0; u < units && !dead; u += du) {
            const Unit8 x = unit_of(u);
            float2 sum[HC / 2];
#pragma unroll
            for (int j = 0; j < HC / 2; ++j) sum[j] = make_float2(0.f, 0.f);
            const int mine = min(max(x.rows - h * HC, 0), HC);  // columns of this half in use
            for (int b = 0; b < nb; ++b, ++it) {
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
                    if (CG == 2) arrive_cluster_relaxed(empty_bar + 8 * a);
                    else mbar_arrive(acc_empty + a);
                    mbar_arrive(sc_empty + slot);
                }
                if (++a == NA) { a = 0; pa ^= 1; }
            }
            if (dead) break;
            const int m = x.m0 + 32 * q + lane;
            const int n = m < p.N ? mine : 0;
            const int64_t at = ((int64_t)x.row0 + h * HC) * p.ld + m;
            if (p.f32) {
                float *o = static_cast<float *>(p.out) + at;
#pragma unroll
                for (int j = 0; j < HC; ++j)
                    if (j < n) o[j * p.ld] = j & 1 ? sum[j / 2].y : sum[j / 2].x;
            } else {
                __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + at;
#pragma unroll
                for (int j = 0; j < HC; ++j)
                    if (j < n) o[j * p.ld] = __float2bfloat16_rn(j & 1 ? sum[j / 2].y : sum[j / 2].x);
            }
            __syncwarp();
        }
        if (dead && lane == 0) { raise_status(p.status, FT_ERR_TIMEOUT); *abort_flag = 1; }
    }

    tc::fence_before_sync();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();
    tc::fence_after_sync();
    if (warp == 1) tmem_dealloc<CG>(tmem, NA * BN);
}

namespace {

template <int CG, int BN>
cudaError_t launch8(const CUtensorMap &w, const CUtensorMap &x, const Group8Params &p, int64_t max_units, cudaStream_t s)
{
    using T = Ring8<CG, BN>;
    auto kern = group_gemm_fp8_kernel<CG, BN>;
    const size_t smem = 1024 + T::stages * T::stage + 4 * T::slots * BN + 8 * (2 * T::stages + 2 * T::acc + 2 * T::slots) +
                        16 + 4 * 2 * (size_t)(p.E + 1);
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    int64_t grid = sm_count() / CG;
    if (max_units < grid) grid = max_units;
    if (grid < 1) grid = 1;
    const cudaError_t le = launch_cluster(kern, dim3((unsigned)grid * CG), dim3(kThreads8), smem, CG, s, w, x, p);
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
    p.f32 = g.out_f32;
    p.status = g.status;
    injected_stall(&p.wait_ns, &p.skip_producer);
    constexpr int BN = 256;
    CUtensorMap w, x;
    const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    if (!make_tensor_map_3d(&w, u8, g.w, g.K, g.N, g.E, g.K, (uint64_t)g.K * g.N, kStep8, kTileM,
                            CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_tensor_map_2d(&x, u8, g.x, g.K, g.P, g.ld_x, kStep8, Ring8<1, BN>::box_rows, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    const int64_t units = (int64_t)((g.N + kTileM - 1) / kTileM) * (g.P / BN + (g.E < g.P ? g.E : g.P));
    return launch8<1, BN>(w, x, p, units, s);
}

}  // namespace ftmoe
