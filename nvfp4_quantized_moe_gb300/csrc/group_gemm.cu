// Grouped bf16 products over ragged expert batches, and their gradients. Expert e owns the rows
// [offs[e], offs[e + 1]) of x, y, dx and dy:
//
//   forward  y[p, n]     = sum_k x[p, k]  w[e, n, k]      M axis n, N axis p, contraction k
//   dgrad    dx[p, k]    = sum_n dy[p, n] w[e, n, k]      M axis k, N axis p, contraction n
//   wgrad    dw[e, n, k] = sum_p dy[p, n] x[p, k]         M axis k, N axis n, contraction p
//
// Operands go from global memory through TMA (128-byte swizzle) into a ring of shared-memory
// stages of 64 contraction steps and from there into tcgen05.mma (kind::f16, bf16 operands,
// fp32 accumulators in tensor memory). An operand whose contraction axis is not the contiguous
// one (w in dgrad, both in wgrad) is read by the tensor cores as it lies (the descriptor's
// transposed form), so nothing is transposed in memory. Sums are fp32 and rounded once, at the
// store.
#include <cuda_bf16.h>

#include "group_gemm.cuh"

namespace ftmoe {

namespace {

using namespace grp;

constexpr int kThreadsG = 256;  // warps: 0 TMA, 1 MMA, 2 tail rows (wgrad), 3 idle, 4..7 epilogue
constexpr int kStep = 64;       // contraction steps per stage
constexpr int kMaxStages = 12;

template <int CG, int BN>
struct Ring {
    static constexpr int b_bytes = BN / CG * kChunkBytes;
    static constexpr int stage = kABytes + b_bytes;
    static constexpr int stages = (200 * 1024) / stage < kMaxStages ? (200 * 1024) / stage : kMaxStages;
    // rows of one TMA box of a row-major B operand: short boxes, so that a short tile loads no
    // more rows than it has (to within a box)
    static constexpr int box_rows = BN <= 32 ? 16 : 32;
};

struct GroupParams {
    const int *offs;      // [E + 1], or null: one expert that owns all P rows
    int E, P;
    int M;                // size of the M axis
    int N;                // wgrad: size of the N axis
    int R;                // forward, dgrad: contraction length
    void *out;            // forward, dgrad: [P][ld]; wgrad: [E][N][M]
    int64_t ld;
    int f32;              // out is fp32 (else bf16)
    int accumulate;       // wgrad, fp32: add to what out holds
    int *status;
    uint64_t wait_ns;
    int skip_producer;
};

// kind::f16 instruction descriptor: bf16 A and B, fp32 D; bits 15/16 = A/B not contiguous along
// the contraction axis.
__device__ __forceinline__ uint32_t idesc_bf16(int M, int N, bool a_mn, bool b_mn)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

template <int CG>
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    if constexpr (CG == 1) {
        tc::mma_f16(d, a, b, idesc, accumulate);
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    }
}

// One unit of work: a 128 x CG by (up to) BN tile of the output.
struct Unit {
    int e, m0;        // expert, first M index of this CTA
    int col0, cols;   // N axis: first index and count (rows p, or columns n of wgrad)
    int half;         // N indices this CTA loads (all, or its half of a pair's)
    int r0, R;        // contraction range
};

}  // namespace

// WG: the wgrad form (both operands transposed, ragged contraction); A_MN: A transposed.
template <int CG, int BN, bool A_MN, bool WG>
__global__ void __launch_bounds__(kThreadsG, 1)
    group_gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                      const __grid_constant__ GroupParams p)
{
    static_assert(!WG || A_MN, "wgrad reads both operands transposed");
    using T = Ring<CG, BN>;
    constexpr int S = T::stages;
    constexpr int kGran = WG ? 64 : 16;  // N indices per CTA come in multiples of this
    pdl_enter();
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + S * T::stage);
    uint64_t *empty = full + S, *tail = empty + S, *acc_full = tail + S, *acc_empty = acc_full + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_empty + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *sh_flag = reinterpret_cast<int *>(tmem_slot + 2);
    int *sh_offs = reinterpret_cast<int *>(tmem_slot + 4), *sh_tiles = sh_offs + p.E + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0;
    const bool leader = rank == 0;
    const uint64_t wl = p.wait_ns ? p.wait_ns : kWaitNs;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(full + i, CG);   // each CTA's producer (or tail warp)
            mbar_init(empty + i, 1);   // the MMA commit
            mbar_init(tail + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + i, 1);
            mbar_init(acc_empty + i, 4 * CG);  // every epilogue warp
        }
        *abort_flag = 0;
        fence_mbar_init();
        tc::prefetch_map(&map_a);
        tc::prefetch_map(&map_b);
    }
    if (warp == 1) tmem_alloc<CG>(tmem_slot, 2 * BN);
    const bool valid = build_table(p.offs, p.E, p.P, BN, sh_offs, sh_tiles, sh_flag);
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = valid ? FT_OK : FT_ERR_INVALID_ROUTING;
    tc::fence_before_sync();
    if constexpr (CG == 2) cluster_sync();
    else __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;

    const int m_tiles = (p.M + kTileM * CG - 1) / (kTileM * CG);
    const int n_tiles = (p.N + BN - 1) / BN;  // wgrad
    const int units = WG ? p.E * n_tiles * m_tiles : sh_tiles[p.E] * m_tiles;
    const int u0 = blockIdx.x / CG, du = gridDim.x / CG;
    auto unit_of = [&](int u) {
        Unit r;
        const int t = u / m_tiles;
        r.m0 = ((u - t * m_tiles) * CG + (int)rank) * kTileM;
        if (WG) {
            r.e = t / n_tiles;
            r.col0 = (t - r.e * n_tiles) * BN;
            r.cols = min(BN, p.N - r.col0);
            r.r0 = sh_offs[r.e];
            r.R = max(sh_offs[r.e + 1] - r.r0, 0);
        } else {
            const Tile x = find_tile(t, p.E, BN, 16 * CG, sh_offs, sh_tiles);
            r.e = x.e;
            r.col0 = x.row0;
            r.cols = x.rows;
            r.r0 = 0;
            r.R = p.R;
        }
        r.half = ((r.cols + CG - 1) / CG + kGran - 1) / kGran * kGran;
        return r;
    };
    bool dead = false;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0 && !p.skip_producer) {
            int s = 0, it = 0;
            uint32_t ph = 1;
            for (int u = u0; u < units && !dead; u += du) {
                const Unit x = unit_of(u);
                const int nb = (x.R + kStep - 1) / kStep;
                const int boxes = WG ? x.half / 64 : (x.half + T::box_rows - 1) / T::box_rows;
                const uint32_t bytes = kABytes + boxes * (WG ? 64 * kChunkBytes : T::box_rows * kChunkBytes);
                for (int b = 0; b < nb; ++b, ++it) {
                    if (!mbar_wait_timed(empty + s, ph, abort_flag, wl)) { dead = true; break; }
                    unsigned char *sa = smem + s * T::stage, *sb = sa + kABytes;
                    const int k0 = b * kStep;
                    uint32_t bar;
                    if (WG && b == nb - 1 && (x.R & 15)) {  // the tail warp completes this stage
                        bar = smem_u32(tail + s);
                        mbar_arrive_expect_tx(tail + s, bytes);
                    } else {
                        bar = CG == 2 ? map_rank(full + s, 0) : smem_u32(full + s);
                        if (CG == 2) arrive_expect_tx_cluster(bar, bytes);
                        else mbar_arrive_expect_tx(full + s, bytes);
                    }
                    if (WG) {
                        load_2d<CG>(sa, &map_a, x.m0, x.r0 + k0, bar);
                        load_2d<CG>(sa + 8192, &map_a, x.m0 + 64, x.r0 + k0, bar);
                        for (int i = 0; i < boxes; ++i)
                            load_2d<CG>(sb + i * 8192, &map_b, x.col0 + (int)rank * x.half + 64 * i, x.r0 + k0, bar);
                    } else {
                        if (A_MN) {
                            load_3d<CG>(sa, &map_a, x.m0, k0, x.e, bar);
                            load_3d<CG>(sa + 8192, &map_a, x.m0 + 64, k0, x.e, bar);
                        } else {
                            load_3d<CG>(sa, &map_a, k0, x.m0, x.e, bar);
                        }
                        for (int i = 0; i < boxes; ++i)
                            load_2d<CG>(sb + i * T::box_rows * kChunkBytes, &map_b, k0,
                                        x.col0 + (int)rank * x.half + i * T::box_rows, bar);
                    }
                    if (++s == S) { s = 0; ph ^= 1; }
                }
            }
            if (dead) { raise_status(p.status, FT_ERR_TIMEOUT); *abort_flag = 1; }
            if (dead && leader)  // every issued copy lands before the exit (normally the MMAs have waited for them)
                for (int i = 0; i < S && i < it; ++i) {
                    const int last = it - 1 - i;
                    mbar_wait_timed(full + last % S, (last / S) & 1, nullptr, wl);
                }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0 && leader) {
            int s = 0, uc = 0;
            uint32_t ph = 0;
            for (int u = u0; u < units && !dead; u += du) {
                const Unit x = unit_of(u);
                if (WG && x.R == 0) continue;  // nothing to add up: the epilogue writes zeros
                const int nb = (x.R + kStep - 1) / kStep;
                if (!wait_cluster(acc_empty + (uc & 1), ((uc >> 1) & 1) ^ 1, abort_flag, wl)) { dead = true; break; }
                tc::fence_after_sync();
                const uint32_t acc = tmem + (uint32_t)(uc & 1) * BN;
                const uint32_t idesc = idesc_bf16(kTileM * CG, x.half * CG, A_MN, WG);
                for (int b = 0; b < nb; ++b) {
                    if (!wait_cluster(full + s, ph, abort_flag, wl)) { dead = true; break; }
                    tc::fence_after_sync();
                    const uint32_t a0 = smem_u32(smem + s * T::stage), b0 = a0 + kABytes;
                    const int k16 = min(4, (x.R - b * kStep + 15) / 16);  // beyond the contraction's end: not read
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (j >= k16) break;
                        const uint64_t ad = A_MN ? sw128_desc_mn(a0 + 2048 * j) : tc::sw128_desc(a0 + 32 * j);
                        const uint64_t bd = WG ? sw128_desc_mn(b0 + 2048 * j) : tc::sw128_desc(b0 + 32 * j);
                        mma_bf16<CG>(acc, ad, bd, idesc, (b | j) != 0);
                    }
                    commit<CG>(empty + s);
                    if (++s == S) { s = 0; ph ^= 1; }
                }
                if (dead) break;
                commit<CG>(acc_full + (uc & 1));
                ++uc;
            }
            if (dead) { raise_status(p.status, FT_ERR_TIMEOUT); *abort_flag = 1; }
        }
    } else if (WG && warp == 2 && !p.skip_producer) {
        // ------------------------------------------------------------ tail rows (wgrad)
        // The last stage of an expert's rows also holds rows of the next expert. The MMAs take
        // 16 rows at a time: the rows from R to the next multiple of 16 become zeros in both
        // operands (also where the neighbour's values are not finite).
        int s = 0;
        uint32_t phases = 0;  // bit s: parity of tail[s]
        for (int u = u0; u < units && !dead; u += du) {
            const Unit x = unit_of(u);
            const int nb = (x.R + kStep - 1) / kStep;
            if (nb == 0) continue;
            s = (s + nb - 1) % S;  // the unit's last stage
            if (x.R & 15) {
                if (!warp_wait(tail + s, (phases >> s) & 1, abort_flag, wl)) { dead = true; break; }
                phases ^= 1u << s;
                const int first = x.R - (nb - 1) * kStep, rows = 16 - (first & 15);
                unsigned char *sa = smem + s * T::stage;
                const int boxes = 2 + x.half / 64;
                for (int i = lane; i < boxes * rows * 8; i += 32) {
                    const int box = i / (rows * 8), r = (i / 8) % rows;
                    *reinterpret_cast<uint4 *>(sa + box * 8192 + (first + r) * kChunkBytes + (i & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
                }
                asm volatile("fence.proxy.async;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    if (CG == 2) arrive_cluster(map_rank(full + s, 0));
                    else mbar_arrive(full + s);
                }
            }
            if (++s == S) s = 0;
        }
        if (dead && lane == 0) { raise_status(p.status, FT_ERR_TIMEOUT); *abort_flag = 1; }
    } else if (warp >= 4) {
        // ------------------------------------------------------------ epilogue
        // thread = TMEM lane = M index; the N indices are the columns
        const int q = warp & 3;
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * q) << 16);
        const uint32_t empty_bar = CG == 2 ? map_rank(acc_empty, 0) : smem_u32(acc_empty);
        int uc = 0;
        for (int u = u0; u < units && !dead; u += du) {
            const Unit x = unit_of(u);
            const bool none = WG && x.R == 0;
            if (none && p.accumulate) continue;
            if (!none) {
                if (!warp_wait(acc_full + (uc & 1), (uc >> 1) & 1, abort_flag, wl)) { dead = true; break; }
                tc::fence_after_sync();
            }
            const int m = x.m0 + 32 * q + lane;
            const int64_t first = WG ? (int64_t)x.e * p.N + x.col0 : x.col0;
            for (int c0 = 0; c0 < x.cols; c0 += 32) {
                uint32_t v[32];
                if (none) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0u;
                } else {
                    tc::ld32(lane_addr + (uint32_t)(uc & 1) * BN + c0, v);
                    tc::wait_ld();
                    if (c0 + 32 >= x.cols) {  // read out: the next unit's MMAs may start
                        tc::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) arrive_cluster(empty_bar + 8 * (uc & 1));
                    }
                }
                const int n = m < p.M ? min(32, x.cols - c0) : 0;
                if (p.f32) {
                    float *o = static_cast<float *>(p.out) + (first + c0) * p.ld + m;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j < n) {
                            float a = __uint_as_float(v[j]);
                            if (WG && p.accumulate) a += o[j * p.ld];
                            o[j * p.ld] = a;
                        }
                } else {
                    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + (first + c0) * p.ld + m;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j < n) o[j * p.ld] = __float2bfloat16_rn(__uint_as_float(v[j]));
                }
                __syncwarp();
            }
            if (!none) ++uc;
        }
        if (dead && lane == 0) { raise_status(p.status, FT_ERR_TIMEOUT); *abort_flag = 1; }
    }

    // wind down; a pair leaves together (its MMAs and barriers reach into both CTAs)
    tc::fence_before_sync();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();
    tc::fence_after_sync();
    if (warp == 1) tmem_dealloc<CG>(tmem, 2 * BN);
}

namespace {

template <int CG, int BN, bool A_MN, bool WG>
cudaError_t launch(const CUtensorMap &a, const CUtensorMap &b, const GroupParams &p, int64_t max_units, cudaStream_t s)
{
    using T = Ring<CG, BN>;
    auto kern = group_gemm_kernel<CG, BN, A_MN, WG>;
    const size_t smem = 1024 + T::stages * T::stage + 8 * (3 * T::stages + 4) + 16 + 4 * 2 * (size_t)(p.E + 1);
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    int64_t grid = sm_count() / CG;
    if (max_units < grid) grid = max_units;
    if (grid < 1) grid = 1;
    const cudaError_t le = launch_cluster(kern, dim3((unsigned)grid * CG), dim3(kThreadsG), smem, CG, s, a, b, p);
    if (le != cudaSuccess) return le;
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_group_gemm(const GroupGemm &g, cudaStream_t s)
{
    GroupParams p = {};
    p.offs = g.offs;
    p.E = g.E;
    p.P = g.P;
    p.out = g.out;
    p.ld = g.ld_out;
    p.f32 = g.out_f32;
    p.accumulate = g.accumulate;
    p.status = g.status;
    injected_stall(&p.wait_ns, &p.skip_producer);
    const bool wg = g.form == kGroupWgrad;
    p.M = g.form == kGroupForward ? g.N : g.K;
    p.N = g.N;
    p.R = g.form == kGroupForward ? g.K : g.N;
    constexpr int BN = 256;
    const int box_rows = Ring<1, BN>::box_rows;
    const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    CUtensorMap a, b;
    bool ok;
    if (wg) {  // A: x [P][K] read along k; B: dy [P][N] read along n
        ok = make_tensor_map_2d(&a, bf, g.x, g.K, g.P, 2 * (uint64_t)g.ld_x, 64, kStep, CU_TENSOR_MAP_SWIZZLE_128B) &&
             make_tensor_map_2d(&b, bf, g.dy, g.N, g.P, 2 * (uint64_t)g.ld_dy, 64, kStep, CU_TENSOR_MAP_SWIZZLE_128B);
    } else {   // A: w [E][N][K]; B: x [P][K] or dy [P][N]
        const bool fw = g.form == kGroupForward;
        ok = make_tensor_map_3d(&a, bf, g.w, g.K, g.N, g.E, 2 * (uint64_t)g.K, 2 * (uint64_t)g.K * g.N, 64,
                                fw ? kTileM : kStep, CU_TENSOR_MAP_SWIZZLE_128B) &&
             make_tensor_map_2d(&b, bf, fw ? g.x : g.dy, fw ? g.K : g.N, g.P,
                                2 * (uint64_t)(fw ? g.ld_x : g.ld_dy), 64, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
    }
    if (!ok) return cudaErrorInvalidValue;
    const int64_t m_tiles = (p.M + kTileM - 1) / kTileM;
    const int64_t tiles = wg ? (int64_t)g.E * ((g.N + BN - 1) / BN) : g.P / BN + (g.E < g.P ? g.E : g.P);
    const int64_t units = m_tiles * tiles;
    if (wg) return launch<1, BN, true, true>(a, b, p, units, s);
    if (g.form == kGroupDgrad) return launch<1, BN, true, false>(a, b, p, units, s);
    return launch<1, BN, false, false>(a, b, p, units, s);
}

}  // namespace ftmoe
