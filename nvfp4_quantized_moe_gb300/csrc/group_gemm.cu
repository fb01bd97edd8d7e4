// Grouped bf16 products over ragged expert batches, and their gradients. Expert e owns the rows
// [offs[e], offs[e + 1]) of x, y, dx and dy:
//
//   forward  y[p, n]     = sum_k x[p, k]  w[e, n, k]      M axis n, N axis p, contraction k
//   dgrad    dx[p, k]    = sum_n dy[p, n] w[e, n, k]      M axis k, N axis p, contraction n
//   wgrad    dw[e, n, k] = sum_p dy[p, n] x[p, k]         M axis k, N axis n, contraction p
//
// Operands go from global memory through TMA (128-byte swizzle) into a ring of shared-memory
// stages of 64 contraction steps and from there into tcgen05.mma (kind::f16, bf16 operands,
// fp32 accumulators in tensor memory, two of them so that one is stored while the next fills).
// An operand whose contraction axis is not the contiguous one (w in dgrad, both in wgrad) is read
// by the tensor cores as it lies (the descriptor's transposed form), so nothing is transposed in
// memory. Sums are fp32 and rounded once, at the store.
//
// What bounds it, measured on one GB300 (copy bandwidth 6.78 TB/s, cuBLAS bf16 1932 TFLOP/s):
//   - many rows per expert: the tensor cores. Dense 4864 x 4096 x 4096 takes 84 us, 1940 TFLOP/s
//     (cuBLAS 82). Tiles of 256 x 256 by pairs of CTAs: one CTA alone would have to load 48 KB per
//     stage that its MMAs finish in a quarter of a microsecond.
//   - few rows: the weights' one pass through memory. 64 tokens that reach 222 of 256 experts of 1024 x 2048
//     (0.93 GB) take 139 us, 6.7 TB/s; 2560 rows over 256 experts of 4096 x 4096 (8.6 GB) 1.20 ms in dgrad,
//     7.2 TB/s. DRAM traffic equals what the operands hold.
//   - both at once, where a few experts have most rows: the weights of the others, then the MMAs of these.
//     4096 Zipf-distributed tokens that reach 165 of those 256 experts of 4096 x 4096 (dgrad, 6.1 GB) take
//     1.16 ms, 5.2 TB/s; its 133 experts below 128 rows alone 0.68, the others alone 0.59.
//   - a handful of rows: the chain of latencies from launch to store. One token over 8 of 256
//     experts (2048 x 512) takes 6.7 us, one expert of 2048 x 2048 with 4 rows 7.0 us.
//   - wgrad: the output. fp32 dw [256, 1024, 2048] (2.1 GB) of 65536 rows takes 394 us with 256 rows
//     per expert (6.5 TB/s read and written) and 510 us with Zipf-distributed ones, where the large
//     experts' MMAs and the small ones' stores add up in each SM.
//     Added to dw (4.3 GB read and written), 256 rows each take 801 us, as reductions that L2 carries
//     out; read, added and stored by the warps, each value's latency waited for, 2525 us.
//   - wgrad of few tiles: the rows of an expert, shared by a cluster. One expert of 256 x 2048 with
//     8192 rows takes 22 us (not shared 54).
#include <cuda_bf16.h>

#include "group_gemm.cuh"

namespace ftmoe {

namespace {

using namespace grp;

constexpr int kStep = 64;       // contraction steps per stage
// Long sums are cut into parts of this many stages, added in registers: the tensor cores truncate
// where an fp32 addition rounds, so that the error of one long accumulation grows with its length
// (fp32 outputs: 5e-6 relative over 8192 steps, against 4.4e-7 for sums in parts of 512; elementary
// operations in fp32 have 1.7e-7).
constexpr int kPartStages = 8;
// bf16 outputs round at 2^-9 (2e-3) on average and keep one accumulation over up to kLongRows steps. Over 4096
// steps single roundings then fall to the other side than with fp32 sums, 1e-4 in norm, and the error against
// 64 bits is the same. Products of one sign, whose losses add up, come out 3e-5 low after 8192 steps and 4e-4
// after 65536, the widest contraction of forward and dgrad; after a million it is 0.6%, after four 2.6%, and
// an expert may have that many rows: wgrad of more than kLongRows rows adds up parts of kLongStages
// too, which lose 3e-5 at most (256 truncations of 2^-23). Its epilogue holds 128 running sums a thread, at a
// cost where units are short (256 experts of 1024 x 2048, us without / with: 256 rows each 294 / 354, 512
// 443 / 455, 1024 764 / 771; one of 256 x 256 with 2^21 rows 1676 / 1682).
constexpr int kLongRows = 65536;
constexpr int kLongStages = 64;
// wgrad: units handed out ahead of the epilogue. Small units need the distance to keep loads in
// flight, and a large one in between makes those behind it wait (Zipf-distributed rows, fp32 dw
// [256, 1024, 2048]: 2 ahead 524 us, 3 502, 4 513, 6 534).
constexpr int kAhead = 3;

// Tile variants. CG: CTAs per tile of the M axis (a pair shares its B operand and halves what
// each SM must load per multiplication); BN: largest extent along the N axis.
template <int CG, int BN, bool WG>
struct Ring {
    static constexpr int b_bytes = BN / CG * kChunkBytes;
    static constexpr int stage = kABytes + b_bytes;
    // rows of one TMA box of a row-major B operand: short boxes, so that a short tile loads no
    // more rows than it has (to within a box)
    static constexpr int box_rows = BN <= 32 ? 16 : 32;
    // warps: 0 TMA, 1 MMA, 2 tail rows (wgrad only), then eight for the epilogue. No more: an fp32
    // epilogue holds 128 running sums a thread, and every further warp takes registers from it.
    static constexpr int roles = WG ? 3 : 2;
    static constexpr int threads = 32 * (roles + 8);
    static constexpr int fit = 216 * 1024 / stage;
    // (eight keep memory busy; with ten a decode step of 64 tokens took 152 us, with eight 142)
    static constexpr int stages = fit < 8 ? fit : 8;
};

struct GroupParams {
    const int *offs;      // [E + 1], or null: one expert that owns all P rows
    int E, P;
    int M;                // size of the M axis
    int N;                // wgrad: size of the N axis
    int R;                // forward, dgrad: contraction length
    void *out;            // forward, dgrad: [P][ld]; wgrad: [E][N][ld]
    int64_t ld;
    int split;            // CTAs (one cluster) that share a unit's contraction
    int *counter;         // units handed out so far (zero at launch), or null: units go in turn
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
    int col0, cols;   // N axis: first index and count (rows p, or n of wgrad)
    int half;         // N indices this CTA loads (all, or its half of a pair's)
    int r0, R;        // contraction range
};

}  // namespace

// WG: the wgrad form (both operands transposed, ragged contraction); A_MN: A transposed; ACC: wgrad
// that adds to what dw holds (a kernel of its own: the branch in the stores cost the plain one 8%,
// in registers: 256 experts of 1024 x 2048 with 256 rows each 396 and 426 us); LONG: wgrad into bf16
// of more than kLongRows rows.
template <int CG, int BN, bool A_MN, bool WG, bool F32, bool ACC, bool LONG>
__global__ void __launch_bounds__(Ring<CG, BN, WG>::threads, 1)
    group_gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                      const __grid_constant__ GroupParams p)
{
    static_assert(!WG || A_MN, "wgrad reads both operands transposed");
    static_assert(!ACC || (WG && F32), "only wgrad adds, in fp32");
    static_assert(!LONG || (WG && !F32), "fp32 outputs always add up parts");
    constexpr bool kSums = F32 || LONG;        // parts and their running sums
    constexpr int kPart = F32 ? kPartStages : kLongStages;
    using T = Ring<CG, BN, WG>;
    constexpr int S = T::stages;
    constexpr int kGran = WG ? 64 : 16;        // N indices per CTA come in multiples of this
    constexpr bool kSplit = CG == 1;
    constexpr int HC = BN / 2;                 // columns of one half's epilogue warps
    constexpr int W = HC < 32 ? HC : 32;       // columns per tensor-memory load
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + S * T::stage);
    uint64_t *empty = full + S, *tail = empty + S, *peer_tail = tail + S, *acc_full = peer_tail + S,
             *acc_empty = acc_full + 2, *unit_full = acc_empty + 2, *unit_empty = unit_full + kAhead;
    int *sh_unit = reinterpret_cast<int *>(unit_empty + kAhead);  // the next units
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sh_unit + kAhead);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *sh_flag = reinterpret_cast<int *>(tmem_slot + 2);
    int *sh_offs = reinterpret_cast<int *>(tmem_slot + 4), *sh_tiles = sh_offs + p.E + 1;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int split = kSplit ? p.split : 1;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0;
    const bool leader = rank == 0;
    const uint64_t wl = p.wait_ns ? p.wait_ns : kWaitNs;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(full + i, 1);       // the leader's producer (or tail warp), for both CTAs of a pair
            mbar_init(empty + i, 1);      // the MMA commit
            mbar_init(tail + i, 1);       // wgrad: this CTA's copies of a stage that has tail rows
            mbar_init(peer_tail + i, 1);  // wgrad, leader: the other CTA's tail rows are zeroed
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + i, 1);
            mbar_init(acc_empty + i, 8 * CG);  // every epilogue warp
        }
        for (int i = 0; i < kAhead; ++i) {
            mbar_init(unit_full + i, 1);
            mbar_init(unit_empty + i, CG * 10);  // all warps that take units: MMA, tail and epilogue; the other CTA's
                                                 // producer, tail and epilogue
        }
        if (CG == 2 && !leader)
            for (int i = 0; i < kAhead; ++i) mbar_arrive_expect_tx(unit_full + i, 4);
        *abort_flag = 0;
        fence_mbar_init();
        tc::prefetch_map(&map_a);
        tc::prefetch_map(&map_b);
    }
    if (warp == 1) tmem_alloc<CG>(tmem_slot, 2 * BN);
    pdl_enter();  // (only now: the set-up above overlaps the end of the kernel before)
    const bool valid = build_table(p.offs, p.E, p.P, BN, sh_offs, sh_tiles, sh_flag);
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = valid ? FT_OK : FT_ERR_INVALID_ROUTING;
    tc::fence_before_sync();
    if constexpr (CG == 2) cluster_sync();
    else __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = uniform(*tmem_slot);

    const int m_tiles = (p.M + kTileM * CG - 1) / (kTileM * CG);
    const int n_tiles = (p.N + BN - 1) / BN;  // wgrad
    const int units = WG ? p.E * n_tiles * m_tiles : uniform(sh_tiles[p.E]) * m_tiles;
    const int u0 = blockIdx.x / (CG * split), du = gridDim.x / (CG * split);
    const int part = kSplit ? (int)(blockIdx.x % split) : 0;
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
    auto uniform_unit = [](Unit x) {
        x.e = uniform(x.e); x.m0 = uniform(x.m0); x.col0 = uniform(x.col0); x.cols = uniform(x.cols);
        x.half = uniform(x.half); x.r0 = uniform(x.r0); x.R = uniform(x.R);
        return x;
    };
    // this CTA's stages [first, last) of a contraction of R steps
    auto first_stage = [&](int R) { return kSplit ? (R + kStep - 1) / kStep * part / split : 0; };
    auto last_stage = [&](int R) {
        const int nb = (R + kStep - 1) / kStep;
        return kSplit ? nb * (part + 1) / split : nb;
    };
    bool dead = false;
    // The warp's next unit, or -1 after the last one. With a counter (wgrad, whose units cost as much
    // as their expert has rows), the leader's producer hands them out: whoever is done takes the
    // next. Dealt out in turn, the largest experts' units ended last on some CTAs (Zipf-distributed
    // rows, fp32 dw [256, 1024, 2048]: 587 us). Forward and dgrad units cost about the same; there
    // the counter gained nothing. (Pairs only: the ring's stores go from CTA to CTA of a cluster.)
    constexpr bool kCounted = WG && CG == 2;
    const bool counted = kCounted && p.counter;
    const uint32_t unit_empty_bar = CG == 2 ? map_rank(unit_empty, 0) : 0;
    int turn = 0;
    auto next_unit = [&]() {
        int u;
        if (!counted) {
            u = u0 + turn * du;
        } else {
            const int i = turn % kAhead;
            if (!warp_wait(unit_full + i, (turn / kAhead) & 1, abort_flag, wl)) { dead = true; return -1; }
            u = uniform(*(volatile int *)(sh_unit + i));
            __syncwarp();
            if (lane == 0) {
                if (warp == 0) mbar_arrive_expect_tx(unit_full + i, 4);  // (the other CTA's producer: the slot's next unit)
                arrive_cluster_relaxed(unit_empty_bar + 8 * i);
            }
        }
        ++turn;
        return u < units ? u : -1;
    };

    // The leader's producer: the counter's next unit, for itself and the ring.
    int ticket = u0;  // (the first is this CTA's or pair's own)
    auto hand_out = [&]() {
        const int i = turn % kAhead, u = uniform(ticket);
        if (!warp_wait(unit_empty + i, ((turn / kAhead) & 1) ^ 1, abort_flag, wl)) { dead = true; return -1; }
        // into both CTAs; the asynchronous store completes the barrier's phase by itself
        if (lane == 0) mbar_arrive_expect_tx(unit_full + i, 4);
        if (lane < CG)
            asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(
                             map_rank(sh_unit + i, lane)),
                         "r"(u), "r"(map_rank(unit_full + i, lane))
                         : "memory");
        __syncwarp();
        if (lane == 0 && u < units) ticket = du + atomicAdd(p.counter, 1);  // (known by the next turn)
        ++turn;
        return u < units ? u : -1;
    };

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (!p.skip_producer) {
            const bool one = elect_one();
            int s = 0, it = 0;
            uint32_t ph = 1;
            for (int u; (u = kCounted && counted && leader ? hand_out() : next_unit()) >= 0 && !dead;) {
                const Unit x = uniform_unit(unit_of(u));
                const int nb = last_stage(x.R);
                const int boxes = WG ? x.half / 64 : (x.half + T::box_rows - 1) / T::box_rows;
                const uint32_t bytes = kABytes + boxes * (WG ? 64 * kChunkBytes : T::box_rows * kChunkBytes);
                for (int b = first_stage(x.R); b < nb; ++b, ++it) {
                    if (!warp_wait(empty + s, ph, abort_flag, wl)) { dead = true; break; }
                    unsigned char *sa = smem + s * T::stage, *sb = sa + kABytes;
                    const int k0 = b * kStep;
                    // a stage with tail rows is completed by the tail warp
                    const bool tails = WG && (b + 1) * kStep >= x.R && (x.R & 15);
                    const uint32_t bar = tails ? smem_u32(tail + s) : CG == 2 ? map_rank(full + s, 0) : smem_u32(full + s);
                    if (one) {
                        // the leader expects both CTAs' bytes (equally many); the other's may land first
                        if (tails) mbar_arrive_expect_tx(tail + s, bytes);
                        else if (leader) mbar_arrive_expect_tx(full + s, CG * bytes);
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
                    }
                    __syncwarp();
                    if (++s == S) { s = 0; ph ^= 1; }
                }
            }
            // The last stages' MMAs also arrive in the other CTA: neither leaves before all have.
            for (int i = 0; CG == 2 && i < S && !dead; ++i) {
                if (!warp_wait(empty + s, ph, abort_flag, wl)) dead = true;
                if (++s == S) { s = 0; ph ^= 1; }
            }
            if (dead && lane == 0) { raise_status(p.status, FT_ERR_TIMEOUT); *abort_flag = 1; }
            if (dead && leader)  // every issued copy lands before the exit (normally the MMAs have waited for them)
                for (int i = 0; i < S && i < it; ++i) {
                    const int last = it - 1 - i;
                    mbar_wait_timed(full + last % S, (last / S) & 1, nullptr, wl);
                }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (leader) {
            const bool one = elect_one();
            int s = 0, ac = 0;
            uint32_t ph = 0;
            for (int u; (u = next_unit()) >= 0 && !dead;) {
                const Unit x = uniform_unit(unit_of(u));
                const int b0 = first_stage(x.R), nb = last_stage(x.R);
                const uint32_t idesc = idesc_bf16(kTileM * CG, x.half * CG, A_MN, WG);
                // (an expert without rows has no stages: the epilogue writes zeros on its own)
                for (int b = b0; b < nb; ++b) {
                    const bool starts = kSums ? (b - b0) % kPart == 0 : b == b0;
                    const bool ends = b == nb - 1 || (kSums && (b - b0) % kPart == kPart - 1);
                    if (starts && !warp_wait(acc_empty + (ac & 1), ((ac >> 1) & 1) ^ 1, abort_flag, wl)) { dead = true; break; }
                    if (!warp_wait(full + s, ph, abort_flag, wl)) { dead = true; break; }
                    tc::fence_after_sync();
                    const uint32_t acc = tmem + (uint32_t)(ac & 1) * BN;
                    const uint32_t a0 = smem_u32(smem + s * T::stage), bb = a0 + kABytes;
                    const int k16 = min(4, (x.R - b * kStep + 15) / 16);  // beyond the contraction's end: not read
                    // 16 contraction steps further: 2048 bytes (transposed) or 32, in units of 16
                    const uint64_t ad = A_MN ? sw128_desc_mn(a0) : tc::sw128_desc(a0);
                    const uint64_t bd = WG ? sw128_desc_mn(bb) : tc::sw128_desc(bb);
                    if (one) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (j < k16)
                                mma_bf16<CG>(acc, ad + j * (A_MN ? 128 : 2), bd + j * (WG ? 128 : 2), idesc, !starts || j != 0);
                        commit<CG>(empty + s);
                        if (ends) commit<CG>(acc_full + (ac & 1));
                    }
                    __syncwarp();
                    if (ends) ++ac;
                    if (++s == S) { s = 0; ph ^= 1; }
                }
            }
            if (dead && lane == 0) { raise_status(p.status, FT_ERR_TIMEOUT); *abort_flag = 1; }
        }
    } else if (WG && warp == 2 && !p.skip_producer) {
        // ------------------------------------------------------------ tail rows (wgrad)
        // The last stage of an expert's rows also holds rows of the next expert. The MMAs take
        // 16 rows at a time: the rows from R to the next multiple of 16 become zeros in both
        // operands (also where the neighbour's values are not finite).
        int s = 0;
        uint32_t phases = 0;  // bit s: parity of tail[s]
        for (int u; (u = next_unit()) >= 0 && !dead;) {
            const Unit x = unit_of(u);
            const int nb = last_stage(x.R), n = nb - first_stage(x.R);
            if (n == 0) continue;
            s = (s + n - 1) % S;  // the unit's last stage here
            if (nb * kStep >= x.R && (x.R & 15)) {
                const uint32_t parity = (phases >> s) & 1;
                if (!warp_wait(tail + s, parity, abort_flag, wl)) { dead = true; break; }
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
                if (!leader) {
                    if (lane == 0) arrive_cluster(map_rank(peer_tail + s, 0));
                } else {
                    if (CG == 2) {
                        const bool ok = wait_cluster(peer_tail + s, parity, abort_flag, wl);
                        if (!__all_sync(0xFFFFFFFFu, ok)) { dead = true; break; }
                    }
                    if (lane == 0) mbar_arrive(full + s);
                }
            }
            if (++s == S) s = 0;
        }
        if (dead && lane == 0) { raise_status(p.status, FT_ERR_TIMEOUT); *abort_flag = 1; }
    } else if (warp >= T::roles) {
        // ------------------------------------------------------------ epilogue
        // thread = TMEM lane = M index; the warp takes columns [h * HC, h * HC + HC) of the tile
        const int q = warp & 3, h = (warp - T::roles) >> 2;
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * q) << 16) + h * HC;
        const uint32_t empty_bar = CG == 2 ? map_rank(acc_empty, 0) : 0;
        int ac = 0;
        for (int u; (u = next_unit()) >= 0 && !dead;) {
            const Unit x = unit_of(u);
            const int nb = last_stage(x.R) - first_stage(x.R);
            const int parts = kSums ? (nb + kPart - 1) / kPart : nb > 0;
            if (ACC && parts == 0 && split == 1) continue;
            const int mine = min(max(x.cols - h * HC, 0), HC);  // columns of this half in use
            const int m = x.m0 + 32 * q + lane;

            // W columns at offset c of this half, as sums, to where they go: lanes lie along the contiguous
            // axis of out, so that a store instruction writes a whole line without a detour
            const int64_t row0 = (WG ? (int64_t)x.e * p.N : 0) + x.col0 + h * HC;
            auto emit = [&](int c, const float (&v)[W]) {
                if (kSplit && split > 1) {
                    // (every stage of the ring has been read by the time the last sums are complete)
                    float *red = reinterpret_cast<float *>(smem);
#pragma unroll
                    for (int j = 0; j < W; ++j) red[(h * HC + c + j) * kTileM + 32 * q + lane] = v[j];
                } else {
                    store_rows<F32, W>(v, m, p.M, row0 + c, mine - c, p.out, p.ld, ACC);
                }
            };
            float sum[kSums ? HC : 1];  // the parts' running sums
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
                    if constexpr (kSums) {
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
                if (lane == 0) {
                    if (CG == 2) arrive_cluster_relaxed(empty_bar + 8 * (ac & 1));
                    else mbar_arrive(acc_empty + (ac & 1));
                }
            }
            if (dead) break;
            if (kSums || parts == 0) {
#pragma unroll
                for (int c = 0; c < HC; c += W) {
                    if (c >= mine) break;
                    float f[W];
#pragma unroll
                    for (int j = 0; j < W; ++j) f[j] = kSums && parts ? sum[kSums ? c + j : 0] : 0.f;
                    emit(c, f);
                }
            }
        }
        if (dead && lane == 0) { raise_status(p.status, FT_ERR_TIMEOUT); *abort_flag = 1; }
    }

    // wind down; a cluster leaves together (its MMAs, barriers and sums reach into all its CTAs)
    tc::fence_before_sync();
    __syncthreads();
    if constexpr (kSplit) {
        if (split > 1) {  // one unit per cluster: add its CTAs' sums, always in the same order
            cluster_sync();
            if (u0 < units) {
                const Unit x = unit_of(u0);
                add_parts<F32>(reinterpret_cast<const float *>(smem), x.cols, x.m0, p.M, (WG ? (int64_t)x.e * p.N : 0) + x.col0,
                               p.out, p.ld, split, part, ACC);
            }
            cluster_sync();
        }
    }
    if constexpr (CG == 2) cluster_sync();
    tc::fence_after_sync();
    if (warp == 1) tmem_dealloc<CG>(tmem, 2 * BN);
}

namespace {

template <int CG, int BN, bool A_MN, bool WG, bool F32, bool ACC, bool LONG>
cudaError_t launch(const CUtensorMap (&maps)[2], GroupParams &p, int64_t max_units, int32_t *plan, cudaStream_t s)
{
    using T = Ring<CG, BN, WG>;
    auto kern = group_gemm_kernel<CG, BN, A_MN, WG, F32, ACC, LONG>;
    constexpr size_t fixed = 1024 + T::stages * T::stage + 8 * (4 * T::stages + 4 + 2 * kAhead) + 4 * kAhead + 16;
    constexpr size_t most = fixed + table_bytes(kGroupMaxExperts);
    static_assert(most <= 227 * 1024, "shared memory");
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess) return e;
    static ClusterLimit clusters;
    // Few units: the CTAs of a cluster share one unit's contraction (wgrad: an expert's rows), at least
    // two stages each, as long as all clusters run at once.
    p.split = 1;
    const int64_t steps = WG ? p.P / p.E : p.R;
    if (CG == 1)
        while (p.split < 8 && steps >= 4 * kStep * p.split && max_units <= clusters.get(kern, 2 * p.split, T::threads, most))
            p.split *= 2;
    int64_t grid = p.split > 1 ? max_units : clusters.get(kern, CG, T::threads, most);
    if (max_units < grid) grid = max_units;
    if (grid < 1) grid = 1;
    const bool counted = WG && CG == 2 && p.E > 1 && max_units > 4 * grid;  // units of unlike cost, several each
    if (plan) {
        write_plan(plan, CG, BN, p.split, counted);
        return cudaSuccess;
    }
    if (counted) {
        const cudaError_t me = cudaMemsetAsync(p.status + 16, 0, sizeof(int), s);
        if (me != cudaSuccess) return me;
        p.counter = p.status + 16;
    }
    const int cluster = CG * p.split;
    const cudaError_t le = launch_cluster(kern, dim3((unsigned)grid * cluster), dim3(T::threads), fixed + table_bytes(p.E), cluster, s,
                                          maps[0], maps[1], p);
    if (le != cudaSuccess) return le;
    count_launches(1);
    return cudaGetLastError();
}

template <int CG, int BN, bool A_MN, bool WG>
cudaError_t launch_typed(const GroupGemm &g, const CUtensorMap (&maps)[2], GroupParams &p, cudaStream_t s)
{
    const int64_t m_tiles = (p.M + kTileM * CG - 1) / (kTileM * CG);
    const int64_t tiles = WG ? (int64_t)g.E * ((p.N + BN - 1) / BN) : g.P / BN + (g.E < g.P ? g.E : g.P);
    if constexpr (WG) {
        if (g.accumulate) return launch<CG, BN, A_MN, WG, true, true, false>(maps, p, m_tiles * tiles, g.plan, s);
        if (!g.out_f32 && g.P > kLongRows) return launch<CG, BN, A_MN, WG, false, false, true>(maps, p, m_tiles * tiles, g.plan, s);
    }
    if (g.out_f32) return launch<CG, BN, A_MN, WG, true, false, false>(maps, p, m_tiles * tiles, g.plan, s);
    return launch<CG, BN, A_MN, WG, false, false, false>(maps, p, m_tiles * tiles, g.plan, s);
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
    p.status = g.status;
    injected_stall(&p.wait_ns, &p.skip_producer);
    const bool wg = g.form == kGroupWgrad, fw = g.form == kGroupForward;
    p.M = fw ? g.N : g.K;
    p.N = g.N;
    p.R = fw ? g.K : g.N;
    // The tile's extent along the rows, by the rows per expert that has any. Measured on 256 experts
    // of 1024 x 2048 (forward, us, with 32 / 128 / 256 = a pair of CTAs): 12 rows 162 / 165 / 165, 32
    // rows 184 / 171 / 170, 96 rows 403 / 191 / 185, 256 rows 959 / 328 / 235. Where the pairs' tiles
    // leave most SMs idle, smaller tiles and a shared contraction win: one expert of 2048 x 2048 with
    // 192 rows 11.9 / 9.6 / 13.1.
    const int64_t per = g.P / (g.E < g.P ? g.E : g.P);
    const int64_t pairs = (p.M + 255) / 256 * (g.P / 256 + (g.E < g.P ? g.E : g.P));
    const int bn = wg ? 256 : per <= 24 ? 32 : p.M <= kTileM || 4 * pairs < sm_count() ? 128 : 256;
    const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
    CUtensorMap maps[2];
    bool ok = true;
    if (g.plan) {  // nothing to read
    } else if (wg) {  // A: x [P][K] read along k; B: dy [P][N] read along n
        ok = make_tensor_map_2d(&maps[0], bf, g.x, g.K, g.P, 2 * (uint64_t)g.ld_x, 64, kStep, sw) &&
             make_tensor_map_2d(&maps[1], bf, g.dy, g.N, g.P, 2 * (uint64_t)g.ld_dy, 64, kStep, sw);
    } else {   // A: w [E][N][K]; B: x [P][K] or dy [P][N]
        ok = make_tensor_map_3d(&maps[0], bf, g.w, g.K, g.N, g.E, 2 * (uint64_t)g.K, 2 * (uint64_t)g.K * g.N, 64,
                                fw ? kTileM : kStep, sw) &&
             make_tensor_map_2d(&maps[1], bf, fw ? g.x : g.dy, fw ? g.K : g.N, g.P, 2 * (uint64_t)(fw ? g.ld_x : g.ld_dy), 64,
                                bn <= 32 ? Ring<1, 32, false>::box_rows : Ring<1, 128, false>::box_rows, sw);
    }
    if (!ok) return cudaErrorInvalidValue;
    if (wg) {
        // Pairs, unless their tiles leave more than half of the SMs idle: then single CTAs that share
        // the rows (fp32, pairs / shared, us: one expert of 256 x 2048 with 8192 rows 53.6 / 22.2, 1024
        // x 2048 with 1999 rows 19.2 / 17.0; 8 of 512 x 512 with 128 rows each, too few to share, 7.6 / 7.3).
        // Nor with one or two stages a unit, where a pair's shared operand saves little, if there are so
        // few units that the counter and its memset are a tenth of the time (fp32, pairs / single, us:
        // 128 of 640 x 512 with 19 rows each 43.7 / 35.6, with 94 46.5 / 38.9; 256 of 264 x 320 with 36
        // 45.6 / 31.4; but 64 of 1024 x 1024, Zipf, 256 on average 89.2 / 103.7), or if the output is bf16,
        // whose units are too short to hide a pair's handshakes (256 of 1024 x 2048 with 16 rows 246 /
        // 214, with 64 263 / 230; fp32 350 / 371; nearly all experts empty, where the counter helps,
        // bf16 85 / 101).
        const int64_t tiles = (int64_t)g.E * ((g.N + 255) / 256) * ((g.K + 255) / 256);
        const bool few = 4 * tiles < sm_count(), small = g.P / g.E < 2 * kStep;
        const bool quick = small && (tiles <= 8 * sm_count() || (!g.out_f32 && g.P / g.E >= 8));
        return p.M <= kTileM || few || quick ? launch_typed<1, 256, true, true>(g, maps, p, s)
                                             : launch_typed<2, 256, true, true>(g, maps, p, s);
    }
    if (fw) {
        if (bn == 32) return launch_typed<1, 32, false, false>(g, maps, p, s);
        if (bn == 128) return launch_typed<1, 128, false, false>(g, maps, p, s);
        return launch_typed<2, 256, false, false>(g, maps, p, s);
    }
    if (bn == 32) return launch_typed<1, 32, true, false>(g, maps, p, s);
    if (bn == 128) return launch_typed<1, 128, true, false>(g, maps, p, s);
    return launch_typed<2, 256, true, false>(g, maps, p, s);
}

}  // namespace ftmoe
