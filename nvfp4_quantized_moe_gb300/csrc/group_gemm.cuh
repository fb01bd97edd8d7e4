// Shared parts of the grouped products over ragged expert batches (group_gemm.cu,
// group_gemm_fp8.cu): the table of the experts' rows in shared memory, the list of output tiles
// it gives, and the inline PTX that one CTA or a pair of CTAs needs beyond tcgen05.cuh.
//
// Orientation. The tensor cores compute D[M = 128 lanes][N columns]. The wide, regular axis of
// the output (the weight rows) lies along M and the ragged one (an expert's rows) along N, whose
// size per instruction is any multiple of 16: a batch of 5 rows costs a 16-column instruction
// instead of a 128-row one, and the tail of an expert's batch is not padded to a tile.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ftmoe_device.cuh"
#include "ftmoe_internal.h"
#include "tcgen05.cuh"

namespace ftmoe {
namespace grp {

constexpr int kTileM = 128;          // weight rows of one CTA's tile (TMEM lanes)
constexpr int kChunkBytes = 128;     // bytes of the contraction axis per stage (the swizzle width)
constexpr int kABytes = kTileM * kChunkBytes;

// Shared memory of the experts' table. The limit of a kernel's shared memory belongs to the kernel,
// not to a call: it is always set to what kGroupMaxExperts need, so that calls with unlike numbers of
// experts, made by several threads at once, do not lower it for each other.
constexpr size_t table_bytes(int E) { return 4 * 2 * ((size_t)E + 1); }

// ---------------------------------------------------------------- issuing warps
//
// One thread issues the copies and the MMAs, but its whole warp runs the loop around them: their
// operands live in registers that a warp shares, and only where the compiler sees that a value is
// the same in all lanes does it keep the value there. In a branch of lane 0 alone every operand of
// every instruction was moved over first: 94 cycles per MMA, and 700 per stage of four that the
// tensor cores finish in 512.

__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// ---------------------------------------------------------------- clusters

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// shared::cluster address of `p`'s counterpart in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(const void *p, uint32_t rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// The same without ordering this thread's earlier memory accesses (a release at cluster scope waits
// for all of them: half a microsecond per arrival in the pipelines here). For arrivals that hand
// over tensor memory, whose reads tcgen05.wait::ld has completed.
__device__ __forceinline__ void arrive_cluster_relaxed(uint32_t bar)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// mbar_wait_timed whose success also orders what other CTAs of the cluster released.
__device__ __forceinline__ bool wait_cluster(uint64_t *bar, uint32_t parity, volatile int *abort_flag, uint64_t limit_ns)
{
    auto poll = [&]() {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity), "r"(kSuspendHintNs)
            : "memory");
        return ok != 0;
    };
    if (poll()) return true;
    const uint64_t t0 = globaltimer();
    for (;;) {
        if (poll()) return true;
        if (abort_flag && *abort_flag) return false;
        if (globaltimer() - t0 > limit_ns) return false;
    }
}

// All lanes of a warp wait; the answer is the same in every lane.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag, uint64_t limit_ns)
{
    const bool ok = wait_cluster(bar, parity, abort_flag, limit_ns);
    return __all_sync(0xFFFFFFFFu, ok);
}

// ---------------------------------------------------------------- tcgen05 for one CTA or a pair

template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t *dst, uint32_t ncols)
{
    if constexpr (CG == 1) {
        tc::tmem_alloc(dst, ncols);
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}

template <int CG>
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols)
{
    if constexpr (CG == 1) {
        tc::tmem_dealloc(taddr, ncols);
    } else {
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
    }
}

// Arrive on `bar` (for a pair: on both CTAs' `bar`) once every MMA issued so far by this
// thread has completed.
template <int CG>
__device__ __forceinline__ void commit(uint64_t *bar)
{
    if constexpr (CG == 1) {
        tc::commit(bar);
    } else {
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_u32(bar)),
            "h"((uint16_t)3)
            : "memory");
    }
}

// Tiled TMA loads into this CTA's shared memory that signal the barrier at the shared::cluster
// address `bar` (of this CTA, or for a pair of either).
template <int CG>
__device__ __forceinline__ void load_2d(void *dst, const CUtensorMap *map, int c0, int c1, uint32_t bar)
{
    if constexpr (CG == 1) {
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
            "[%4];" ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar) : "memory");
    } else {
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
            "[%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
            : "memory");
    }
}

template <int CG>
__device__ __forceinline__ void load_3d(void *dst, const CUtensorMap *map, int c0, int c1, int c2, uint32_t bar)
{
    if constexpr (CG == 1) {
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
            "[%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1),
            "r"(c2), "r"(bar) : "memory");
    } else {
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
            "[%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1),
            "r"(c2), "r"(bar) : "memory");
    }
}

// Shared-memory descriptor of an operand whose contraction axis is NOT contiguous: boxes of 64
// 16-bit elements (128 bytes, 128-byte swizzle) by 64 contraction steps, 8 KB apart (leading
// byte offset); 8 contraction steps are 1024 bytes (stride byte offset).
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t smem_addr)
{
    uint64_t d = 0;
    d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(8192 >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// W consecutive 32-bit columns of this thread's TMEM lane.
template <int W>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&v)[W])
{
    if constexpr (W == 32) tc::ld32(addr, v);
    else tc::ld16(addr, v);
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}

// ---------------------------------------------------------------- stores

// *to += v, without waiting for what it holds. Each element gets one such addition in a launch, so
// that there is no order to depend on. (The addition in L2 takes subnormal values for zero.)
__device__ __forceinline__ void add_global(float *to, float v)
{
    asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(to), "f"(v) : "memory");
}

// W columns of a tile whose lane is the M index m: columns are the rows row0, row0 + 1, ... of
// `out` (`rows` of them at most), m (< M) is the place in the row. Called by whole warps.
// bf16 rows with pairs (M even, every row 4-byte aligned): neighbouring lanes trade one value each,
// so that a lane holds two neighbours of one row and a store covers two rows.
template <bool F32, int W, bool PAIRS = true>
__device__ __forceinline__ void store_rows(const float (&v)[W], int m, int M, int64_t row0, int rows, void *out, int64_t ld,
                                           bool accumulate = false)
{
    if constexpr (F32) {
        const int n = m < M ? rows : 0;
        float *o = static_cast<float *>(out) + row0 * ld + m;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            if (j < n) {
                if (accumulate) add_global(o, v[j]);
                else *o = v[j];
            }
            o += ld;
        }
    } else if constexpr (PAIRS) {
        const int odd = m & 1, n = m < M ? rows - odd : 0;
        uint16_t *o = static_cast<uint16_t *>(out) + (row0 + odd) * ld + (m - odd);
#pragma unroll
        for (int j = 0; j < W; j += 2) {
            const uint32_t a = bf16x2(v[j], v[j + 1]), b = __shfl_xor_sync(0xFFFFFFFFu, a, 1);
            if (j < n) *reinterpret_cast<uint32_t *>(o) = __byte_perm(a, b, odd ? 0x3276 : 0x5410);
            o += 2 * ld;
        }
    } else {
        const int n = m < M ? rows : 0;
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(out) + row0 * ld + m;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            if (j < n) *o = __float2bfloat16_rn(v[j]);
            o += ld;
        }
    }
}

// The sums of a tile whose contraction the `split` CTAs of a cluster shared: each left its part in
// its own `red` [cols][128]; the CTAs add and store a share of the elements each (or add them to
// out), parts always in the same order. Between two cluster barriers, by all threads.
template <bool F32>
__device__ __forceinline__ void add_parts(const float *red, int cols, int m0, int M, int64_t row0, void *out, int64_t ld,
                                          int split, int part, bool accumulate = false)
{
    constexpr int kMax = 8;
    // four neighbours of one row at a time, all parts' loads in flight together
    for (int i = 4 * (threadIdx.x + blockDim.x * part); i < cols * kTileM; i += 4 * blockDim.x * split) {
        float4 v[kMax];
#pragma unroll
        for (int r = 0; r < kMax; ++r)
            if (r < split)
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(v[r].x), "=f"(v[r].y), "=f"(v[r].z), "=f"(v[r].w)
                             : "r"(map_rank(red + i, r))
                             : "memory");
        float4 a = v[0];
#pragma unroll
        for (int r = 1; r < kMax; ++r)
            if (r < split) { a.x += v[r].x; a.y += v[r].y; a.z += v[r].z; a.w += v[r].w; }
        const int m = m0 + i % kTileM;
        const int64_t at = (row0 + i / kTileM) * ld + m;
        const float o[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (m + j < M) {
                if constexpr (F32) {
                    if (accumulate) add_global(static_cast<float *>(out) + at + j, o[j]);
                    else static_cast<float *>(out)[at + j] = o[j];
                } else static_cast<__nv_bfloat16 *>(out)[at + j] = __float2bfloat16_rn(o[j]);
            }
    }
}

// ---------------------------------------------------------------- the experts' rows

// Tiles of one launch. An expert's n rows are cut into ceil(n / BN) tiles of equal length
// (rounded up to `gran`), so that no tile is a thin remainder.
struct Tile {
    int e;      // expert
    int row0;   // first row of the tile
    int rows;   // its rows
};

// Offsets of the experts (clamped into [0, P], never decreasing inside an expert) and the
// running count of their tiles, in shared memory: [E + 1] ints each. Run by all threads.
// Returns whether the offsets were valid. `sh_flag` is one int of shared memory.
__device__ __forceinline__ bool build_table(const int *offs, int E, int P, int BN, int *sh_offs, int *sh_tiles, int *sh_flag)
{
    if (threadIdx.x == 0) *sh_flag = 0;
    __syncthreads();
    for (int i = threadIdx.x; i <= E; i += blockDim.x) {
        const int v = offs ? __ldg(offs + i) : (i ? P : 0);
        sh_offs[i] = min(max(v, 0), P);
        bool bad = v < 0 || v > P;
        if (i < E && offs) bad |= __ldg(offs + i + 1) < v;
        if (bad) *sh_flag = 1;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        int base = 0;
        for (int i0 = 0; i0 < E; i0 += 32) {
            const int i = i0 + threadIdx.x;
            int t = i < E ? (max(sh_offs[i + 1] - sh_offs[i], 0) + BN - 1) / BN : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xFFFFFFFFu, t, d);
                if ((int)threadIdx.x >= d) t += o;
            }
            if (i < E) sh_tiles[i + 1] = base + t;
            base += __shfl_sync(0xFFFFFFFFu, t, 31);
        }
        if (threadIdx.x == 0) sh_tiles[0] = 0;
    }
    __syncthreads();
    return *sh_flag == 0;
}

__device__ __forceinline__ Tile find_tile(int t, int E, int BN, int gran, const int *sh_offs, const int *sh_tiles)
{
    int lo = 0, hi = E;  // sh_tiles[lo] <= t < sh_tiles[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sh_tiles[mid] <= t) lo = mid;
        else hi = mid;
    }
    const int n = sh_offs[lo + 1] - sh_offs[lo], nt = (n + BN - 1) / BN, j = t - sh_tiles[lo];
    const int len = ((n + nt - 1) / nt + gran - 1) / gran * gran;
    Tile r;
    r.e = lo;
    r.row0 = sh_offs[lo] + j * len;
    r.rows = max(min(len, n - j * len), 0);
    return r;
}

// ---------------------------------------------------------------- the same table, with one barrier
//
// For kernels one warp of which looks tiles up: every warp finds what lies before its own experts by itself, so that one
// barrier is all that the table takes (the caller synchronises before it is used), and a warp finds a tile's expert
// with two ballots. Tiles begin at multiples of ALIGN rows (find_aligned_tile). Returns whether the offsets were valid; if
// not, there are no tiles (ranges that overlap could be E times the work, and more units than a launch is made for).
// (In the 8-bit product's wide kernel this costs registers that it does not have: 80 us instead of 75 for 4096^3.)
template <int ALIGN>
__device__ __forceinline__ bool build_tiles(const int *offs, int E, int P, int BN, int *sh_offs, int *sh_tiles)
{
    bool bad = false;
    for (int i = threadIdx.x; i <= E; i += blockDim.x) {
        const int v = offs ? __ldg(offs + i) : (i ? P : 0), next = offs && i < E ? __ldg(offs + i + 1) : v;
        sh_offs[i] = min(max(v, 0), P);
        bad |= v < 0 || v > P || (offs && next < v);
    }
    const bool valid = !__syncthreads_or(bad);
    auto tiles = [&](int i) {
        const int first = sh_offs[i], last = sh_offs[i + 1];
        return valid && last > first ? (last - (ALIGN > 1 ? first / ALIGN * ALIGN : first) + BN - 1) / BN : 0;
    };
    const int lane = threadIdx.x & 31, warps = blockDim.x / 32;
    for (int i0 = 32 * (threadIdx.x >> 5); i0 < E; i0 += 32 * warps) {
        int base = 0;
        for (int i = lane; i < i0; i += 32) base += tiles(i);
        base = __reduce_add_sync(0xFFFFFFFFu, base);
        const int i = i0 + lane;
        int t = i < E ? tiles(i) : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xFFFFFFFFu, t, d);
            if (lane >= d) t += o;
        }
        if (i < E) sh_tiles[i + 1] = base + t;
    }
    if (threadIdx.x == 0) sh_tiles[0] = 0;
    return valid;
}

// Tile t, of expert e.
__device__ __forceinline__ Tile tile_of(int t, int e, int BN, int gran, const int *sh_offs, const int *sh_tiles)
{
    const int n = sh_offs[e + 1] - sh_offs[e], nt = (n + BN - 1) / BN, j = t - sh_tiles[e];
    const int len = ((n + nt - 1) / nt + gran - 1) / gran * gran;
    Tile r;
    r.e = e;
    r.row0 = sh_offs[e] + j * len;
    r.rows = max(min(len, n - j * len), 0);
    return r;
}

// The expert of tile t, by a whole warp: the last one whose running count is t or less.
__device__ __forceinline__ int expert_of(int t, int E, const int *sh_tiles)
{
    const int lane = threadIdx.x & 31;
    const int c = __popc(__ballot_sync(0xFFFFFFFFu, 32 * lane < E && sh_tiles[32 * lane] <= t)) - 1;  // its group of 32
    const int i = 32 * c + lane;
    return 32 * c + __popc(__ballot_sync(0xFFFFFFFFu, i < E && sh_tiles[i] <= t)) - 1;
}

// The same where the first tile of an expert begins at the multiple of ALIGN at or before its first row and the
// others BN rows apart: row0 may lie before the expert's rows [first, first + n), which `lo` and `hi` give relative to it.
struct AlignedTile {
    int e, row0, lo, hi;
};

template <int ALIGN>
__device__ __forceinline__ AlignedTile find_aligned_tile(int t, int E, int BN, const int *sh_offs, const int *sh_tiles)
{
    const int lo = expert_of(t, E, sh_tiles);
    AlignedTile r;
    r.e = lo;
    r.row0 = sh_offs[lo] / ALIGN * ALIGN + (t - sh_tiles[lo]) * BN;
    r.lo = max(sh_offs[lo] - r.row0, 0);
    r.hi = min(sh_offs[lo + 1] - r.row0, BN);
    return r;
}

}  // namespace grp
}  // namespace ftmoe
