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

}  // namespace grp
}  // namespace ftmoe
