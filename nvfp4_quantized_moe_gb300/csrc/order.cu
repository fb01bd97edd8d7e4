// Tokens sorted by expert and back. Slot s = t k + j is token t's j-th expert; slot[p] is the slot of the sorted row p
// (ft_moe_align with block = 1) and pos[s] the row of slot s, its inverse:
//
//   dispatch            out[p] = x[slot[p] / k], block scales and row weights along, pos
//   dispatch backward   dx[t] = sum_j dout[pos[t k + j]],   dw[s] = drow_w[pos[s]]
//   combine             out[t] = add[t] + sum_j w[s] y[pos[s]]
//   combine backward    dy[pos[s]] = w[s] dout[t],   dw[s] = <dout[t], y[pos[s]]>
//
// Bound by memory: k rows are read for one that is written, or the other way round, each once; what repeats (a
// token's row on its way to k experts) repeats in L2. Sums run over j in order, in fp32, and every output element is
// written by one thread, so that results do not change from run to run. A row number out of range (a slot that no
// row holds, a padding row) is skipped or read as zero: no value of slot or pos makes a kernel leave its arrays.
//
// Measured on one GB300, 8192 tokens of 2048 bf16 columns to 8 experts each (Zipf): dispatch with positions and weights
// (302 MB, most of it written) 52.7 us, 5.7 TB/s; in 8 bits with block scales 27.8 us; combine with added rows 58 us (50
// without) and dispatch's backward 51 us (5.8 TB/s, read); combine's backward with the weights' gradients (570 MB) 85 us,
// 6.7 TB/s. 64 tokens: 3 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ftmoe_device.cuh"
#include "ftmoe_internal.h"
#include "row_ops.cuh"

namespace ftmoe {

using namespace rows;

namespace {

constexpr int kOrderThreads = 256;
// Up to this many slots one CTA clears and fills pos by itself; above, a memset goes before the launch.
constexpr int kPosByOneCta = 2048;
// Sorted rows beyond this many bytes, which L2 cannot hold, leave as streaming stores: 65536 rows of 4 KB 52.7 us,
// as plain ones 58.2.
constexpr int64_t kStreamBytes = 100 << 20;

__device__ __forceinline__ int rows_of(const DispatchParams &p)
{
    return p.count ? min(max(__ldg(p.count), 0), p.P) : p.P;
}

// What the first p.small CTAs of a dispatch carry: positions, row weights, block scales.
__device__ __forceinline__ void dispatch_small(const DispatchParams &p, int n)
{
    const int slots = p.T * p.k;
    // positions: cleared and filled by the first CTA alone, or, cleared before the launch, by all
    const int me = blockIdx.x * kOrderThreads + threadIdx.x, threads = p.small * kOrderThreads;
    if (p.pos && p.clear && blockIdx.x == 0) {
        for (int i = threadIdx.x; i < slots; i += kOrderThreads) p.pos[i] = -1;
        __syncthreads();
    }
    const bool alone = p.clear;
    if ((p.pos || p.row_w) && (!alone || blockIdx.x == 0))
        for (int r = alone ? threadIdx.x : me; r < n; r += alone ? kOrderThreads : threads) {
            const int s = __ldg(p.slot + r);
            const bool in = s >= 0 && s < slots;
            if (p.pos && in) atomicMax(p.pos + s, r);
            if (p.row_w) p.row_w[r] = in ? __ldg(p.w + s) : 0.f;
        }
    // block scales: a thread takes up to eight blocks of a row, all loads in flight; neighbours take neighbouring rows
    const int groups = (p.blocks + 7) / 8;
    for (int64_t i = me; i < (int64_t)groups * p.P; i += threads) {
        const int g = (int)(i / p.P), r = (int)(i - (int64_t)g * p.P);
        if (r >= n) continue;
        const int s = __ldg(p.slot + r);
        const bool in = s >= 0 && s < slots;
        const uint32_t *from = p.x_scale + (int64_t)8 * g * p.ld_xs + (in ? s / p.k : 0);
        uint32_t *to = p.out_scale + (int64_t)8 * g * p.ld_os + r;
        uint32_t v[8];
#pragma unroll
        for (int b = 0; b < 8; ++b) v[b] = in && 8 * g + b < p.blocks ? __ldg(from + b * p.ld_xs) : 0u;
#pragma unroll
        for (int b = 0; b < 8; ++b)
            if (8 * g + b < p.blocks) to[b * p.ld_os] = v[b];
    }
}

}  // namespace

// The first `small` CTAs carry what is small (positions, row weights, block scales), the others the rows: a warp
// takes 32 x kUnits pieces of T (16, 4 or 2 bytes, the largest that rows are made of) of one row at a time.
template <typename T, int kUnits>
__global__ void __launch_bounds__(kOrderThreads) dispatch_kernel(const __grid_constant__ DispatchParams p)
{
    pdl_enter();
    const int n = rows_of(p), slots = p.T * p.k;
    if ((int)blockIdx.x < p.small) {
        dispatch_small(p, n);
        return;
    }
    const int lane = threadIdx.x & 31;
    const int pieces = p.row_bytes / (int)sizeof(T), chunks = (pieces + 32 * kUnits - 1) / (32 * kUnits);
    const int64_t units = (int64_t)n * chunks;
    const int64_t step = (int64_t)(gridDim.x - p.small) * (kOrderThreads / 32);
    for (int64_t u = (int64_t)(blockIdx.x - p.small) * (kOrderThreads / 32) + (threadIdx.x >> 5); u < units; u += step) {
        const int r = (int)(u / chunks), c0 = (int)(u - (int64_t)r * chunks) * 32 * kUnits + lane;
        const int s = __ldg(p.slot + r);
        const bool in = s >= 0 && s < slots;
        const T *from = reinterpret_cast<const T *>(p.x + (in ? s / p.k : 0) * p.ld_x);
        T *to = reinterpret_cast<T *>(p.out + r * p.ld_out);
        T v[kUnits];
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            v[i] = T{};
            if (in && c0 + 32 * i < pieces) v[i] = __ldg(from + c0 + 32 * i);
        }
#pragma unroll
        for (int i = 0; i < kUnits; ++i)
            if (c0 + 32 * i < pieces) {
                if (p.stream) __stcs(to + c0 + 32 * i, v[i]);
                else to[c0 + 32 * i] = v[i];
            }
    }
}

// Rows of at most 16 pieces: p.team threads (a power of two) per row, so that a warp takes several (65536 rows of 24 bf16:
// 5.9 us, a warp each 14.5).
template <typename T>
__global__ void __launch_bounds__(kOrderThreads) dispatch_narrow_kernel(const __grid_constant__ DispatchParams p)
{
    pdl_enter();
    const int n = rows_of(p), slots = p.T * p.k;
    if ((int)blockIdx.x < p.small) {
        dispatch_small(p, n);
        return;
    }
    const int per = kOrderThreads / p.team, c = threadIdx.x & (p.team - 1);
    const bool live = c < p.row_bytes / (int)sizeof(T);
    const int64_t step = (int64_t)(gridDim.x - p.small) * per;
    for (int64_t r = (int64_t)(blockIdx.x - p.small) * per + threadIdx.x / p.team; r < n; r += step) {
        const int s = __ldg(p.slot + r);
        T v = T{};
        if (live && s >= 0 && s < slots) v = __ldg(reinterpret_cast<const T *>(p.x + s / p.k * p.ld_x) + c);
        if (live) reinterpret_cast<T *>(p.out + r * p.ld_out)[c] = v;
    }
}

// 8 values of a row (or one) as they lie in memory. load_own: of an operand that an output of the kernel may be.
template <bool F32, bool VEC>
struct Raw {
    uint4 q[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const char *row, int c)
    {
        const uint4 *p = reinterpret_cast<const uint4 *>(row + c * (F32 ? 4 : 2));
        q[0] = __ldg(p);
        if constexpr (F32) q[1] = __ldg(p + 1);
    }
    __device__ __forceinline__ void load_own(const char *row, int c)
    {
        const uint4 *p = reinterpret_cast<const uint4 *>(row + c * (F32 ? 4 : 2));
        q[0] = ld_own_v4(p);
        if constexpr (F32) q[1] = ld_own_v4(p + 1);
    }
    __device__ __forceinline__ void open(float (&v)[8]) const
    {
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                v[4 * i] = __uint_as_float(q[i].x);
                v[4 * i + 1] = __uint_as_float(q[i].y);
                v[4 * i + 2] = __uint_as_float(q[i].z);
                v[4 * i + 3] = __uint_as_float(q[i].w);
            }
        } else {
            unpack8(q[0], v);
        }
    }
};

template <bool F32>
struct Raw<F32, false> {
    uint32_t q;
    __device__ __forceinline__ void load(const char *row, int c)
    {
        if constexpr (F32) q = __ldg(reinterpret_cast<const uint32_t *>(row) + c);
        else q = (uint32_t)__ldg(reinterpret_cast<const uint16_t *>(row) + c) << 16;
    }
    __device__ __forceinline__ void load_own(const char *row, int c)
    {
        if constexpr (F32) q = reinterpret_cast<const uint32_t *>(row)[c];
        else q = (uint32_t)reinterpret_cast<const uint16_t *>(row)[c] << 16;
    }
    __device__ __forceinline__ void open(float (&v)[1]) const { v[0] = __uint_as_float(q); }
};

// Combine, and the backward of dispatch (no weights): p.team threads per token (a power of two), 8 columns each (or four,
// apart, where rows are not made of 16-byte pieces), the loads of several rows in flight together. They stay as they lie
// in memory until all are issued: widened to fp32 at once, eight rows took 90 registers a thread, and two CTAs an SM were
// too few (8192 tokens of 2048 columns, top 8, bf16: 162 us, now 59). WIDE: a CTA per token, known to the compiler (67 us
// otherwise); narrow rows share a CTA (24 columns: 3.8 us, a CTA each 23).
template <bool YF32, bool OF32, bool VEC, bool WIDE>
__global__ void __launch_bounds__(kOrderThreads) combine_rows_kernel(const __grid_constant__ CombineParams p)
{
    constexpr int W = VEC ? 8 : 1, J = YF32 ? 4 : 8, C = VEC ? 1 : 4;
    pdl_enter();
    const int team = WIDE ? kOrderThreads : p.team, me = threadIdx.x & (team - 1);
    const int64_t t = (int64_t)blockIdx.x * (kOrderThreads / team) + threadIdx.x / team;
    if (t >= p.T) return;
    const int *pos = p.pos + t * p.k;
    const float *w = p.w ? p.w + t * p.k : nullptr;
    if (p.dw && blockIdx.y == 0)
        for (int j = me; j < p.k; j += team) {
            const int r = __ldg(pos + j);
            p.dw[t * p.k + j] = r >= 0 && r < p.P ? __ldg(p.drow_w + r) : 0.f;
        }
    const int c0 = W * (blockIdx.y * C * team + me);
    if (c0 >= p.H) return;
    float acc[C][W] = {};
    for (int j0 = 0; j0 < p.k; j0 += J) {
        Raw<YF32, VEC> v[J][C] = {};
        float f[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            f[j] = 0.f;
            if (j0 + j < p.k) {
                const int r = __ldg(pos + j0 + j);
                if (r >= 0 && r < p.P) {
                    f[j] = w ? __ldg(w + j0 + j) : 1.f;
#pragma unroll
                    for (int n = 0; n < C; ++n)
                        if (c0 + n * team < p.H)
                            v[j][n].load(static_cast<const char *>(p.y) + r * p.ld_y * (YF32 ? 4 : 2), c0 + n * team);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int n = 0; n < C; ++n) {
                float a[W];
                v[j][n].open(a);
#pragma unroll
                for (int i = 0; i < W; ++i) acc[n][i] = fmaf(f[j], a[i], acc[n][i]);
            }
    }
    const int size = OF32 ? 4 : 2;
    char *out = static_cast<char *>(p.out) + t * p.ld_out * size;
    Raw<OF32, VEC> add[C] = {};  // (all loads before the first store: add may be out)
    if (p.add) {
#pragma unroll
        for (int n = 0; n < C; ++n)
            if (c0 + n * team < p.H) add[n].load_own(static_cast<const char *>(p.add) + t * p.ld_add * size, c0 + n * team);
    }
#pragma unroll
    for (int n = 0; n < C; ++n) {
        const int c = c0 + n * team;
        if (c >= p.H) break;
        if (p.add) {
            float a[W];
            add[n].open(a);
#pragma unroll
            for (int i = 0; i < W; ++i) acc[n][i] += a[i];
        }
        if constexpr (VEC) {
            if constexpr (OF32) {
                float4 *o = reinterpret_cast<float4 *>(reinterpret_cast<float *>(out) + c);
                o[0] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
                o[1] = make_float4(acc[n][4], acc[n][5], acc[n][6], acc[n][7]);
            } else {
                *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(out) + c) = pack8(acc[n]);
            }
        } else if constexpr (OF32) {
            reinterpret_cast<float *>(out)[c] = acc[n][0];
        } else {
            reinterpret_cast<uint16_t *>(out)[c] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[n][0]));
        }
    }
}

// Elements from the last 32 x T boundary of memory to `p`: a warp that stores an element a lane begins there, so that its
// stores are whole sectors (combine's backward, 65536 rows of 2047 bf16: 235 us without this, 210 with it). Vectors are
// aligned as they are.
template <bool VEC, typename T>
__device__ __forceinline__ int lead(const T *p)
{
    return VEC ? 0 : (int)(reinterpret_cast<uintptr_t>(p) / sizeof(T) % 32);
}

// One warp per slot (neighbouring warps share a token, whose row then comes from L1).
template <bool DF32, bool YF32, bool VEC>
__global__ void __launch_bounds__(kOrderThreads) combine_backward_kernel(const __grid_constant__ CombineBackParams p)
{
    constexpr int W = VEC ? 8 : 1, U = VEC ? 4 : 8;
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t slots = (int64_t)p.T * p.k, step = (int64_t)gridDim.x * (kOrderThreads / 32);
    for (int64_t s = (int64_t)blockIdx.x * (kOrderThreads / 32) + (threadIdx.x >> 5); s < slots; s += step) {
        const int r = __ldg(p.pos + s);
        const bool in = r >= 0 && r < p.P;
        if (!in) {
            if (p.dw && lane == 0) p.dw[s] = 0.f;
            continue;
        }
        const float f = p.w ? __ldg(p.w + s) : 1.f;
        const char *d = static_cast<const char *>(p.dout) + s / p.k * p.ld_dout * (DF32 ? 4 : 2);
        const char *y = static_cast<const char *>(p.y) + r * p.ld_y * (YF32 ? 4 : 2);
        uint16_t *o = static_cast<uint16_t *>(p.dy) + r * p.ld_dy;
        float sum = 0.f;
        for (int c0 = W * lane - lead<VEC>(o); c0 < p.H; c0 += 32 * W * U) {
            Raw<DF32, VEC> a[U];
            Raw<YF32, VEC> b[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int c = c0 + 32 * W * i;
                if (c >= 0 && c < p.H && p.dw) b[i].load(y, c);
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int c = c0 + 32 * W * i;
                if (c >= 0 && c < p.H) a[i].load(d, c);
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int c = c0 + 32 * W * i;
                if (c < 0 || c >= p.H) continue;
                float u[W], v[W];
                a[i].open(u);
                if (p.dw) {
                    b[i].open(v);
#pragma unroll
                    for (int j = 0; j < W; ++j) sum = fmaf(u[j], v[j], sum);
                }
#pragma unroll
                for (int j = 0; j < W; ++j) u[j] *= f;
                if constexpr (VEC) *reinterpret_cast<uint4 *>(o + c) = pack8(u);
                else o[c] = __bfloat16_as_ushort(__float2bfloat16_rn(u[0]));
            }
        }
        if (p.dw) {
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, m);
            if (lane == 0) p.dw[s] = sum;
        }
    }
}

namespace {

using CombineKernel = void (*)(CombineParams);
template <bool... Known>
CombineKernel combine_kernel()
{
    return combine_rows_kernel<Known...>;
}
template <bool... Known, typename... Rest>
CombineKernel combine_kernel(bool next, Rest... rest)
{
    return next ? combine_kernel<Known..., true>(rest...) : combine_kernel<Known..., false>(rest...);
}

bool vec16(const void *p, int64_t row_bytes) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && row_bytes % 16 == 0; }

}  // namespace

cudaError_t launch_dispatch(DispatchParams p, cudaStream_t s)
{
    const int slots = p.T * p.k;
    p.clear = slots <= kPosByOneCta && p.P <= kPosByOneCta;
    p.stream = (int64_t)p.P * p.row_bytes > kStreamBytes;
    if (p.pos && !p.clear) {
        const cudaError_t e = cudaMemsetAsync(p.pos, 0xFF, sizeof(int) * (size_t)slots, s);
        if (e != cudaSuccess) return e;
    }
    const int per = kOrderThreads / 32;
    const auto made_of = [&](int n) {
        return p.row_bytes % n == 0 && p.ld_x % n == 0 && p.ld_out % n == 0 && reinterpret_cast<uintptr_t>(p.x) % n == 0 &&
               reinterpret_cast<uintptr_t>(p.out) % n == 0;
    };
    const int piece = made_of(16) ? 16 : made_of(4) ? 4 : 2, unit = piece == 16 ? 4 : piece == 4 ? 8 : 16;
    const int chunks = (p.row_bytes / piece + 32 * unit - 1) / (32 * unit);
    const int64_t want = ((int64_t)p.P * chunks + per - 1) / per, most = (int64_t)sm_count() * 32;
    // CTAs for what is small: a thread per slot or eight scales, up to four CTAs per SM
    const int64_t items = (int64_t)p.P * (p.blocks > 0 ? (p.blocks + 7) / 8 : 1), each = (items + kOrderThreads - 1) / kOrderThreads;
    p.small = 0;
    if (p.pos || p.row_w || p.blocks) p.small = p.clear && !p.blocks ? 1 : (int)(each < 4 * sm_count() ? each : 4 * sm_count());
    const int pieces = p.row_bytes / piece;
    if (pieces <= 16) {
        p.team = 1;
        while (p.team < pieces) p.team *= 2;
        const int rows = kOrderThreads / p.team;
        const int64_t ctas = ((int64_t)p.P + rows - 1) / rows;
        auto narrow = piece == 16 ? dispatch_narrow_kernel<uint4> : piece == 4 ? dispatch_narrow_kernel<uint32_t>
                                                                            : dispatch_narrow_kernel<uint16_t>;
        FT_LAUNCH(narrow, dim3((unsigned)(ctas < most ? ctas : most) + p.small), dim3(kOrderThreads), 0, s, p);
        count_launches(1);
        return cudaGetLastError();
    }
    const unsigned grid = (unsigned)(want < most ? want : most) + p.small;
    auto kern = piece == 16 ? dispatch_kernel<uint4, 4> : piece == 4 ? dispatch_kernel<uint32_t, 8> : dispatch_kernel<uint16_t, 16>;
    FT_LAUNCH(kern, dim3(grid), dim3(kOrderThreads), 0, s, p);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_combine_rows(CombineParams p, bool y_f32, bool out_f32, cudaStream_t s)
{
    const int ys = y_f32 ? 4 : 2, os = out_f32 ? 4 : 2;
    const bool vec = p.H % 8 == 0 && vec16(p.y, p.ld_y * ys) && vec16(p.out, p.ld_out * os) && vec16(p.add, p.ld_add * os);
    const int each = vec ? 8 : 4;  // columns of a thread
    p.team = 1;
    while (p.team < kOrderThreads && p.team * each < p.H) p.team *= 2;
    const int tokens = kOrderThreads / p.team, cols = p.team * each;
    const dim3 grid((p.T + tokens - 1) / tokens, (p.H + cols - 1) / cols);
    const bool wide = p.team == kOrderThreads;
    auto kern = combine_kernel(y_f32, out_f32, vec, wide);
    FT_LAUNCH(kern, grid, dim3(kOrderThreads), 0, s, p);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_combine_backward(const CombineBackParams &p, bool dout_f32, bool y_f32, cudaStream_t s)
{
    const int ds = dout_f32 ? 4 : 2, ys = y_f32 ? 4 : 2;
    const bool vec = p.H % 8 == 0 && vec16(p.dout, p.ld_dout * ds) && vec16(p.dy, p.ld_dy * 2) &&
                     (!p.dw || vec16(p.y, p.ld_y * ys));
    const int64_t want = ((int64_t)p.T * p.k + kOrderThreads / 32 - 1) / (kOrderThreads / 32), most = (int64_t)sm_count() * 32;
    auto kern = dout_f32 ? (y_f32 ? (vec ? combine_backward_kernel<true, true, true> : combine_backward_kernel<true, true, false>)
                                  : (vec ? combine_backward_kernel<true, false, true> : combine_backward_kernel<true, false, false>))
                         : (y_f32 ? (vec ? combine_backward_kernel<false, true, true> : combine_backward_kernel<false, true, false>)
                                  : (vec ? combine_backward_kernel<false, false, true> : combine_backward_kernel<false, false, false>));
    FT_LAUNCH(kern, dim3((unsigned)(want < most ? want : most)), dim3(kOrderThreads), 0, s, p);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace ftmoe
