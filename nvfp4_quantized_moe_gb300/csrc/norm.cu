// Root-mean-square norm of rows in front of an expert layer, with the residual's addition, and its gradient:
//
//   s = x + r (stored in r's type; s = x without a residual)   rstd = (mean s^2 + eps)^(-1/2)
//   y = s rstd (o + w)        into bf16 (the router's and the bf16 products' input), into e4m3 with a scale per
//                             128 columns (the 8-bit products' input), or both
//   dx = ds + rstd (g - n mean(g n))       with n = s rstd, g = dy (o + w), ds the gradient that reaches s past the norm
//   dw = sum over the rows of dy n
//
// Bound by memory: every operand is read once and every result written once. A row stays in registers between
// its sum of squares and its outputs, so that nothing is read twice; sums are fp32. The norm is that of s as it is
// stored, so that the backward pass, which has only the stored s, is the gradient of what was computed.
//
// Measured on one GB300, in a captured graph over inputs larger than L2: 8192 rows of 2048 with a bf16 residual (134 MB)
// 24.0 us, 5.6 TB/s, where a plain copy of as many bytes takes 27.7; 1999 rows of 4096 with an fp32 residual into 8 bits
// (90 MB) 18.5 us; one row 2.4 us. Backward of 8192 rows of 2048 (134 MB) 26.1 us, 5.2 TB/s, and 32.9 with the weight's
// gradient, whose 608 partial sums are written, read and added by a second launch; 64 rows 2.0 and 5.7. Rows that are not
// made of 16-byte pieces go an element at a time: 8192 rows of 2047 40.7 us, backward 56. A whole CTA per row from 257
// columns on, the loads of all of a thread's columns in flight (compared when 2048 columns on 256 threads took 25.7 us: on
// 128 25.8, 64 31.5, 32 38.3; one row 2.6, 3.2, 4.9, 7.5).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ftmoe_device.cuh"
#include "ftmoe_internal.h"
#include "row_ops.cuh"

namespace ftmoe {

using namespace rows;

namespace {

// Sum over the TPR threads of a row, the same in all of them and from run to run. `red` holds one float per warp
// of the CTA; rows of one warp need none. (Sums in turn take two `red` by turns: then one barrier each is enough.)
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *red)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    if constexpr (TPR > 32) {
        constexpr int kWarps = TPR / 32;
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        const int first = threadIdx.x / TPR * kWarps;
        const int lane = threadIdx.x & 31;
        v = lane < kWarps ? red[first + lane] : 0.f;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    }
    return v;
}

// 8 values of a row: VEC: from column c on, by 16-byte loads; else an element at a time, `step` columns apart, up to H.
// OWN: of an operand that an output of the kernel may be (ordinary loads, as ld_own_v4's).
template <bool F32, bool VEC, bool OWN = false>
__device__ __forceinline__ void get8(const void *row, int c, int step, int H, float (&v)[8])
{
    static_assert(!VEC || !OWN, "fetch8");
    if constexpr (VEC) {
        load8<F32>(row, c, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int at = c + i * step;
            const float *f = static_cast<const float *>(row) + at;
            const uint16_t *h = static_cast<const uint16_t *>(row) + at;
            v[i] = 0.f;
            if (at < H)
                v[i] = F32 ? (OWN ? *f : __ldg(f)) : __uint_as_float((uint32_t)(OWN ? *h : __ldg(h)) << 16);
        }
    }
}

template <bool F32, bool VEC>
__device__ __forceinline__ void put8(void *row, int c, int step, int H, const float (&v)[8])
{
    if constexpr (VEC) {
        if constexpr (F32) {
            float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(row) + c);
            p[0] = make_float4(v[0], v[1], v[2], v[3]);
            p[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(row) + c) = pack8(v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i * step < H) {
                if (F32) static_cast<float *>(row)[c + i * step] = v[i];
                else static_cast<uint16_t *>(row)[c + i * step] = __bfloat16_as_ushort(__float2bfloat16_rn(v[i]));
            }
    }
}

// o + w for 8 columns.
template <bool VEC>
__device__ __forceinline__ void gain8(const void *w, bool f32, float offset, int c, int step, int H, float (&g)[8])
{
    if (f32) get8<true, VEC>(w, c, step, H, g);
    else get8<false, VEC>(w, c, step, H, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] += offset;
}

// 8 values as they lie in memory. OWN: of an operand that an output of the kernel may be.
template <bool F32>
struct Raw8 {
    uint4 q[F32 ? 2 : 1];
};

template <bool F32, bool VEC, bool OWN = false>
__device__ __forceinline__ void fetch8(const void *row, int c, int step, int H, Raw8<F32> &r)
{
    if constexpr (VEC) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const char *>(row) + c * (F32 ? 4 : 2));
        r.q[0] = OWN ? ld_own_v4(p) : ldg_nc_v4(p);
        if constexpr (F32) r.q[1] = OWN ? ld_own_v4(p + 1) : ldg_nc_v4(p + 1);
    } else {
        float v[8];
        get8<F32, false, OWN>(row, c, step, H, v);
        if constexpr (F32) {
            r.q[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
            r.q[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
        } else {
            r.q[0] = pack8(v);  // (exact: the values are bf16)
        }
    }
}

template <bool F32>
__device__ __forceinline__ void open8(const Raw8<F32> &r, float (&v)[8])
{
    if constexpr (F32) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[4 * i] = __uint_as_float(r.q[i].x);
            v[4 * i + 1] = __uint_as_float(r.q[i].y);
            v[4 * i + 2] = __uint_as_float(r.q[i].z);
            v[4 * i + 3] = __uint_as_float(r.q[i].w);
        }
    } else {
        unpack8(r.q[0], v);
    }
}

constexpr int cta_threads(int tpr) { return tpr > 128 ? tpr : 128; }

}  // namespace

// TPR threads per row, NV vectors of 8 columns each; RES: 0 no residual, 1 a bf16 one, 2 an fp32 one. (512 threads: three
// CTAs an SM, 40 registers a thread; with more and two CTAs, 2048 rows of 8192 columns take 31.2 us instead of 27.0.)
template <int TPR, int NV, int RES, bool VEC>
__global__ void __launch_bounds__(cta_threads(TPR), TPR == 512 ? 3 : 0) rmsnorm_kernel(const __grid_constant__ NormParams p)
{
    constexpr int kRows = cta_threads(TPR) / TPR;
    __shared__ float red[32];
    pdl_enter();
    const int t = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
    const bool live = row < p.rows;
    const int H = p.H;
    // a thread's i-th eight columns: neighbouring ones, or (an element at a time) TPR apart, so that a warp's lie together
    // (8-bit codes want neighbouring ones all the same)
    const int step = VEC || p.codes ? 1 : TPR;
    auto at = [&](int i) { return VEC || p.codes ? 8 * (t + i * TPR) : t + 8 * i * TPR; };
    float v[NV][8];
    float sq = 0.f;
    constexpr bool F32 = RES == 2;
    const uint16_t *xr = static_cast<const uint16_t *>(p.x) + row * p.ld_x;
    const char *rr = static_cast<const char *>(p.residual) + row * p.ld_residual * (F32 ? 4 : 2);
    char *sr = static_cast<char *>(p.total) + row * p.ld_total * (F32 ? 4 : 2);
    // (the loads of all columns stand before the first store, which may go over the residual)
    Raw8<false> xq[NV] = {};
    Raw8<F32> rq[NV] = {};
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (live && at(i) < H) {
                fetch8<false, true>(xr, at(i), step, H, xq[i]);
                if constexpr (RES != 0) fetch8<F32, true, true>(rr, at(i), step, H, rq[i]);
            }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = at(i);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        if (VEC) open8(xq[i], v[i]);
        else if (live && c < H) get8<false, false>(xr, c, step, H, v[i]);
    }
    if constexpr (RES != 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = at(i);
            if (live && c < H) {
                float r[8];
                if constexpr (VEC) open8(rq[i], r);
                else get8<F32, false, true>(rr, c, step, H, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[i][j] += r[j];
                    if (!F32) v[i][j] = __bfloat162float(__float2bfloat16_rn(v[i][j]));
                }
                put8<F32, VEC>(sr, c, step, H, v[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) sq = fmaf(v[i][j], v[i][j], sq);
    const float rstd = __frsqrt_rn(__fdiv_rn(row_sum<TPR>(sq, red), (float)H) + p.eps);
    if (live && t == 0 && p.rstd) p.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = at(i);
        if (8 * (i * TPR) >= H) break;
        if (c < H) {
            float g[8];
            gain8<VEC>(p.w, p.w_f32, p.offset, c, step, H, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * g[j];
        }
        if (live && c < H && p.y) put8<false, VEC>(static_cast<uint16_t *>(p.y) + row * p.ld_y, c, step, H, v[i]);
        if (p.codes) {  // 16 neighbouring threads hold a block of 128 columns (zero beyond the row)
            const float s = block_scale(v[i]);
            if (live && c < H) {
                *reinterpret_cast<uint2 *>(p.codes + row * p.ld_codes + c) = block_codes(v[i], s);
                if ((t & 15) == 0) p.scales[(c / 128) * p.ld_scales + row] = s;
            }
        }
    }
}

// Gradient. A CTA takes every gridDim-th group of rows, and its threads always the same columns, so that the
// weight's gradient adds up in registers; the CTAs' sums go to the workspace [gridDim][H] and
// norm_weight_kernel adds them in order. The next rows' loads are in flight while these are worked on.
template <int TPR, int NV, bool F32, bool VEC>
__global__ void __launch_bounds__(cta_threads(TPR), 1024 / cta_threads(TPR)) rmsnorm_backward_kernel(const __grid_constant__ NormBackParams p)
{
    constexpr int kRows = cta_threads(TPR) / TPR;
    extern __shared__ float sh_sum[];  // [kRows - 1][H] where several rows share a CTA
    __shared__ float red[2][32];
    pdl_enter();
    const int t = threadIdx.x % TPR, team = threadIdx.x / TPR;
    const int H = p.H;
    constexpr int step = VEC ? 1 : TPR;  // columns as in the forward kernel
    auto at = [&](int i) { return VEC ? 8 * (t + i * TPR) : t + 8 * i * TPR; };
    float acc[NV][8] = {};
    constexpr bool kAhead = !F32;  // (an fp32 dtotal has no registers to wait in: loaded where its row's sum begins)
    Raw8<F32> total[NV] = {}, past[NV] = {};
    Raw8<false> dy[NV] = {};
    float rstd = 0.f;
    auto fetch = [&](int64_t row) {
        if (row >= p.rows) return;
        const char *sr = static_cast<const char *>(p.total) + row * p.ld_total * (F32 ? 4 : 2);
        const char *pr = static_cast<const char *>(p.dtotal) + row * p.ld_dtotal * (F32 ? 4 : 2);
        const uint16_t *dr = static_cast<const uint16_t *>(p.dy) + row * p.ld_dy;
        rstd = __ldg(p.rstd + row);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = at(i);
            if (c < H) {
                fetch8<F32, VEC>(sr, c, step, H, total[i]);
                fetch8<false, VEC>(dr, c, step, H, dy[i]);
                if (kAhead && p.dtotal) fetch8<F32, VEC, true>(pr, c, step, H, past[i]);
            }
        }
    };
    const int64_t stride = (int64_t)gridDim.x * kRows;
    fetch((int64_t)blockIdx.x * kRows + team);
    int turn = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * kRows; row0 < p.rows; row0 += stride, turn ^= 1) {
        const int64_t row = row0 + team;
        const bool live = row < p.rows;
        char *out = static_cast<char *>(p.dx) + row * p.ld_dx * (F32 ? 4 : 2);
        const char *pr = static_cast<const char *>(p.dtotal) + row * p.ld_dtotal * (F32 ? 4 : 2);
        float n[NV][8], g[NV][8];
        Raw8<F32> ds[NV] = {};
        const float r = rstd;
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = at(i);
            open8(total[i], n[i]);
            open8(dy[i], g[i]);
            if (kAhead) ds[i] = past[i];
            else if (live && c < H && p.dtotal) fetch8<F32, VEC, true>(pr, c, step, H, ds[i]);
            if (live && c < H) {
                float w[8];
                gain8<VEC>(p.w, p.w_f32, p.offset, c, step, H, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    n[i][j] *= r;
                    acc[i][j] = fmaf(g[i][j], n[i][j], acc[i][j]);
                    g[i][j] *= w[j];
                    dot = fmaf(g[i][j], n[i][j], dot);
                }
            }
        }
        fetch(row + stride);
        const float mean = __fdiv_rn(row_sum<TPR>(dot, red[turn]), (float)H);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = at(i);
            if (live && c < H) {
                float d[8];
                open8(ds[i], d);
#pragma unroll
                for (int j = 0; j < 8; ++j) n[i][j] = fmaf(r, fmaf(-n[i][j], mean, g[i][j]), d[j]);
                put8<F32, VEC>(out, c, step, H, n[i]);
            }
        }
    }
    if (!p.part) return;
    if constexpr (kRows > 1) {  // the CTA's rows, in order
        if (team > 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int c = at(i) + j * step;
                    if (c < H) sh_sum[(team - 1) * H + c] = acc[i][j];
                }
        }
        __syncthreads();
        if (team > 0) return;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = at(i) + j * step;
                for (int k = 0; c < H && k < kRows - 1; ++k) acc[i][j] += sh_sum[k * H + c];
            }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = at(i) + j * step;
            if (c < H) p.part[(int64_t)blockIdx.x * H + c] = acc[i][j];
        }
}

// dw[c] = (dw[c] +) the sum of part[i][c] over i: 32 columns per CTA, each of its 32 warps a share of the parts (all
// loads in flight), the shares joined in order. Bound by the latency of two rounds of loads: 608 parts of 2048 columns
// take 6.7 us by themselves under a profiler, nothing in L1; with eight warps a CTA they took three times as long.
constexpr int kJoinWarps = 32;
__global__ void __launch_bounds__(32 * kJoinWarps)
    norm_weight_kernel(const float *__restrict__ part, int parts, int H, float *__restrict__ dw, int accumulate)
{
    __shared__ float sum[kJoinWarps][32];
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < H)
        for (int i0 = warp; i0 < parts; i0 += 16 * kJoinWarps) {
            float v[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int i = i0 + k * kJoinWarps;
                v[k] = i < parts ? part[(int64_t)i * H + c] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) s += v[k];
        }
    sum[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < H) {
        s = 0.f;
#pragma unroll
        for (int k = 0; k < kJoinWarps; ++k) s += sum[k][lane];
        dw[c] = accumulate ? dw[c] + s : s;
    }
}

namespace {

bool vec16(const void *p, int64_t ld, int size) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0; }

template <int TPR, int NV, int RES>
cudaError_t launch_norm(const NormParams &p, bool vec, cudaStream_t s)
{
    constexpr int kRows = cta_threads(TPR) / TPR;
    const dim3 grid((unsigned)((p.rows + kRows - 1) / kRows));
    if (vec) FT_LAUNCH(rmsnorm_kernel<TPR, NV, RES, true>, grid, dim3(cta_threads(TPR)), 0, s, p);
    else FT_LAUNCH(rmsnorm_kernel<TPR, NV, RES, false>, grid, dim3(cta_threads(TPR)), 0, s, p);
    count_launches(1);
    return cudaGetLastError();
}

template <int RES>
cudaError_t launch_norm_sized(const NormParams &p, bool vec, cudaStream_t s)
{
    const int nv = (p.H + 7) / 8;
    if (nv <= 32) return launch_norm<32, 1, RES>(p, vec, s);
    if (nv <= 128) return launch_norm<128, 1, RES>(p, vec, s);
    if (nv <= 256) return launch_norm<256, 1, RES>(p, vec, s);
    if (nv <= 512) return launch_norm<256, 2, RES>(p, vec, s);
    if (nv <= 1024) return launch_norm<512, 2, RES>(p, vec, s);
    return launch_norm<1024, 2, RES>(p, vec, s);
}

template <int TPR, int NV, bool F32>
cudaError_t launch_back(NormBackParams p, bool vec, int grid, cudaStream_t s)
{
    constexpr int kRows = cta_threads(TPR) / TPR;
    const size_t smem = p.part ? (size_t)(kRows - 1) * p.H * 4 : 0;
    if (vec) FT_LAUNCH(rmsnorm_backward_kernel<TPR, NV, F32, true>, dim3(grid), dim3(cta_threads(TPR)), smem, s, p);
    else FT_LAUNCH(rmsnorm_backward_kernel<TPR, NV, F32, false>, dim3(grid), dim3(cta_threads(TPR)), smem, s, p);
    count_launches(1);
    return cudaGetLastError();
}

// Rows of one CTA of the backward kernel, by the row's length.
int back_rows(int H) { return H <= 256 ? 4 : 1; }

template <bool F32>
cudaError_t launch_back_sized(const NormBackParams &p, bool vec, int grid, cudaStream_t s)
{
    const int nv = (p.H + 7) / 8;
    if (nv <= 32) return launch_back<32, 1, F32>(p, vec, grid, s);
    if (nv <= 128) return launch_back<128, 1, F32>(p, vec, grid, s);
    if (nv <= 256) return launch_back<256, 1, F32>(p, vec, grid, s);
    if (nv <= 512) return launch_back<512, 1, F32>(p, vec, grid, s);
    if (nv <= 1024) return launch_back<1024, 1, F32>(p, vec, grid, s);
    return launch_back<1024, 2, F32>(p, vec, grid, s);
}

}  // namespace

cudaError_t launch_rmsnorm(const NormParams &p, cudaStream_t s)
{
    const int sz = p.total_f32 ? 4 : 2;
    const bool vec = p.H % 8 == 0 && vec16(p.x, p.ld_x, 2) && vec16(p.w, 0, 1) && (!p.y || vec16(p.y, p.ld_y, 2)) &&
                     (!p.residual || (vec16(p.residual, p.ld_residual, sz) && vec16(p.total, p.ld_total, sz)));
    if (!p.residual) return launch_norm_sized<0>(p, vec, s);
    return p.total_f32 ? launch_norm_sized<2>(p, vec, s) : launch_norm_sized<1>(p, vec, s);
}

int norm_parts(int rows, int H)
{
    const int per = back_rows(H), all = (rows + per - 1) / per, most = 2 * 152 * (H <= 1024 ? 4 : H <= 2048 ? 2 : 1);
    return all < most ? all : most;
}

cudaError_t launch_rmsnorm_backward(NormBackParams p, float *dw, int accumulate, void *workspace, cudaStream_t s)
{
    const int sz = p.total_f32 ? 4 : 2, grid = norm_parts(p.rows, p.H);
    const bool vec = p.H % 8 == 0 && vec16(p.dy, p.ld_dy, 2) && vec16(p.w, 0, 1) && vec16(p.total, p.ld_total, sz) &&
                     vec16(p.dx, p.ld_dx, sz) && (!p.dtotal || vec16(p.dtotal, p.ld_dtotal, sz));
    p.part = dw ? static_cast<float *>(workspace) : nullptr;
    const cudaError_t e = p.total_f32 ? launch_back_sized<true>(p, vec, grid, s) : launch_back_sized<false>(p, vec, grid, s);
    if (e != cudaSuccess || !dw) return e;
    FT_LAUNCH(norm_weight_kernel, dim3((p.H + 31) / 32), dim3(32 * kJoinWarps), 0, s, (const float *)p.part, grid, p.H, dw, accumulate);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace ftmoe
