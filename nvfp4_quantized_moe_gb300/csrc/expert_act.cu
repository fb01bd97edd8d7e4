// Row kernels around the grouped products: 8-bit quantization of activation rows, and the SwiGLU
// step between an expert's two products (forward, forward stored in 8 bits, backward). All are
// bound by memory: each value is read once and written once, sums and maxima stay in fp32.
//
//   quantize   scale = max(amax / 448, 2^-126) over 128 values of a row, code = e4m3(v * (1 / scale)),
//              each step one correctly rounded fp32 operation, codes to nearest even
//   SwiGLU     h = w * g * s * u with s = 1 / (1 + e^-g) and the row's weight w (or 1)
//   backward   dg = w dh u s (1 + g (1 - s)),  du = w dh g s,  dw = sum dh g s u
//
// Measured on one GB300 (copy bandwidth 6.78 TB/s), 65536 rows: SwiGLU forward (512 columns) 29.1 us,
// 6.9 TB/s; backward 53.8 us, 6.2 TB/s; in 8 bits 29.1 us, 5.8 TB/s (two special functions and the
// scaling per value); quantizer (2048 columns) 67.6 us, 6.0 TB/s.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ftmoe_device.cuh"
#include "ftmoe_internal.h"

namespace ftmoe {

namespace {

__device__ __forceinline__ void unpack8(uint4 q, float (&v)[8])
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8])
{
    return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}

// 8 values of a row starting at `col` (aligned to 8 elements).
template <bool F32>
__device__ __forceinline__ void load8(const void *row, int col, float (&v)[8])
{
    if constexpr (F32) {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(row) + col);
        const float4 a = __ldg(p), b = __ldg(p + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        unpack8(ldg_nc_v4(static_cast<const uint16_t *>(row) + col), v);
    }
}

// Four e4m3 codes, nearest even, saturating at 448; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// The 16 lanes of a half warp hold 8 values each of one 128-value block: returns its scale.
// Magnitudes are compared as integers, so that a NaN (whose bits exceed infinity's) is the
// maximum and reaches the scale: a block that holds a value that is not finite has no finite value.
__device__ __forceinline__ float block_scale(const float (&v)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    const float s = __fdiv_rn(__uint_as_float(m), 448.0f);
    return s < 0x1p-126f ? 0x1p-126f : s;
}

__device__ __forceinline__ uint2 block_codes(const float (&v)[8], float scale)
{
    const float r = __frcp_rn(scale);
    return make_uint2(e4m3x4(v[0] * r, v[1] * r, v[2] * r, v[3] * r), e4m3x4(v[4] * r, v[5] * r, v[6] * r, v[7] * r));
}

// s = 1 / (1 + e^-g) as (1/4) / (1/4 + e^-g / 4), with e^-g / 4 = 2^(-g log2(e) - 2): one multiply-add before the
// power of two, and a divisor that stays below 2^126 where s is 1e-38 and g s u may be of any size (the fast
// reciprocal gives zero above 2^126, which 1 + e^-g passes below g = -87.3). s is 0 below -88.7. The exponent is
// off by |g| 2^-23 at most and the power by 2^-22: s is within 2^-21 near zero and 1e-5 at g = -88, relative; the
// stores round to 2^-9 (bf16) or 2^-5 (8 bits) on average. (From e^-|g|, 65536 x 512 in 8 bits take 32.7 us, backward
// 55.8; as here 29.1 and 53.8.)
__device__ __forceinline__ float sigmoid(float g)
{
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fmaf(g, -1.4426950408889634f, -2.0f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(0.25f + e));
    return 0.25f * r;
}

constexpr int kActThreads = 256;
// Quantizing kernels: 16 lanes per row and block of 128; 8 rows per CTA, so that the scales of a block
// fill a 32-byte sector. (65536 x 2048 bf16: 67.7 us, with 16 rows per CTA 70.0.)
constexpr int kQuantThreads = 128;
constexpr int kRowsPerCta = kQuantThreads / 16;

}  // namespace

// A CTA takes its rows by several blocks of 128 columns, whose loads are all in flight before the
// first is used: 65536 x 2048 bf16 rows take 67.7 us (5.9 TB/s), one block at a time 86, eight 79.
// (A launch that does not fill the SMs takes one: more CTAs are then faster.)
template <bool F32, int kBlocks>
__global__ void __launch_bounds__(kQuantThreads)
    quantize_fp8_kernel(const void *__restrict__ src, int64_t ld, int rows, int K, uint8_t *__restrict__ codes,
                        int64_t ld_codes, float *__restrict__ scales, int64_t ld_scales)
{
    pdl_enter();
    const int row = blockIdx.x * kRowsPerCta + (threadIdx.x >> 4), l = threadIdx.x & 15;
    const int b0 = blockIdx.y * kBlocks, c0 = 128 * b0 + 8 * l;
    const void *from = static_cast<const char *>(src) + (int64_t)row * ld * (F32 ? 4 : 2);
    float v[kBlocks][8] = {};
#pragma unroll
    for (int i = 0; i < kBlocks; ++i)
        if (row < rows && c0 + 128 * i < K) load8<F32>(from, c0 + 128 * i, v[i]);
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
        if (128 * (b0 + i) >= K) break;
        const float s = block_scale(v[i]);
        if (row < rows && c0 + 128 * i < K)
            *reinterpret_cast<uint2 *>(codes + row * ld_codes + c0 + 128 * i) = block_codes(v[i], s);
        if (row < rows && l == 0) scales[(b0 + i) * ld_scales + row] = s;
    }
}

// (One block per thread and 16 rows per CTA here: with the exponentials in between, more threads hide
// more than longer ones: 65536 x 512 took 31.5 us, two blocks 33.9, four 43.2, 8 rows 34.3,
// all with a slower sigmoid than today's, whose 29.1 is with this one.)
__global__ void __launch_bounds__(kActThreads)
    swiglu_quantize_fp8_kernel(const uint16_t *__restrict__ gu, int64_t ld, const float *__restrict__ w, int rows, int I,
                               uint8_t *__restrict__ codes, int64_t ld_codes, float *__restrict__ scales,
                               int64_t ld_scales)
{
    pdl_enter();
    const int row = blockIdx.x * (kActThreads / 16) + (threadIdx.x >> 4), l = threadIdx.x & 15;
    const int col = blockIdx.y * 128 + 8 * l;
    const bool in = row < rows && col < I;
    float h[8] = {};
    if (in) {
        float g[8], u[8];
        load8<false>(gu + row * ld, col, g);
        load8<false>(gu + row * ld + I, col, u);
        const float f = w ? __ldg(w + row) : 1.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = f * (g[i] * sigmoid(g[i]) * u[i]);
    }
    const float s = block_scale(h);
    if (in) *reinterpret_cast<uint2 *>(codes + row * ld_codes + col) = block_codes(h, s);
    if (row < rows && l == 0) scales[blockIdx.y * ld_scales + row] = s;
}

// One warp per row. VEC: 8 columns per lane and step (everything 16-byte aligned), else one.
template <bool VEC>
__global__ void __launch_bounds__(kActThreads)
    swiglu_kernel(const uint16_t *__restrict__ gu, int64_t ld, const float *__restrict__ w, int rows, int I,
                  uint16_t *__restrict__ h, int64_t ld_h)
{
    pdl_enter();
    const int lane = threadIdx.x & 31, warps = gridDim.x * (kActThreads / 32);
    for (int row = blockIdx.x * (kActThreads / 32) + (threadIdx.x >> 5); row < rows; row += warps) {
        const uint16_t *gr = gu + row * ld, *ur = gr + I;
        uint16_t *o = h + row * ld_h;
        const float f = w ? __ldg(w + row) : 1.0f;
        if constexpr (VEC) {
            for (int c = 8 * lane; c < I; c += 512) {  // two steps' loads in flight together
                uint4 q[2][2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (c + 256 * k >= I) break;
                    q[k][0] = ldg_nc_v4(gr + c + 256 * k);
                    q[k][1] = ldg_nc_v4(ur + c + 256 * k);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (c + 256 * k >= I) break;
                    float g[8], u[8];
                    unpack8(q[k][0], g);
                    unpack8(q[k][1], u);
#pragma unroll
                    for (int i = 0; i < 8; ++i) g[i] = f * (g[i] * sigmoid(g[i]) * u[i]);
                    *reinterpret_cast<uint4 *>(o + c + 256 * k) = pack8(g);
                }
            }
        } else {
            for (int c = lane; c < I; c += 32) {
                const float g = __uint_as_float((uint32_t)__ldg(gr + c) << 16), u = __uint_as_float((uint32_t)__ldg(ur + c) << 16);
                o[c] = __bfloat16_as_ushort(__float2bfloat16_rn(f * (g * sigmoid(g) * u)));
            }
        }
    }
}

template <bool VEC>
__global__ void __launch_bounds__(kActThreads)
    swiglu_backward_kernel(const uint16_t *__restrict__ gu, int64_t ld, const float *__restrict__ w,
                           const uint16_t *__restrict__ dh, int64_t ld_dh, int rows, int I, uint16_t *__restrict__ dgu,
                           int64_t ld_dgu, float *__restrict__ dw)
{
    pdl_enter();
    const int lane = threadIdx.x & 31, warps = gridDim.x * (kActThreads / 32);
    for (int row = blockIdx.x * (kActThreads / 32) + (threadIdx.x >> 5); row < rows; row += warps) {
        const uint16_t *gr = gu + row * ld, *ur = gr + I, *dr = dh + row * ld_dh;
        uint16_t *og = dgu + row * ld_dgu, *ou = og + I;
        const float f = w ? __ldg(w + row) : 1.0f;
        float sum = 0.f;
        auto one = [&](float g, float u, float d, float &dg, float &du) {
            const float s = sigmoid(g), gs = g * s, fd = f * d;
            dg = fd * u * (s * (1.0f + g * (1.0f - s)));
            du = fd * gs;
            sum = fmaf(d, gs * u, sum);
        };
        if constexpr (VEC) {
            for (int c = 8 * lane; c < I; c += 512) {  // two steps' loads in flight together
                uint4 q[2][3];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (c + 256 * k >= I) break;
                    q[k][0] = ldg_nc_v4(gr + c + 256 * k);
                    q[k][1] = ldg_nc_v4(ur + c + 256 * k);
                    q[k][2] = ldg_nc_v4(dr + c + 256 * k);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (c + 256 * k >= I) break;
                    float g[8], u[8], d[8];
                    unpack8(q[k][0], g);
                    unpack8(q[k][1], u);
                    unpack8(q[k][2], d);
#pragma unroll
                    for (int i = 0; i < 8; ++i) one(g[i], u[i], d[i], g[i], u[i]);
                    *reinterpret_cast<uint4 *>(og + c + 256 * k) = pack8(g);
                    *reinterpret_cast<uint4 *>(ou + c + 256 * k) = pack8(u);
                }
            }
        } else {
            for (int c = lane; c < I; c += 32) {
                float dg, du;
                one(__uint_as_float((uint32_t)__ldg(gr + c) << 16), __uint_as_float((uint32_t)__ldg(ur + c) << 16),
                    __uint_as_float((uint32_t)__ldg(dr + c) << 16), dg, du);
                og[c] = __bfloat16_as_ushort(__float2bfloat16_rn(dg));
                ou[c] = __bfloat16_as_ushort(__float2bfloat16_rn(du));
            }
        }
        if (dw) {  // the same order of additions on every run
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            if (lane == 0) dw[row] = sum;
        }
    }
}

static bool vec_ok(const void *p, int64_t ld, int I)
{
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0 && I % 8 == 0;
}

static int row_grid(int rows)
{
    const int per = kActThreads / 32, cap = sm_count() * 8;
    const int g = (rows + per - 1) / per;
    return g < cap ? g : cap;
}

cudaError_t launch_quantize_fp8(const void *src, bool f32, int64_t ld, int rows, int K, uint8_t *codes, int64_t ld_codes,
                                float *scales, int64_t ld_scales, cudaStream_t s)
{
    const int by_rows = (rows + kRowsPerCta - 1) / kRowsPerCta, nb = (K + 127) / 128;
    const int per = (int64_t)by_rows * nb < 32 * sm_count() ? 1 : 4;
    auto kern = f32 ? (per == 1 ? quantize_fp8_kernel<true, 1> : quantize_fp8_kernel<true, 4>)
                    : (per == 1 ? quantize_fp8_kernel<false, 1> : quantize_fp8_kernel<false, 4>);
    FT_LAUNCH(kern, dim3(by_rows, (nb + per - 1) / per), dim3(kQuantThreads), 0, s, src, ld, rows, K, codes, ld_codes, scales,
              ld_scales);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_swiglu_quantize_fp8(const void *gu, int64_t ld_gu, const float *w, int rows, int I, uint8_t *codes,
                                       int64_t ld_codes, float *scales, int64_t ld_scales, cudaStream_t s)
{
    FT_LAUNCH(swiglu_quantize_fp8_kernel, dim3((rows + kActThreads / 16 - 1) / (kActThreads / 16), (I + 127) / 128), dim3(kActThreads),
              0, s, static_cast<const uint16_t *>(gu), ld_gu, w, rows, I, codes, ld_codes, scales, ld_scales);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_swiglu(const void *gu, int64_t ld_gu, const float *w, int rows, int I, void *h, int64_t ld_h,
                          cudaStream_t s)
{
    auto kern = vec_ok(gu, ld_gu, I) && vec_ok(h, ld_h, I) ? swiglu_kernel<true> : swiglu_kernel<false>;
    FT_LAUNCH(kern, dim3(row_grid(rows)), dim3(kActThreads), 0, s, static_cast<const uint16_t *>(gu), ld_gu, w, rows, I,
              static_cast<uint16_t *>(h), ld_h);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_swiglu_backward(const void *gu, int64_t ld_gu, const float *w, const void *dh, int64_t ld_dh, int rows,
                                   int I, void *dgu, int64_t ld_dgu, float *dw, cudaStream_t s)
{
    auto kern = vec_ok(gu, ld_gu, I) && vec_ok(dh, ld_dh, I) && vec_ok(dgu, ld_dgu, I) ? swiglu_backward_kernel<true>
                                                                                     : swiglu_backward_kernel<false>;
    FT_LAUNCH(kern, dim3(row_grid(rows)), dim3(kActThreads), 0, s, static_cast<const uint16_t *>(gu), ld_gu, w,
              static_cast<const uint16_t *>(dh), ld_dh, rows, I, static_cast<uint16_t *>(dgu), ld_dgu, dw);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace ftmoe
