// Building blocks of the row kernels: 16-byte loads and stores of bf16 and fp32 rows, e4m3 codes with their block
// scales, the sigmoid.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "ftmoe_device.cuh"

namespace ftmoe {
namespace rows {

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

}  // namespace rows
}  // namespace ftmoe
