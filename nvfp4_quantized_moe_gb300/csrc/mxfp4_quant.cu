// Rows in microscaled 4-bit floating point (MXFP4), as the grouped 4-bit product reads them: e2m1 codes, two to a
// byte, with a power of two as scale for every 32 columns of a row.
//
//   scale = 2^s, the smallest power of two with amax <= 6 * 2^s   (s >= -127; stored as the byte s + 127)
//   code  = e2m1(v * 2^-s), to nearest, ties to even
//
// 6 is the largest e2m1 value: nothing saturates, and the largest value of a block is off by at most a quarter of
// itself (half a step; the scale that the floor of log2 amax gives would cut values between 6 and 8 down to 6). The
// scaling is exact, so that codes and scales are a function of the inputs alone. A block that holds an infinity or a
// NaN gets the scale byte 255, the format's NaN: all its values are NaN.
//
// Scale bytes of four neighbouring blocks (128 columns) lie together as a word. Rows of a batch have the words of one
// 128 columns side by side, [K / 128][rows]; weights have them in the tiles of 128 rows x 128 columns that the tensor
// cores take, word 4 (n % 32) + n / 32 of 128 for row n.
//
// Bound by memory: 65536 x 2048 bf16 values (0.34 GB read and written) take 57 us, 6.0 TB/s, as a plain copy of that size;
// SwiGLU of 65536 x 512 (0.15 GB) 30 us, where the exponentials count as much.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ftmoe_device.cuh"
#include "ftmoe_internal.h"
#include "row_ops.cuh"

namespace ftmoe {

using namespace rows;

namespace {

constexpr int kThreads4 = 128;
constexpr int kQuantRows = kThreads4 / 8;  // quantizer: rows per CTA
constexpr int kRows4 = kThreads4 / 16;     // SwiGLU

// Eight e2m1 codes of x * r, the first in the lowest nibble.
__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[8], float r)
{
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2)  // two products per instruction
        asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmul.rn.f32x2 a, a, b;\n\t"
            "mov.b64 {%0, %1}, a;\n\t}"
            : "=f"(v[i]), "=f"(v[i + 1])
            : "f"(x[i]), "f"(x[i + 1]), "f"(r));
    uint32_t w;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return w;
}

// Scale byte of a block whose largest magnitude has the fp32 bits m: m's exponent field less 2, one more where the
// mantissa is above 1.5.
__device__ __forceinline__ uint32_t scale_byte(uint32_t m)
{
    return m >= 0x7F800000u ? 255u : (uint32_t)max((int)((m + 0x3FFFFFu) >> 23) - 2, 0);
}

// 2^-s: 254 - byte in the exponent field (byte <= 253 for finite blocks).
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float((254u - min(byte, 253u)) << 23); }

// The 16 lanes of a half warp hold 8 values each of 128 columns (zero beyond the row): the codes of this lane's and
// the word of the four blocks' scale bytes.
__device__ __forceinline__ uint32_t block_codes4(const float (&v)[8], uint32_t &word)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    const uint32_t byte = scale_byte(m);
    uint32_t w = byte << (8 * ((threadIdx.x & 15) >> 2));
    w |= __shfl_xor_sync(0xFFFFFFFFu, w, 4);
    w |= __shfl_xor_sync(0xFFFFFFFFu, w, 8);
    word = w;
    return e2m1x8(v, inverse_scale(byte));
}

// Where the scale word of row `row`, columns [128 b, 128 b + 128) goes.
__device__ __forceinline__ int64_t word_at(const Quant4Params &p, int row, int b)
{
    if (p.tile_rows == 0) return b * p.ld_scales + row;
    const int e = row / p.tile_rows, n = row - e * p.tile_rows;
    const int nt = (p.tile_rows + 127) / 128, kt = (p.K + 127) / 128;
    return (((int64_t)e * nt + n / 128) * kt + b) * 128 + n % 32 * 4 + n % 128 / 32;
}

}  // namespace

// Sixteen values of a lane as they lie in memory: the first and the third (even lanes), or the second and the fourth
// eight of a block of 32, so that a load of two neighbouring lanes is one whole sector.
template <bool F32>
struct Half32 {
    uint4 q[F32 ? 4 : 2];
    __device__ __forceinline__ void load(const void *row, int c)
    {
        const char *p = static_cast<const char *>(row) + (int64_t)c * (F32 ? 4 : 2);
        if constexpr (F32) {
            q[0] = ldg_nc_v4(p); q[1] = ldg_nc_v4(p + 16); q[2] = ldg_nc_v4(p + 64); q[3] = ldg_nc_v4(p + 80);
        } else {
            q[0] = ldg_nc_v4(p); q[1] = ldg_nc_v4(p + 32);
        }
    }
    // Largest magnitude as the bits of an fp32 (a NaN, whose bits exceed infinity's, is the largest).
    __device__ __forceinline__ uint32_t amax() const
    {
        uint32_t m = 0;
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                m = max(max(m, max(q[i].x & 0x7FFFFFFFu, q[i].y & 0x7FFFFFFFu)), max(q[i].z & 0x7FFFFFFFu, q[i].w & 0x7FFFFFFFu));
        } else {  // two bf16 magnitudes at a time
#pragma unroll
            for (int i = 0; i < 2; ++i)
                m = __vmaxu2(__vmaxu2(m, __vmaxu2(q[i].x & 0x7FFF7FFFu, q[i].y & 0x7FFF7FFFu)),
                             __vmaxu2(q[i].z & 0x7FFF7FFFu, q[i].w & 0x7FFF7FFFu));
            m = max(m & 0xFFFF0000u, m << 16);
        }
        return m;
    }
    // Codes of the first or second eight values, scaled by r.
    __device__ __forceinline__ uint32_t codes(int half, float r) const
    {
        float v[8];
        if constexpr (F32) {
            const uint4 a = q[2 * half], b = q[2 * half + 1];
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
        } else {
            unpack8(q[half], v);
        }
        return e2m1x8(v, r);
    }
};

// 8 lanes per row and 128 columns; kBlocks times 128 columns per CTA, whose loads are all in flight before the first
// is used. Bound by its instructions as much as by memory: with 8 values a lane, each widened before its
// maximum is taken, 65536 x 2048 bf16 values took 61 us and 11 instructions a value.
template <bool F32, int kBlocks>
__global__ void __launch_bounds__(kThreads4) quantize_mxfp4_kernel(const __grid_constant__ Quant4Params p)
{
    pdl_enter();
    const int row = blockIdx.x * kQuantRows + (threadIdx.x >> 3), l = threadIdx.x & 7, odd = l & 1;
    const int b0 = blockIdx.y * kBlocks, c0 = 128 * b0 + 32 * (l >> 1);  // the lane's block of 32
    const void *from = static_cast<const char *>(p.src) + (int64_t)row * p.ld_src * (F32 ? 4 : 2);
    Half32<F32> v[kBlocks] = {};
#pragma unroll
    for (int i = 0; i < kBlocks; ++i)
        if (row < p.rows && c0 + 128 * i < p.K) v[i].load(from, c0 + 128 * i + 8 * odd);
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
        if (128 * (b0 + i) >= p.K) break;
        uint32_t m = v[i].amax();
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        const uint32_t byte = scale_byte(m);
        const float r = inverse_scale(byte);
        const uint32_t a = v[i].codes(0, r), b = v[i].codes(1, r);
        // neighbours trade, so that each has eight bytes in a row
        const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, odd ? a : b, 1);
        if (row < p.rows && c0 + 128 * i < p.K)
            *reinterpret_cast<uint2 *>(p.codes + row * p.ld_codes + (c0 + 128 * i) / 2 + 8 * odd) =
                odd ? make_uint2(other, b) : make_uint2(a, other);
        uint32_t word = byte << (8 * (l >> 1));
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
        if (row < p.rows && l == 0) p.scales[word_at(p, row, b0 + i)] = word;
    }
}

// w * silu(gate) * up of rows [gate, up], quantized.
__global__ void __launch_bounds__(kThreads4) swiglu_quantize_mxfp4_kernel(const __grid_constant__ Quant4Params p)
{
    pdl_enter();
    const int row = blockIdx.x * kRows4 + (threadIdx.x >> 4), l = threadIdx.x & 15;
    const int col = blockIdx.y * 128 + 8 * l;
    const bool in = row < p.rows && col < p.K;
    const uint16_t *gu = static_cast<const uint16_t *>(p.src) + row * p.ld_src;
    float h[8] = {};
    if (in) {
        float g[8], u[8];
        load8<false>(gu, col, g);
        load8<false>(gu + p.K, col, u);
        const float f = p.w ? __ldg(p.w + row) : 1.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = f * (g[i] * sigmoid(g[i]) * u[i]);
    }
    uint32_t word;
    const uint32_t codes = block_codes4(h, word);
    if (in) *reinterpret_cast<uint32_t *>(p.codes + row * p.ld_codes + col / 2) = codes;
    if (row < p.rows && l == 0) p.scales[blockIdx.y * p.ld_scales + row] = word;
}

// Scale bytes [E][N][K / 32] into tiles: one word per thread, zeros beyond N and K.
__global__ void __launch_bounds__(256)
    pack_mxfp4_scales_kernel(const uint8_t *__restrict__ src, int E, int N, int K, uint32_t *__restrict__ tiles)
{
    pdl_enter();
    const int nt = (N + 127) / 128, kt = (K + 127) / 128, blocks = K / 32;
    const int64_t words = (int64_t)E * nt * kt * 128, step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < words; i += step) {
        const int in_tile = (int)(i % 128);
        const int64_t tile = i / 128;
        const int b = (int)(tile % kt);
        const int64_t et = tile / kt;
        const int n = (int)(et % nt) * 128 + in_tile % 4 * 32 + in_tile / 4;
        uint32_t w = 0;
        if (n < N) {
            const uint8_t *row = src + (et / nt * N + n) * (int64_t)blocks;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (4 * b + j < blocks) w |= (uint32_t)__ldg(row + 4 * b + j) << (8 * j);
        }
        tiles[i] = w;
    }
}

cudaError_t launch_quantize_mxfp4(const Quant4Params &p, bool f32, cudaStream_t s)
{
    const int by_rows = (p.rows + kQuantRows - 1) / kQuantRows, nb = (p.K + 127) / 128;
    const int per = (int64_t)by_rows * nb < 32 * sm_count() ? 1 : 2;
    auto kern = f32 ? (per == 1 ? quantize_mxfp4_kernel<true, 1> : quantize_mxfp4_kernel<true, 2>)
                    : (per == 1 ? quantize_mxfp4_kernel<false, 1> : quantize_mxfp4_kernel<false, 2>);
    FT_LAUNCH(kern, dim3(by_rows, (nb + per - 1) / per), dim3(kThreads4), 0, s, p);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_swiglu_quantize_mxfp4(const Quant4Params &p, cudaStream_t s)
{
    FT_LAUNCH(swiglu_quantize_mxfp4_kernel, dim3((p.rows + kRows4 - 1) / kRows4, (p.K + 127) / 128), dim3(kThreads4), 0, s, p);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_pack_mxfp4_scales(const uint8_t *src, int E, int N, int K, uint32_t *tiles, cudaStream_t s)
{
    const int64_t words = (int64_t)E * ((N + 127) / 128) * ((K + 127) / 128) * 128;
    const int64_t want = (words + 255) / 256, most = (int64_t)sm_count() * 32;
    FT_LAUNCH(pack_mxfp4_scales_kernel, dim3((unsigned)(want < most ? want : most)), dim3(256), 0, s, src, E, N, K, tiles);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace ftmoe
