// extern "C" entry points of the grouped expert products and the row kernels around them:
// argument validation and launches. See include/ft_moe.h for the contract of every call.
#include <cuda_runtime.h>
#include <stdarg.h>
#include <stdio.h>

#include "ft_moe.h"
#include "ftmoe_internal.h"

namespace ftmoe {

static ft_status reject(ft_status code, const char *fmt, ...)
{
    char text[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof(text), fmt, ap);
    va_end(ap);
    return report_error(code, text);
}

static ft_status finish(cudaError_t e, const char *what)
{
    if (e == cudaSuccess) return report_error(FT_OK, "");
    return reject(FT_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

static bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

constexpr int kMaxRows = 1 << 25;   // T <= 2^20 tokens of up to 32 slots
constexpr int kMaxWidth = 1 << 16;
constexpr size_t kGroupWorkspace = 256;  // the status word

static ft_status check_sizes(int E, int P, int N, int K, int unit_n, int unit_k)
{
    if (E <= 0 || P < 0 || N <= 0 || K <= 0)
        return reject(FT_ERR_INVALID_ARG, "need E, N, K > 0 and P >= 0 (got E %d, P %d, N %d, K %d)", E, P, N, K);
    if (E > kGroupMaxExperts || P > kMaxRows || N > kMaxWidth || K > kMaxWidth)
        return reject(FT_ERR_UNSUPPORTED, "need E <= 1024, P <= 2^25, N and K <= 65536");
    if (N % unit_n || K % unit_k)
        return reject(FT_ERR_UNSUPPORTED, "need N a multiple of %d and K a multiple of %d (got N %d, K %d)", unit_n, unit_k,
                      N, K);
    return FT_OK;
}

static ft_status check_group(const int32_t *offs, int E, const void *workspace, size_t bytes)
{
    if (!offs && E != 1) return reject(FT_ERR_INVALID_ARG, "offs may be NULL for one expert only (got E %d)", E);
    if (!aligned(offs, 4)) return reject(FT_ERR_INVALID_ARG, "offs must be 4-byte aligned");
    if (!workspace || !aligned(workspace, 256))
        return reject(FT_ERR_INVALID_ARG, "workspace must be non-NULL and 256-byte aligned");
    if (bytes < kGroupWorkspace) return reject(FT_ERR_WORKSPACE, "workspace needs %zu bytes", kGroupWorkspace);
    return FT_OK;
}

// A matrix operand: rows `ld` elements apart, 16-byte aligned rows.
static ft_status check_matrix(const char *name, const void *p, int64_t ld, int cols, int unit)
{
    if (!p || !aligned(p, 16)) return reject(FT_ERR_INVALID_ARG, "%s must be non-NULL and 16-byte aligned", name);
    if (ld < cols || ld % unit || ld > (int64_t)1 << 32)
        return reject(FT_ERR_INVALID_ARG, "the row stride of %s must be a multiple of %d elements, at least %d (got %lld)", name,
                      unit, cols, (long long)ld);
    return FT_OK;
}

static ft_status check_out_dtype(int32_t dtype)
{
    if (dtype != FT_DTYPE_BF16 && dtype != FT_DTYPE_F32)
        return reject(FT_ERR_INVALID_ARG, "the output's dtype must be FT_DTYPE_BF16 or FT_DTYPE_F32");
    return FT_OK;
}

#define FT_TRY(...)                       \
    do {                                  \
        const ft_status st_ = __VA_ARGS__; \
        if (st_ != FT_OK) return st_;     \
    } while (0)

// No rows: nothing to compute, the status word is cleared.
static ft_status no_rows(void *workspace, cudaStream_t s)
{
    return finish(cudaMemsetAsync(workspace, 0, sizeof(int), s), "clearing the status word");
}

}  // namespace ftmoe

using namespace ftmoe;

extern "C" {

ft_status ft_moe_group_workspace_size(int32_t E, int32_t P, int32_t N, int32_t K, size_t *bytes)
{
    if (!bytes) return reject(FT_ERR_INVALID_ARG, "bytes is NULL");
    FT_TRY(check_sizes(E, P, N, K, 1, 1));
    *bytes = kGroupWorkspace;
    return report_error(FT_OK, "");
}

ft_status ft_moe_group_gemm(const void *x, int64_t ld_x, const void *w, const int32_t *offs, int32_t E, int32_t P,
                            int32_t N, int32_t K, void *y, int64_t ld_y, int32_t y_dtype, void *workspace,
                            size_t workspace_bytes, void *stream)
{
    FT_NVTX_RANGE("ft_moe_group_gemm");
    FT_TRY(check_sizes(E, P, N, K, 8, 8));
    FT_TRY(check_out_dtype(y_dtype));
    FT_TRY(check_group(offs, E, workspace, workspace_bytes));
    if (P == 0) return no_rows(workspace, static_cast<cudaStream_t>(stream));
    FT_TRY(check_matrix("x", x, ld_x, K, 8));
    FT_TRY(check_matrix("w", w, K, K, 8));
    FT_TRY(check_matrix("y", y, ld_y, N, 8));
    GroupGemm g = {};
    g.form = kGroupForward;
    g.offs = offs; g.E = E; g.P = P; g.N = N; g.K = K;
    g.x = x; g.ld_x = ld_x; g.w = w;
    g.out = y; g.ld_out = ld_y; g.out_f32 = y_dtype == FT_DTYPE_F32;
    g.status = static_cast<int *>(workspace);
    const StallScope stall;
    return finish(launch_group_gemm(g, static_cast<cudaStream_t>(stream)), "grouped product launch");
}

ft_status ft_moe_group_gemm_dgrad(const void *dy, int64_t ld_dy, const void *w, const int32_t *offs, int32_t E, int32_t P,
                                  int32_t N, int32_t K, void *dx, int64_t ld_dx, int32_t dx_dtype, void *workspace,
                                  size_t workspace_bytes, void *stream)
{
    FT_NVTX_RANGE("ft_moe_group_gemm_dgrad");
    FT_TRY(check_sizes(E, P, N, K, 8, 8));
    FT_TRY(check_out_dtype(dx_dtype));
    FT_TRY(check_group(offs, E, workspace, workspace_bytes));
    if (P == 0) return no_rows(workspace, static_cast<cudaStream_t>(stream));
    FT_TRY(check_matrix("dy", dy, ld_dy, N, 8));
    FT_TRY(check_matrix("w", w, K, K, 8));
    FT_TRY(check_matrix("dx", dx, ld_dx, K, 8));
    GroupGemm g = {};
    g.form = kGroupDgrad;
    g.offs = offs; g.E = E; g.P = P; g.N = N; g.K = K;
    g.dy = dy; g.ld_dy = ld_dy; g.w = w;
    g.out = dx; g.ld_out = ld_dx; g.out_f32 = dx_dtype == FT_DTYPE_F32;
    g.status = static_cast<int *>(workspace);
    const StallScope stall;
    return finish(launch_group_gemm(g, static_cast<cudaStream_t>(stream)), "grouped input-gradient launch");
}

ft_status ft_moe_group_gemm_wgrad(const void *dy, int64_t ld_dy, const void *x, int64_t ld_x, const int32_t *offs, int32_t E,
                                  int32_t P, int32_t N, int32_t K, void *dw, int32_t dw_dtype, int32_t accumulate,
                                  void *workspace, size_t workspace_bytes, void *stream)
{
    FT_NVTX_RANGE("ft_moe_group_gemm_wgrad");
    FT_TRY(check_sizes(E, P, N, K, 8, 8));
    FT_TRY(check_out_dtype(dw_dtype));
    if (accumulate != 0 && accumulate != 1) return reject(FT_ERR_INVALID_ARG, "accumulate must be 0 or 1");
    if (accumulate && dw_dtype != FT_DTYPE_F32)
        return reject(FT_ERR_UNSUPPORTED, "accumulate needs an fp32 dw (bf16 sums would lose the small terms)");
    FT_TRY(check_group(offs, E, workspace, workspace_bytes));
    FT_TRY(check_matrix("dw", dw, K, K, 8));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (P == 0) {
        if (!accumulate) {
            const size_t bytes = (size_t)E * N * K * (dw_dtype == FT_DTYPE_F32 ? 4 : 2);
            const cudaError_t e = cudaMemsetAsync(dw, 0, bytes, s);
            if (e != cudaSuccess) return finish(e, "clearing dw");
        }
        return no_rows(workspace, s);
    }
    FT_TRY(check_matrix("dy", dy, ld_dy, N, 8));
    FT_TRY(check_matrix("x", x, ld_x, K, 8));
    GroupGemm g = {};
    g.form = kGroupWgrad;
    g.offs = offs; g.E = E; g.P = P; g.N = N; g.K = K;
    g.dy = dy; g.ld_dy = ld_dy; g.x = x; g.ld_x = ld_x;
    g.out = dw; g.ld_out = K; g.out_f32 = dw_dtype == FT_DTYPE_F32; g.accumulate = accumulate;
    g.status = static_cast<int *>(workspace);
    const StallScope stall;
    return finish(launch_group_gemm(g, s), "grouped weight-gradient launch");
}

ft_status ft_moe_group_gemm_fp8(const void *x, int64_t ld_x, const float *x_scale, int64_t ld_xs, const void *w,
                                const float *w_scale, const int32_t *offs, int32_t E, int32_t P, int32_t N, int32_t K, void *y,
                                int64_t ld_y, int32_t y_dtype, void *workspace, size_t workspace_bytes, void *stream)
{
    FT_NVTX_RANGE("ft_moe_group_gemm_fp8");
    FT_TRY(check_sizes(E, P, N, K, 1, 16));
    FT_TRY(check_out_dtype(y_dtype));
    FT_TRY(check_group(offs, E, workspace, workspace_bytes));
    if (P == 0) return no_rows(workspace, static_cast<cudaStream_t>(stream));
    FT_TRY(check_matrix("x", x, ld_x, K, 16));
    FT_TRY(check_matrix("w", w, K, K, 16));
    FT_TRY(check_matrix("y", y, ld_y, N, 1));
    if (!x_scale || !aligned(x_scale, 4) || !w_scale || !aligned(w_scale, 4))
        return reject(FT_ERR_INVALID_ARG, "x_scale and w_scale must be non-NULL and 4-byte aligned");
    if (ld_xs < P) return reject(FT_ERR_INVALID_ARG, "the row stride of x_scale must be at least P");
    GroupGemm8 g = {};
    g.offs = offs; g.E = E; g.P = P; g.N = N; g.K = K;
    g.x = x; g.ld_x = ld_x; g.xs = x_scale; g.ld_xs = ld_xs;
    g.w = w; g.ws = w_scale;
    g.out = y; g.ld_out = ld_y; g.out_f32 = y_dtype == FT_DTYPE_F32;
    g.status = static_cast<int *>(workspace);
    const StallScope stall;
    return finish(launch_group_gemm_fp8(g, static_cast<cudaStream_t>(stream)), "grouped 8-bit product launch");
}

ft_status ft_moe_debug_group_plan(int32_t product, int32_t E, int32_t P, int32_t N, int32_t K, int32_t out_dtype,
                                  int32_t accumulate, int32_t *plan)
{
    if (product < FT_GROUP_FORWARD || product > FT_GROUP_FP8 || P < 1 || !plan || accumulate < 0 ||
        accumulate > (product == FT_GROUP_WGRAD && out_dtype == FT_DTYPE_F32))
        return reject(FT_ERR_INVALID_ARG, "need a product, P >= 1, accumulate for a wgrad into fp32 only, and room for the plan");
    const bool fp8 = product == FT_GROUP_FP8;
    FT_TRY(check_sizes(E, P, N, K, fp8 ? 1 : 8, fp8 ? 16 : 8));
    FT_TRY(check_out_dtype(out_dtype));
    if (fp8) {
        GroupGemm8 g = {};
        g.E = E; g.P = P; g.N = N; g.K = K;
        g.out_f32 = out_dtype == FT_DTYPE_F32;
        g.plan = plan;
        return finish(launch_group_gemm_fp8(g, nullptr), "plan of a grouped 8-bit product");
    }
    GroupGemm g = {};
    g.form = product == FT_GROUP_FORWARD ? kGroupForward : product == FT_GROUP_DGRAD ? kGroupDgrad : kGroupWgrad;
    g.E = E; g.P = P; g.N = N; g.K = K;
    g.out_f32 = out_dtype == FT_DTYPE_F32; g.accumulate = accumulate;
    g.plan = plan;
    return finish(launch_group_gemm(g, nullptr), "plan of a grouped product");
}

// Rows and columns of the row kernels.
static ft_status check_rows(int rows, int cols, int unit)
{
    if (rows < 0 || cols <= 0) return reject(FT_ERR_INVALID_ARG, "need rows >= 0 and columns > 0");
    if (rows > kMaxRows || cols > kMaxWidth || cols % unit)
        return reject(FT_ERR_UNSUPPORTED, "need rows <= 2^25 and columns <= 65536, a multiple of %d (got %d x %d)", unit, rows,
                      cols);
    return FT_OK;
}

// An operand of the SwiGLU kernels that take any alignment.
static ft_status check_values(const char *name, const void *p, int64_t ld, int cols)
{
    if (!p || !aligned(p, 2) || ld < cols)
        return reject(FT_ERR_INVALID_ARG, "%s must be non-NULL, 2-byte aligned, with rows of at least %d elements", name, cols);
    return FT_OK;
}

static ft_status check_scales(const float *scales, int64_t ld, int rows)
{
    if (!scales || !aligned(scales, 4) || ld < rows)
        return reject(FT_ERR_INVALID_ARG, "scales must be non-NULL, 4-byte aligned, with rows of at least %d elements", rows);
    return FT_OK;
}

ft_status ft_moe_quantize_fp8(const void *src, int32_t src_dtype, int64_t ld_src, int32_t rows, int32_t K, uint8_t *codes,
                              int64_t ld_codes, float *scales, int64_t ld_scales, void *stream)
{
    FT_NVTX_RANGE("ft_moe_quantize_fp8");
    if (src_dtype != FT_DTYPE_BF16 && src_dtype != FT_DTYPE_F32)
        return reject(FT_ERR_INVALID_ARG, "src_dtype must be FT_DTYPE_BF16 or FT_DTYPE_F32");
    FT_TRY(check_rows(rows, K, 16));
    if (rows == 0) return report_error(FT_OK, "");
    FT_TRY(check_matrix("src", src, ld_src, K, src_dtype == FT_DTYPE_F32 ? 4 : 8));
    FT_TRY(check_matrix("codes", codes, ld_codes, K, 16));
    FT_TRY(check_scales(scales, ld_scales, rows));
    return finish(launch_quantize_fp8(src, src_dtype == FT_DTYPE_F32, ld_src, rows, K, codes, ld_codes, scales, ld_scales,
                                      static_cast<cudaStream_t>(stream)),
                  "8-bit quantizer launch");
}

ft_status ft_moe_swiglu(const void *gu, int64_t ld_gu, const float *w, int32_t rows, int32_t I, void *h, int64_t ld_h,
                        void *stream)
{
    FT_NVTX_RANGE("ft_moe_swiglu");
    FT_TRY(check_rows(rows, I, 1));
    if (rows == 0) return report_error(FT_OK, "");
    FT_TRY(check_values("gu", gu, ld_gu, 2 * I));
    FT_TRY(check_values("h", h, ld_h, I));
    if (!aligned(w, 4)) return reject(FT_ERR_INVALID_ARG, "w must be 4-byte aligned");
    return finish(launch_swiglu(gu, ld_gu, w, rows, I, h, ld_h, static_cast<cudaStream_t>(stream)), "SwiGLU launch");
}

ft_status ft_moe_swiglu_quantize_fp8(const void *gu, int64_t ld_gu, const float *w, int32_t rows, int32_t I, uint8_t *codes,
                                     int64_t ld_codes, float *scales, int64_t ld_scales, void *stream)
{
    FT_NVTX_RANGE("ft_moe_swiglu_quantize_fp8");
    FT_TRY(check_rows(rows, I, 16));
    if (rows == 0) return report_error(FT_OK, "");
    FT_TRY(check_matrix("gu", gu, ld_gu, 2 * I, 8));
    FT_TRY(check_matrix("codes", codes, ld_codes, I, 16));
    FT_TRY(check_scales(scales, ld_scales, rows));
    if (!aligned(w, 4)) return reject(FT_ERR_INVALID_ARG, "w must be 4-byte aligned");
    return finish(launch_swiglu_quantize_fp8(gu, ld_gu, w, rows, I, codes, ld_codes, scales, ld_scales,
                                             static_cast<cudaStream_t>(stream)),
                  "8-bit SwiGLU launch");
}

ft_status ft_moe_swiglu_backward(const void *gu, int64_t ld_gu, const float *w, const void *dh, int64_t ld_dh, int32_t rows,
                                 int32_t I, void *dgu, int64_t ld_dgu, float *dw, void *stream)
{
    FT_NVTX_RANGE("ft_moe_swiglu_backward");
    FT_TRY(check_rows(rows, I, 1));
    if (rows == 0) return report_error(FT_OK, "");
    FT_TRY(check_values("gu", gu, ld_gu, 2 * I));
    FT_TRY(check_values("dh", dh, ld_dh, I));
    FT_TRY(check_values("dgu", dgu, ld_dgu, 2 * I));
    if (!aligned(w, 4) || !aligned(dw, 4)) return reject(FT_ERR_INVALID_ARG, "w and dw must be 4-byte aligned");
    return finish(launch_swiglu_backward(gu, ld_gu, w, dh, ld_dh, rows, I, dgu, ld_dgu, dw, static_cast<cudaStream_t>(stream)),
                  "SwiGLU backward launch");
}

}  // extern "C"
