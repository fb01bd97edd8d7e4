// extern "C" entry points of what stands around the expert products in a layer: the residual norm, and tokens
// sorted by expert and back. Argument validation and launches; see include/ft_moe.h for the contract of every call.
#include <cuda_runtime.h>
#include <math.h>

#include "api_check.h"
#include "ft_moe.h"
#include "ftmoe_internal.h"

namespace ftmoe {

constexpr int kMaxTopK = 32;

static ft_status check_norm(int rows, int H)
{
    if (rows < 0 || H <= 0) return reject(FT_ERR_INVALID_ARG, "need rows >= 0 and H > 0 (got %d x %d)", rows, H);
    if (rows > kMaxRows || H > kMaxNormWidth)
        return reject(FT_ERR_UNSUPPORTED, "need rows <= 2^25 and H <= %d (got %d x %d)", kMaxNormWidth, rows, H);
    return FT_OK;
}

// Rows of bf16 or fp32 elements, aligned to one element.
static ft_status check_floats(const char *name, const void *p, int64_t ld, int32_t dtype, int cols)
{
    if (dtype != FT_DTYPE_BF16 && dtype != FT_DTYPE_F32)
        return reject(FT_ERR_INVALID_ARG, "the dtype of %s must be FT_DTYPE_BF16 or FT_DTYPE_F32", name);
    if (!p || !aligned(p, dtype == FT_DTYPE_F32 ? 4 : 2) || ld < cols || ld > (int64_t)1 << 32)
        return reject(FT_ERR_INVALID_ARG, "%s must be non-NULL and aligned, with rows of at least %d elements", name, cols);
    return FT_OK;
}

static ft_status check_order(int T, int k, int P)
{
    if (T < 0 || k <= 0 || P < 0) return reject(FT_ERR_INVALID_ARG, "need T >= 0, k > 0 and P >= 0 (got T %d, k %d, P %d)", T, k, P);
    if (k > kMaxTopK || T > 1 << 20 || P > kMaxRows)
        return reject(FT_ERR_UNSUPPORTED, "need k <= %d, T <= 2^20 and P <= 2^25 (got T %d, k %d, P %d)", kMaxTopK, T, k, P);
    return FT_OK;
}

static ft_status check_words(const char *name, const void *p)
{
    if (!p || !aligned(p, 4)) return reject(FT_ERR_INVALID_ARG, "%s must be non-NULL and 4-byte aligned", name);
    return FT_OK;
}

}  // namespace ftmoe

using namespace ftmoe;

extern "C" {

ft_status ft_moe_rmsnorm(const void *x, int64_t ld_x, const void *residual, int64_t ld_residual, void *total,
                         int64_t ld_total, int32_t total_dtype, const void *w, int32_t w_dtype, float w_offset, float eps,
                         int32_t rows, int32_t H, void *y, int64_t ld_y, uint8_t *codes, int64_t ld_codes, float *scales,
                         int64_t ld_scales, float *rstd, void *stream)
{
    FT_NVTX_RANGE("ft_moe_rmsnorm");
    FT_TRY(check_norm(rows, H));
    if (!(eps >= 0.f) || !isfinite(eps) || !isfinite(w_offset))
        return reject(FT_ERR_INVALID_ARG, "need a finite eps >= 0 and a finite w_offset");
    if (codes && H % 16) return reject(FT_ERR_UNSUPPORTED, "8-bit outputs need H a multiple of 16 (got %d)", H);
    if (rows == 0) return report_error(FT_OK, "");
    if (!y && !codes) return reject(FT_ERR_INVALID_ARG, "need y, codes or both");
    FT_TRY(check_floats("x", x, ld_x, FT_DTYPE_BF16, H));
    if (residual || total) {
        FT_TRY(check_floats("residual", residual, ld_residual, total_dtype, H));
        FT_TRY(check_floats("total", total, ld_total, total_dtype, H));
    }
    FT_TRY(check_floats("w", w, H, w_dtype, H));
    if (y) FT_TRY(check_floats("y", y, ld_y, FT_DTYPE_BF16, H));
    if (codes) {
        FT_TRY(check_matrix("codes", codes, ld_codes, H, 16));
        FT_TRY(check_scales(scales, ld_scales, rows));
    }
    if (!aligned(rstd, 4)) return reject(FT_ERR_INVALID_ARG, "rstd must be 4-byte aligned");
    NormParams p = {};
    p.x = x; p.ld_x = ld_x;
    p.residual = residual; p.ld_residual = ld_residual;
    p.total = total; p.ld_total = ld_total; p.total_f32 = total_dtype == FT_DTYPE_F32;
    p.w = w; p.w_f32 = w_dtype == FT_DTYPE_F32; p.offset = w_offset; p.eps = eps;
    p.rows = rows; p.H = H;
    p.y = y; p.ld_y = ld_y;
    p.codes = codes; p.ld_codes = ld_codes; p.scales = scales; p.ld_scales = ld_scales;
    p.rstd = rstd;
    return finish(launch_rmsnorm(p, static_cast<cudaStream_t>(stream)), "RMS norm launch");
}

ft_status ft_moe_rmsnorm_workspace_size(int32_t rows, int32_t H, size_t *bytes)
{
    if (!bytes) return reject(FT_ERR_INVALID_ARG, "bytes is NULL");
    FT_TRY(check_norm(rows, H));
    *bytes = (size_t)norm_parts(rows, H) * H * sizeof(float);
    return report_error(FT_OK, "");
}

ft_status ft_moe_rmsnorm_backward(const void *dy, int64_t ld_dy, const void *total, int64_t ld_total, int32_t total_dtype,
                                  const void *w, int32_t w_dtype, float w_offset, const float *rstd, const void *dtotal,
                                  int64_t ld_dtotal, int32_t rows, int32_t H, void *dx, int64_t ld_dx, float *dw,
                                  int32_t accumulate, void *workspace, size_t workspace_bytes, void *stream)
{
    FT_NVTX_RANGE("ft_moe_rmsnorm_backward");
    FT_TRY(check_norm(rows, H));
    if (!isfinite(w_offset)) return reject(FT_ERR_INVALID_ARG, "need a finite w_offset");
    if (accumulate != 0 && accumulate != 1) return reject(FT_ERR_INVALID_ARG, "accumulate must be 0 or 1");
    if (!aligned(dw, 4)) return reject(FT_ERR_INVALID_ARG, "dw must be 4-byte aligned");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0) {
        if (dw && !accumulate) return finish(cudaMemsetAsync(dw, 0, sizeof(float) * H, s), "clearing dw");
        return report_error(FT_OK, "");
    }
    FT_TRY(check_floats("dy", dy, ld_dy, FT_DTYPE_BF16, H));
    FT_TRY(check_floats("total", total, ld_total, total_dtype, H));
    FT_TRY(check_floats("w", w, H, w_dtype, H));
    FT_TRY(check_words("rstd", rstd));
    if (dtotal) FT_TRY(check_floats("dtotal", dtotal, ld_dtotal, total_dtype, H));
    FT_TRY(check_floats("dx", dx, ld_dx, total_dtype, H));
    if (dw) {
        const size_t need = (size_t)norm_parts(rows, H) * H * sizeof(float);
        if (!workspace || !aligned(workspace, 256))
            return reject(FT_ERR_INVALID_ARG, "workspace must be non-NULL and 256-byte aligned");
        if (workspace_bytes < need) return reject(FT_ERR_WORKSPACE, "workspace needs %zu bytes", need);
    }
    NormBackParams p = {};
    p.dy = dy; p.ld_dy = ld_dy;
    p.total = total; p.ld_total = ld_total; p.total_f32 = total_dtype == FT_DTYPE_F32;
    p.w = w; p.w_f32 = w_dtype == FT_DTYPE_F32; p.offset = w_offset;
    p.rstd = rstd;
    p.dtotal = dtotal; p.ld_dtotal = ld_dtotal;
    p.rows = rows; p.H = H;
    p.dx = dx; p.ld_dx = ld_dx;
    return finish(launch_rmsnorm_backward(p, dw, accumulate, workspace, s), "RMS norm backward launch");
}

ft_status ft_moe_dispatch(const void *x, int64_t ld_x, int32_t row_bytes, int32_t T, int32_t k, const int32_t *slot, int32_t P,
                          const int32_t *count, void *out, int64_t ld_out, const void *x_scale, int64_t ld_xs,
                          int32_t scale_blocks, void *out_scale, int64_t ld_os, const float *w, float *row_w, int32_t *pos,
                          void *stream)
{
    FT_NVTX_RANGE("ft_moe_dispatch");
    FT_TRY(check_order(T, k, P));
    if (row_bytes <= 0 || row_bytes % 2 || scale_blocks < 0)
        return reject(FT_ERR_INVALID_ARG, "need rows of a positive even number of bytes (got %d) and scale_blocks >= 0", row_bytes);
    if (row_bytes > 4 * kMaxWidth || scale_blocks > kMaxWidth / 128)
        return reject(FT_ERR_UNSUPPORTED, "need rows of at most 262144 bytes and at most 512 scale blocks");
    if (!aligned(pos, 4)) return reject(FT_ERR_INVALID_ARG, "pos must be 4-byte aligned");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (P == 0) {
        if (pos && T > 0) return finish(cudaMemsetAsync(pos, 0xFF, sizeof(int32_t) * (size_t)T * k, s), "clearing pos");
        return report_error(FT_OK, "");
    }
    FT_TRY(check_words("slot", slot));
    if (!aligned(count, 4)) return reject(FT_ERR_INVALID_ARG, "count must be 4-byte aligned");
    const auto rows_ok = [&](const void *p, int64_t ld) {
        return p && aligned(p, 2) && ld >= row_bytes && ld % 2 == 0 && ld <= (int64_t)1 << 34;
    };
    if (T > 0 && !rows_ok(x, ld_x))
        return reject(FT_ERR_INVALID_ARG, "x must be non-NULL and 2-byte aligned, with rows at least %d bytes apart", row_bytes);
    if (!rows_ok(out, ld_out))
        return reject(FT_ERR_INVALID_ARG, "out must be non-NULL and 2-byte aligned, with rows at least %d bytes apart", row_bytes);
    if (scale_blocks) {
        if (T > 0) FT_TRY(check_words("x_scale", x_scale));
        FT_TRY(check_words("out_scale", out_scale));
        if (ld_xs < T || ld_os < P) return reject(FT_ERR_INVALID_ARG, "need ld_xs >= T and ld_os >= P");
    }
    if (row_w) {
        FT_TRY(check_words("row_w", row_w));
        if (T > 0) FT_TRY(check_words("w", w));
    }
    DispatchParams p = {};
    p.x = static_cast<const char *>(x); p.ld_x = ld_x;
    p.out = static_cast<char *>(out); p.ld_out = ld_out;
    p.row_bytes = row_bytes;
    p.T = T; p.k = k; p.P = P;
    p.slot = slot; p.count = count;
    p.x_scale = static_cast<const uint32_t *>(x_scale); p.ld_xs = ld_xs;
    p.out_scale = static_cast<uint32_t *>(out_scale); p.ld_os = ld_os;
    p.blocks = scale_blocks;
    p.w = w; p.row_w = row_w;
    p.pos = T > 0 ? pos : nullptr;
    return finish(launch_dispatch(p, s), "dispatch launch");
}

static ft_status combine_rows(const void *y, int64_t ld_y, int32_t y_dtype, const int32_t *pos, const float *w, int32_t T,
                              int32_t k, int32_t P, int32_t H, const void *add, int64_t ld_add, void *out, int64_t ld_out,
                              int32_t out_dtype, const float *drow_w, float *dw, const char *what, void *stream)
{
    FT_TRY(check_order(T, k, P));
    FT_TRY(check_rows(T, H, 1));
    if (T == 0) return report_error(FT_OK, "");
    if (P > 0) FT_TRY(check_floats("the rows", y, ld_y, y_dtype, H));
    FT_TRY(check_words("pos", pos));
    if (!aligned(w, 4)) return reject(FT_ERR_INVALID_ARG, "w must be 4-byte aligned");
    if (add) FT_TRY(check_floats("add", add, ld_add, out_dtype, H));
    FT_TRY(check_floats("the result", out, ld_out, out_dtype, H));
    if (dw) {
        FT_TRY(check_words("dw", dw));
        if (P > 0) FT_TRY(check_words("drow_w", drow_w));
    }
    CombineParams p = {};
    p.y = y; p.ld_y = ld_y;
    p.add = add; p.ld_add = ld_add;
    p.out = out; p.ld_out = ld_out;
    p.pos = pos; p.w = w;
    p.drow_w = drow_w; p.dw = dw;
    p.T = T; p.k = k; p.P = P; p.H = H;
    return finish(launch_combine_rows(p, y_dtype == FT_DTYPE_F32, out_dtype == FT_DTYPE_F32, static_cast<cudaStream_t>(stream)), what);
}

ft_status ft_moe_dispatch_backward(const void *dout, int64_t ld_dout, int32_t dout_dtype, const int32_t *pos, int32_t T,
                                   int32_t k, int32_t P, int32_t H, const float *drow_w, void *dx, int64_t ld_dx,
                                   int32_t dx_dtype, float *dw, void *stream)
{
    FT_NVTX_RANGE("ft_moe_dispatch_backward");
    return combine_rows(dout, ld_dout, dout_dtype, pos, nullptr, T, k, P, H, nullptr, 0, dx, ld_dx, dx_dtype, drow_w, dw,
                        "dispatch backward launch", stream);
}

ft_status ft_moe_combine(const void *y, int64_t ld_y, int32_t y_dtype, const int32_t *pos, const float *w, int32_t T, int32_t k,
                         int32_t P, int32_t H, const void *add, int64_t ld_add, void *out, int64_t ld_out, int32_t out_dtype,
                         void *stream)
{
    FT_NVTX_RANGE("ft_moe_combine");
    return combine_rows(y, ld_y, y_dtype, pos, w, T, k, P, H, add, ld_add, out, ld_out, out_dtype, nullptr, nullptr,
                        "combine launch", stream);
}

ft_status ft_moe_combine_backward(const void *dout, int64_t ld_dout, int32_t dout_dtype, const void *y, int64_t ld_y,
                                  int32_t y_dtype, const int32_t *pos, const float *w, int32_t T, int32_t k, int32_t P,
                                  int32_t H, void *dy, int64_t ld_dy, float *dw, void *stream)
{
    FT_NVTX_RANGE("ft_moe_combine_backward");
    FT_TRY(check_order(T, k, P));
    FT_TRY(check_rows(T, H, 1));
    if (T == 0) return report_error(FT_OK, "");
    FT_TRY(check_floats("dout", dout, ld_dout, dout_dtype, H));
    FT_TRY(check_words("pos", pos));
    if (!aligned(w, 4) || !aligned(dw, 4)) return reject(FT_ERR_INVALID_ARG, "w and dw must be 4-byte aligned");
    if (P > 0) {
        if (dw) FT_TRY(check_floats("y", y, ld_y, y_dtype, H));
        FT_TRY(check_floats("dy", dy, ld_dy, FT_DTYPE_BF16, H));
    }
    CombineBackParams p = {};
    p.dout = dout; p.ld_dout = ld_dout;
    p.y = y; p.ld_y = ld_y;
    p.dy = dy; p.ld_dy = ld_dy;
    p.pos = pos; p.w = w; p.dw = dw;
    p.T = T; p.k = k; p.P = P; p.H = H;
    return finish(launch_combine_backward(p, dout_dtype == FT_DTYPE_F32, y_dtype == FT_DTYPE_F32, static_cast<cudaStream_t>(stream)),
                  "combine backward launch");
}

}  // extern "C"
