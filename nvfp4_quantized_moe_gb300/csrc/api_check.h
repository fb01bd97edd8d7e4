// Argument checks that the entry points of the expert products and of the row kernels around them share.
#pragma once

#include <cuda_runtime.h>
#include <stdarg.h>
#include <stdio.h>

#include "ft_moe.h"
#include "ftmoe_internal.h"

namespace ftmoe {

inline ft_status reject(ft_status code, const char *fmt, ...)
{
    char text[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof(text), fmt, ap);
    va_end(ap);
    return report_error(code, text);
}

inline ft_status finish(cudaError_t e, const char *what)
{
    if (e == cudaSuccess) return report_error(FT_OK, "");
    return reject(FT_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

inline bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

constexpr int kMaxRows = 1 << 25;   // T <= 2^20 tokens of up to 32 slots
constexpr int kMaxWidth = 1 << 16;
// A matrix operand: rows `ld` elements apart, 16-byte aligned rows.
inline ft_status check_matrix(const char *name, const void *p, int64_t ld, int cols, int unit)
{
    if (!p || !aligned(p, 16)) return reject(FT_ERR_INVALID_ARG, "%s must be non-NULL and 16-byte aligned", name);
    if (ld < cols || ld % unit || ld > (int64_t)1 << 32)
        return reject(FT_ERR_INVALID_ARG, "the row stride of %s must be a multiple of %d elements, at least %d (got %lld)", name,
                      unit, cols, (long long)ld);
    return FT_OK;
}

inline ft_status check_out_dtype(int32_t dtype)
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

// Rows and columns of the row kernels.
inline ft_status check_rows(int rows, int cols, int unit)
{
    if (rows < 0 || cols <= 0) return reject(FT_ERR_INVALID_ARG, "need rows >= 0 and columns > 0");
    if (rows > kMaxRows || cols > kMaxWidth || cols % unit)
        return reject(FT_ERR_UNSUPPORTED, "need rows <= 2^25 and columns <= 65536, a multiple of %d (got %d x %d)", unit, rows,
                      cols);
    return FT_OK;
}

// An operand of the SwiGLU kernels that take any alignment.
inline ft_status check_values(const char *name, const void *p, int64_t ld, int cols)
{
    if (!p || !aligned(p, 2) || ld < cols)
        return reject(FT_ERR_INVALID_ARG, "%s must be non-NULL, 2-byte aligned, with rows of at least %d elements", name, cols);
    return FT_OK;
}

inline ft_status check_scales(const float *scales, int64_t ld, int rows)
{
    if (!scales || !aligned(scales, 4) || ld < rows)
        return reject(FT_ERR_INVALID_ARG, "scales must be non-NULL, 4-byte aligned, with rows of at least %d elements", rows);
    return FT_OK;
}

}  // namespace ftmoe
