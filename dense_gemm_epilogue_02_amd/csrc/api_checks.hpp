// api_checks.hpp -- what the C entries of the operators around the GEMMs check
// with (block_api.cpp, model_api.cpp). Host code only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm.h"

namespace mg {

// Failure reporting of gemm_api.cpp.
gemm_status api_fail(gemm_status s, const char *fmt, ...);
gemm_status api_ok();

inline bool is_float(gemm_dtype t) { return t == GEMM_F32 || t == GEMM_F16 || t == GEMM_BF16; }
inline int64_t size_of(gemm_dtype t) { return t == GEMM_F32 ? 4 : 2; }
inline int64_t align16(int64_t n) { return (n + 15) / 16 * 16; }
inline bool misaligned(const void *p, unsigned n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }
inline long long ll(int64_t v) { return (long long)v; }

constexpr int64_t kMaxDim = 1LL << 31;   // rows and columns stay below
constexpr int64_t kMaxElems = 1LL << 46;

inline gemm_status launched(hipError_t e, const char *what) {
    if (e == hipSuccess) return api_ok();
    return api_fail(GEMM_HIP_ERROR, "%s: launch failed: %s (%d)", what, hipGetErrorString(e), (int)e);
}

// A matrix argument: sizes, leading dimension, pointer (needed unless empty).
inline gemm_status check_matrix(const char *what, const char *name, const void *p, gemm_dtype type,
                         int64_t rows, int64_t cols, int64_t ld) {
    if (!is_float(type))
        return api_fail(GEMM_UNSUPPORTED, "%s: %s must be F32, F16 or BF16", what, name);
    if (rows < 0 || cols < 0)
        return api_fail(GEMM_INVALID_ARG, "%s: negative size %lld x %lld of %s", what, ll(rows),
                        ll(cols), name);
    if (rows >= kMaxDim || cols >= kMaxDim)
        return api_fail(GEMM_UNSUPPORTED, "%s: %s has a dimension of 2^31 or more", what, name);
    if (rows == 0 || cols == 0) return GEMM_OK;
    if (!p) return api_fail(GEMM_INVALID_ARG, "%s: %s is NULL", what, name);
    if (rows > 1 && ld < cols)
        return api_fail(GEMM_INVALID_ARG, "%s: leading dimension %lld of %s is below its %lld columns",
                        what, ll(ld), name, ll(cols));
    if (ld > kMaxElems / rows)
        return api_fail(GEMM_UNSUPPORTED, "%s: %s spans more than 2^46 elements", what, name);
    if (misaligned(p, (unsigned)size_of(type)))
        return api_fail(GEMM_INVALID_ARG, "%s: %s is not aligned to its element", what, name);
    return GEMM_OK;
}

inline gemm_status check_vector(const char *what, const char *name, const void *p, gemm_dtype type) {
    if (p && misaligned(p, (unsigned)size_of(type)))
        return api_fail(GEMM_INVALID_ARG, "%s: %s is not aligned to its element", what, name);
    return GEMM_OK;
}

inline gemm_status check_workspace(const char *what, const void *p, int64_t have, int64_t need) {
    if (need <= 0) return GEMM_OK;
    if (!p || have < need)
        return api_fail(GEMM_INVALID_ARG, "%s: workspace of %lld bytes, needs %lld", what,
                        p ? ll(have) : 0LL, ll(need));
    if (misaligned(p, 16))
        return api_fail(GEMM_INVALID_ARG, "%s: workspace is not 16-byte aligned", what);
    return GEMM_OK;
}

#define CHECK(expr)                          \
    do {                                     \
        const gemm_status st_ = (expr);      \
        if (st_ != GEMM_OK) return st_;      \
    } while (0)

}  // namespace mg
