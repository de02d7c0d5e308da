// Argument checks shared by the entry points of api_layer.cpp and api_step.cpp.
#pragma once

#include "host.hpp"

namespace gift {

inline bool dtype_ok(int t) { return t == GIFT_DTYPE_F32 || t == GIFT_DTYPE_BF16; }
inline size_t dtype_size(int t) { return t == GIFT_DTYPE_BF16 ? 2 : 4; }
inline bool aligned_to(const void* p, size_t n) { return (uintptr_t)p % n == 0; }

inline bool size_ok(int64_t rows, int64_t cols) {
  return rows >= 1 && cols >= 1 && rows <= kMaxDim && cols <= kMaxDim && rows * cols <= kMaxElems;
}

// A dense or strided rows x cols matrix.
inline gift_status check_matrix(const char* name, const void* p, int dtype, int64_t rows, int64_t cols,
                                int64_t ld) {
  if (!dtype_ok(dtype)) return fail(GIFT_ERR_INVALID_ARG, "%s: unknown dtype %d", name, dtype);
  if (!size_ok(rows, cols))
    return fail(GIFT_ERR_UNSUPPORTED_SHAPE, "%s: %lld x %lld out of range", name, (long long)rows,
                (long long)cols);
  if (ld < cols || ld > (int64_t(1) << 40))
    return fail(GIFT_ERR_UNSUPPORTED_SHAPE, "%s: leading dimension %lld for rows of %lld", name,
                (long long)ld, (long long)cols);
  if (!p || !aligned_to(p, dtype_size(dtype)))
    return fail(GIFT_ERR_INVALID_ARG, "%s is NULL or not aligned to its elements", name);
  return GIFT_OK;
}

inline gift_status check_flags(const uint32_t* f) {
  return aligned_to(f, 4) ? GIFT_OK : fail(GIFT_ERR_INVALID_ARG, "dev_flags must be 4-byte aligned");
}

inline gift_status check_vec(const char* name, const float* p) {
  return aligned_to(p, 4) ? GIFT_OK : fail(GIFT_ERR_INVALID_ARG, "%s must be 4-byte aligned", name);
}

#define GIFT_TRY(x)                        \
  do {                                     \
    const gift_status try_s = (x);         \
    if (try_s != GIFT_OK) return try_s;    \
  } while (0)

inline gift_status launched(hipError_t e) { return e == hipSuccess ? GIFT_OK : hip_fail(e, "kernel launch"); }

}  // namespace gift
