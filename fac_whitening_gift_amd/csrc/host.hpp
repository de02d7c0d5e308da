// Host-side helpers shared by the entry points (api.cpp, api_layer.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/gift.h"

namespace gift {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxDim = int64_t(1) << 24;
constexpr int64_t kMaxElems = int64_t(1) << 36;

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// Record the one-line detail of gift_last_error() and return s.
gift_status fail(gift_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
gift_status hip_fail(hipError_t e, const char* where);
gift_status check_ws(void* ws, size_t ws_bytes, size_t need);

}  // namespace gift
