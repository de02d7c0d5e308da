// What mx.hip (MXFP4 operands and products), norm.hip (layer and RMS norm)
// and the entry points in api_layer.cpp share.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/gift.h"

namespace gift {

// 16-byte accesses at any element of a T array.  Rows of odd length start
// anywhere; global memory takes wide accesses there, and the element-aligned
// type makes the compiler emit them.
template <class T>
using any16 = unsigned __attribute__((ext_vector_type(4), aligned(sizeof(T))));

template <class T>
__device__ __forceinline__ uint4 ld16(const T* p) {
  return __builtin_bit_cast(uint4, *reinterpret_cast<const any16<T>*>(p));
}
template <class T>
__device__ __forceinline__ void st16(T* p, const uint4& v) {
  *reinterpret_cast<any16<T>*>(p) = __builtin_bit_cast(any16<T>, v);
}
// around the caches
template <class T>
__device__ __forceinline__ void st16_nt(T* p, const uint4& v) {
  __builtin_nontemporal_store(__builtin_bit_cast(any16<T>, v), reinterpret_cast<any16<T>*>(p));
}

constexpr int kMxRows = 64;                      // rows of an operand panel
constexpr int kMxStep = 128;                     // k elements of a step
constexpr int kMxPanel = GIFT_MX_PANEL_BYTES;    // bytes of a panel's step

struct MxPlan {
  int rows;       // of a workgroup: 64 (k_mx_few) or 128 (k_mx_gemm)
  int cols;       // 16, 32, 64 or 128, 256
  int n_split;    // k splits
  int per_split;  // k steps of a split
};
MxPlan mx_plan(int64_t M, int64_t N, int64_t k);
size_t mx_matmul_ws(int64_t M, int64_t N, int64_t k);
int mx_linear_cols(int64_t M, int64_t N, int64_t k);  // 0: two launches

hipError_t launch_mx_quantize(const void* X, int dtype, int64_t rows, int64_t cols, int64_t ld,
                              uint8_t* by_row, uint8_t* by_col, uint32_t* flags, hipStream_t s);
hipError_t launch_mx_dequantize(const uint8_t* A, int64_t rows, int64_t k, void* out, int dtype,
                                int64_t ld, hipStream_t s);
hipError_t launch_mx_matmul(const uint8_t* A, const uint8_t* B, int64_t M, int64_t N, int64_t k,
                            const float* bias, void* C, int dtype, int64_t ldc, bool accumulate,
                            void* ws, hipStream_t s);
hipError_t launch_mx_linear_few(const void* X, int x_dtype, int64_t M, int64_t ldx, const uint8_t* W,
                                int64_t N, int64_t k, const float* bias, void* Y, int dtype,
                                int64_t ldy, uint32_t* flags, hipStream_t s);

// norm.hip
hipError_t launch_norm_forward(const void* X, int dtype, int64_t rows, int64_t d, int kind,
                               const float* weight, const float* bias, float eps, void* Y,
                               float* mean, float* rstd, hipStream_t s);
size_t norm_backward_ws(int64_t rows, int64_t d);
hipError_t launch_norm_backward(const void* dY, const void* X, int dtype, int64_t rows, int64_t d,
                                int kind, const float* weight, const float* mean, const float* rstd,
                                void* dX, float* dweight, float* dbias, bool accumulate, void* ws,
                                hipStream_t s);

}  // namespace gift
