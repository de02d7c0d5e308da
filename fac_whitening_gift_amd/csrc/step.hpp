// What xent.hip (cross entropy over a vocabulary), block_norm.hip (norms
// between blocks), grad_clip.hip (gradient norm and clipping) and the entry
// points in api_step.cpp share.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/gift.h"

namespace gift {

// xent.hip: a bf16 matrix, rows x cols, element (i, j) at i * ld + j
struct XeMatrix {
  const uint16_t* p;
  int64_t rows;
  int64_t cols;
  int64_t ld;
};
struct XeGrad {
  void* dX;        // rows x d bf16, or NULL
  int64_t ld_dx;
  void* dW;        // vocab x d, or NULL
  int dw_dtype;
  int64_t ld_dw;
  bool accumulate;
};
constexpr int64_t kXeMaxRows = int64_t(1) << 20, kXeMaxVocab = int64_t(1) << 20, kXeMaxD = int64_t(1) << 16;

size_t xent_forward_ws(int64_t rows, int64_t d, int64_t vocab);
hipError_t launch_xent_forward(const XeMatrix& X, const XeMatrix& W, const int64_t* targets, float* loss,
                               float* lse, uint32_t* flags, void* ws, hipStream_t s);
size_t xent_backward_ws(int64_t rows, int64_t d, int64_t vocab, bool dx, bool dw, int dw_dtype);
hipError_t launch_xent_backward(const XeMatrix& X, const XeMatrix& W, const int64_t* targets,
                                const float* lse, const float* dloss, const XeGrad& g, void* ws,
                                hipStream_t s);


// block_norm.hip
constexpr int64_t kBlockNormMaxD = 16384;  // widest row that its lanes hold
hipError_t launch_block_norm_forward(const gift_block_norm& p, const void* Y, const void* H, void* H2, void* X,
                                     float* stats, hipStream_t s);
size_t block_norm_backward_ws(int64_t rows, int64_t d, int64_t gates);
hipError_t launch_block_norm_backward(const gift_block_norm& p, const void* dX, const void* dH2, const void* Y,
                                      const void* H2, const float* stats, void* dY, void* dH,
                                      const gift_block_norm_grads& g, bool accumulate, void* ws, hipStream_t s);

// grad_clip.hip
constexpr int kGradMaxTensors = 1 << 16;
bool grad_size_ok(const gift_tensor* t, int n);
size_t grad_ws(int n);
hipError_t launch_grad(const gift_tensor* t, const gift_tensor* out, int n, const double* given, bool scale,
                       float max_norm, float eps, double* sum, float* norm, uint32_t* flags, void* ws, hipStream_t s);

}  // namespace gift
