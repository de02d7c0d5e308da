// Entry points of a training step around its layers (gift_xent_* of
// include/gift.h): argument validation, then the launchers of xent.hip.
#include "checks.hpp"
#include "step.hpp"

using namespace gift;

namespace {

bool xent_size_ok(int64_t rows, int64_t d, int64_t vocab) {
  return rows >= 1 && d >= 1 && vocab >= 1 && rows <= kXeMaxRows && d <= kXeMaxD && vocab <= kXeMaxVocab &&
         rows * d <= kMaxElems && vocab * d <= kMaxElems;
}

gift_status check_xent(const void* X, int64_t rows, int64_t d, int64_t ldx, const void* W, int64_t vocab, int64_t ldw,
                       const int64_t* targets) {
  if (!xent_size_ok(rows, d, vocab))
    return fail(GIFT_ERR_UNSUPPORTED_SHAPE, "%lld rows of %lld over a vocabulary of %lld out of range", (long long)rows,
                (long long)d, (long long)vocab);
  GIFT_TRY(check_matrix("X", X, GIFT_DTYPE_BF16, rows, d, ldx));
  GIFT_TRY(check_matrix("W", W, GIFT_DTYPE_BF16, vocab, d, ldw));
  if (!targets || !aligned_to(targets, 8)) return fail(GIFT_ERR_INVALID_ARG, "targets is NULL or not 8-byte aligned");
  return GIFT_OK;
}

XeMatrix matrix(const void* p, int64_t rows, int64_t cols, int64_t ld) {
  return XeMatrix{static_cast<const uint16_t*>(p), rows, cols, ld};
}

}  // namespace

extern "C" {

size_t gift_xent_forward_workspace_bytes(int64_t rows, int64_t d, int64_t vocab) {
  return xent_size_ok(rows, d, vocab) ? xent_forward_ws(rows, d, vocab) : 0;
}

gift_status gift_xent_forward(const void* X, int64_t rows, int64_t d, int64_t ldx, const void* W, int64_t vocab,
                              int64_t ldw, const int64_t* targets, float* loss, float* lse, uint32_t* dev_flags,
                              void* ws, size_t ws_bytes, void* stream) {
  GIFT_TRY(check_xent(X, rows, d, ldx, W, vocab, ldw, targets));
  GIFT_TRY(check_vec("loss", loss));
  GIFT_TRY(check_vec("lse", lse));
  if (!loss && !lse) return fail(GIFT_ERR_INVALID_ARG, "loss and lse are both NULL");
  if (loss == lse) return fail(GIFT_ERR_INVALID_ARG, "loss and lse are the same buffer");
  GIFT_TRY(check_flags(dev_flags));
  GIFT_TRY(check_ws(ws, ws_bytes, xent_forward_ws(rows, d, vocab)));
  return launched(launch_xent_forward(matrix(X, rows, d, ldx), matrix(W, vocab, d, ldw), targets, loss, lse, dev_flags,
                                      ws, (hipStream_t)stream));
}

size_t gift_xent_backward_workspace_bytes(int64_t rows, int64_t d, int64_t vocab, int want_dx, int want_dw,
                                          int dw_dtype) {
  if (!xent_size_ok(rows, d, vocab) || !dtype_ok(dw_dtype) || (!want_dx && !want_dw)) return 0;
  return xent_backward_ws(rows, d, vocab, want_dx != 0, want_dw != 0, dw_dtype);
}

gift_status gift_xent_backward(const void* X, int64_t rows, int64_t d, int64_t ldx, const void* W, int64_t vocab,
                               int64_t ldw, const int64_t* targets, const float* lse, const float* dloss, void* dX,
                               int64_t ld_dx, void* dW, int dw_dtype, int64_t ld_dw, int accumulate, void* ws,
                               size_t ws_bytes, void* stream) {
  GIFT_TRY(check_xent(X, rows, d, ldx, W, vocab, ldw, targets));
  if (!dX && !dW) return fail(GIFT_ERR_INVALID_ARG, "dX and dW are both NULL");
  if (!lse) return fail(GIFT_ERR_INVALID_ARG, "the forward pass's lse is NULL");
  GIFT_TRY(check_vec("lse", lse));
  GIFT_TRY(check_vec("dloss", dloss));
  if (!dtype_ok(dw_dtype)) return fail(GIFT_ERR_INVALID_ARG, "dW: unknown dtype %d", dw_dtype);
  if (dX) GIFT_TRY(check_matrix("dX", dX, GIFT_DTYPE_BF16, rows, d, ld_dx));
  if (dW) GIFT_TRY(check_matrix("dW", dW, dw_dtype, vocab, d, ld_dw));
  if (dX && dX == dW) return fail(GIFT_ERR_INVALID_ARG, "dX and dW are the same buffer");
  if (accumulate && (!dW || dw_dtype != GIFT_DTYPE_F32)) return fail(GIFT_ERR_INVALID_ARG, "accumulate takes an fp32 dW");
  GIFT_TRY(check_ws(ws, ws_bytes, xent_backward_ws(rows, d, vocab, dX != nullptr, dW != nullptr, dw_dtype)));
  XeGrad g{};
  g.dX = dX;
  g.ld_dx = ld_dx;
  g.dW = dW;
  g.dw_dtype = dw_dtype;
  g.ld_dw = ld_dw;
  g.accumulate = accumulate != 0;
  return launched(launch_xent_backward(matrix(X, rows, d, ldx), matrix(W, vocab, d, ldw), targets, lse, dloss, g, ws,
                                       (hipStream_t)stream));
}

}  // extern "C"
