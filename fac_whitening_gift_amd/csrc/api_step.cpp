// Entry points of a training step around its layers (gift_xent_*,
// gift_block_norm_*, gift_grad_* of include/gift.h): argument validation, then
// the launchers of xent.hip, block_norm.hip and grad_clip.hip.
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

bool block_norm_size_ok(int64_t rows, int64_t d) { return size_ok(rows, d) && d <= kBlockNormMaxD; }

int64_t gates_of(const gift_block_norm& p) { return p.gate ? (p.rows + p.gate_rows - 1) / p.gate_rows : 1; }

gift_status check_block_norm(const gift_block_norm* p) {
  if (!p) return fail(GIFT_ERR_INVALID_ARG, "the block norm is NULL");
  if (!block_norm_size_ok(p->rows, p->d))
    return fail(GIFT_ERR_UNSUPPORTED_SHAPE, "%lld x %lld out of range", (long long)p->rows, (long long)p->d);
  if (p->kind != GIFT_NORM_LAYER && p->kind != GIFT_NORM_RMS)
    return fail(GIFT_ERR_INVALID_ARG, "unknown norm kind %d", p->kind);
  if (!dtype_ok(p->y_dtype) || !dtype_ok(p->h_dtype) ||
      (p->y_dtype == GIFT_DTYPE_F32 && p->h_dtype == GIFT_DTYPE_BF16))
    return fail(GIFT_ERR_INVALID_ARG, "dtypes %d beside a stream of %d", p->y_dtype, p->h_dtype);
  if (!(p->eps >= 0.f && p->eps < 1e30f)) return fail(GIFT_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (!(p->scale > -1e30f && p->scale < 1e30f)) return fail(GIFT_ERR_INVALID_ARG, "scale must be finite");
  if (p->gate && (p->gate_rows < 1 || p->gate_rows > p->rows))
    return fail(GIFT_ERR_UNSUPPORTED_SHAPE, "gate rows of %lld for %lld rows", (long long)p->gate_rows,
                (long long)p->rows);
  if (!p->post && (p->post_weight || p->post_bias))
    return fail(GIFT_ERR_INVALID_ARG, "post_weight and post_bias belong to the norm of y");
  GIFT_TRY(check_vec("weight", p->weight));
  GIFT_TRY(check_vec("bias", p->bias));
  GIFT_TRY(check_vec("post_weight", p->post_weight));
  GIFT_TRY(check_vec("post_bias", p->post_bias));
  return check_vec("gate", p->gate);
}

gift_status check_tensors(const char* name, const gift_tensor* t, int n) {
  if (!t) return fail(GIFT_ERR_INVALID_ARG, "%s is NULL", name);
  if (n < 1 || n > kGradMaxTensors) return fail(GIFT_ERR_UNSUPPORTED_SHAPE, "%d tensors", n);
  for (int i = 0; i < n; ++i) {
    if (!dtype_ok(t[i].dtype)) return fail(GIFT_ERR_INVALID_ARG, "%s %d: unknown dtype %d", name, i, t[i].dtype);
    if (t[i].n < 0 || t[i].n > (int64_t(1) << 45) / (int64_t)dtype_size(t[i].dtype))
      return fail(GIFT_ERR_UNSUPPORTED_SHAPE, "%s %d: %lld elements", name, i, (long long)t[i].n);
    if (t[i].n && (!t[i].data || !aligned_to(t[i].data, dtype_size(t[i].dtype))))
      return fail(GIFT_ERR_INVALID_ARG, "%s %d is NULL or not aligned to its elements", name, i);
  }
  if (!grad_size_ok(t, n)) return fail(GIFT_ERR_UNSUPPORTED_SHAPE, "%s: more than 2^45 bytes", name);
  return GIFT_OK;
}

gift_status check_sum(const double* p) {
  return aligned_to(p, 8) ? GIFT_OK : fail(GIFT_ERR_INVALID_ARG, "sumsq must be 8-byte aligned");
}

// two of the gradients in one buffer
bool any_alike(const gift_block_norm_grads& g) {
  const float* const v[5] = {g.dweight, g.dbias, g.dpost_weight, g.dpost_bias, g.dgate};
  for (int i = 0; i < 5; ++i)
    for (int j = i + 1; j < 5; ++j)
      if (v[i] && v[i] == v[j]) return true;
  return false;
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

gift_status gift_block_norm_forward(const gift_block_norm* p, const void* Y, const void* H, void* H_out, void* X,
                                    float* stats, void* stream) {
  GIFT_TRY(check_block_norm(p));
  GIFT_TRY(check_matrix("Y", Y, p->y_dtype, p->rows, p->d, p->d));
  GIFT_TRY(check_matrix("H", H, p->h_dtype, p->rows, p->d, p->d));
  GIFT_TRY(check_matrix("H_out", H_out, p->h_dtype, p->rows, p->d, p->d));
  GIFT_TRY(check_matrix("X", X, p->y_dtype, p->rows, p->d, p->d));
  if (X == H_out) return fail(GIFT_ERR_INVALID_ARG, "X and H_out are the same buffer");
  if (!stats) return fail(GIFT_ERR_INVALID_ARG, "stats is NULL");
  GIFT_TRY(check_vec("stats", stats));
  return launched(launch_block_norm_forward(*p, Y, H, H_out, X, stats, (hipStream_t)stream));
}

size_t gift_block_norm_backward_workspace_bytes(int64_t rows, int64_t d, int64_t gates) {
  return block_norm_size_ok(rows, d) && gates >= 1 && gates <= rows ? block_norm_backward_ws(rows, d, gates) : 0;
}

gift_status gift_block_norm_backward(const gift_block_norm* p, const void* dX, const void* dH_out, const void* Y,
                                     const void* H_out, const float* stats, void* dY, void* dH,
                                     const gift_block_norm_grads* grads, int accumulate, void* ws, size_t ws_bytes,
                                     void* stream) {
  GIFT_TRY(check_block_norm(p));
  GIFT_TRY(check_matrix("dX", dX, p->y_dtype, p->rows, p->d, p->d));
  if (dH_out) GIFT_TRY(check_matrix("dH_out", dH_out, p->h_dtype, p->rows, p->d, p->d));
  GIFT_TRY(check_matrix("Y", Y, p->y_dtype, p->rows, p->d, p->d));
  GIFT_TRY(check_matrix("H_out", H_out, p->h_dtype, p->rows, p->d, p->d));
  if (dY) GIFT_TRY(check_matrix("dY", dY, p->y_dtype, p->rows, p->d, p->d));
  if (dH) GIFT_TRY(check_matrix("dH", dH, p->h_dtype, p->rows, p->d, p->d));
  if (dY && dY == dH) return fail(GIFT_ERR_INVALID_ARG, "dY and dH are the same buffer");
  if (!stats) return fail(GIFT_ERR_INVALID_ARG, "the forward pass's statistics are NULL");
  GIFT_TRY(check_vec("stats", stats));
  const gift_block_norm_grads g = grads ? *grads : gift_block_norm_grads{};
  const bool vectors = g.dweight || g.dbias || g.dpost_weight || g.dpost_bias || g.dgate;
  if (!dY && !dH && !vectors) return fail(GIFT_ERR_INVALID_ARG, "every gradient is NULL");
  if (!p->post && (g.dpost_weight || g.dpost_bias))
    return fail(GIFT_ERR_INVALID_ARG, "dpost_weight and dpost_bias belong to the norm of y");
  if (!p->gate && g.dgate) return fail(GIFT_ERR_INVALID_ARG, "dgate without a gate");
  if (any_alike(g)) return fail(GIFT_ERR_INVALID_ARG, "two of the vectors' gradients are the same buffer");
  GIFT_TRY(check_vec("dweight", g.dweight));
  GIFT_TRY(check_vec("dbias", g.dbias));
  GIFT_TRY(check_vec("dpost_weight", g.dpost_weight));
  GIFT_TRY(check_vec("dpost_bias", g.dpost_bias));
  GIFT_TRY(check_vec("dgate", g.dgate));
  GIFT_TRY(check_ws(ws, ws_bytes, vectors ? block_norm_backward_ws(p->rows, p->d, gates_of(*p)) : 0));
  return launched(launch_block_norm_backward(*p, dX, dH_out, Y, H_out, stats, dY, dH, g, accumulate != 0, ws,
                                             (hipStream_t)stream));
}

size_t gift_grad_workspace_bytes(int n) { return n < 1 || n > kGradMaxTensors ? 0 : grad_ws(n); }

gift_status gift_grad_norm(const gift_tensor* tensors, int n, double* sumsq, float* norm, uint32_t* dev_flags, void* ws,
                           size_t ws_bytes, void* stream) {
  GIFT_TRY(check_tensors("tensor", tensors, n));
  if (!sumsq && !norm) return fail(GIFT_ERR_INVALID_ARG, "sumsq and norm are both NULL");
  GIFT_TRY(check_sum(sumsq));
  GIFT_TRY(check_vec("norm", norm));
  GIFT_TRY(check_flags(dev_flags));
  GIFT_TRY(check_ws(ws, ws_bytes, grad_ws(n)));
  return launched(launch_grad(tensors, nullptr, n, nullptr, false, 0.f, 0.f, sumsq, norm, dev_flags, ws,
                              (hipStream_t)stream));
}

gift_status gift_grad_clip(const gift_tensor* tensors, const gift_tensor* out, int n, const double* sumsq, float max_norm,
                           float eps, float* norm, uint32_t* dev_flags, void* ws, size_t ws_bytes, void* stream) {
  GIFT_TRY(check_tensors("tensor", tensors, n));
  if (out) {
    GIFT_TRY(check_tensors("out", out, n));
    for (int i = 0; i < n; ++i)
      if (out[i].n != tensors[i].n || out[i].dtype != tensors[i].dtype)
        return fail(GIFT_ERR_INVALID_ARG, "out %d has another size or type than its tensor", i);
  }
  GIFT_TRY(check_sum(sumsq));
  if (!(max_norm >= 0.f && max_norm < __builtin_inff())) return fail(GIFT_ERR_INVALID_ARG, "max_norm must be finite and >= 0");
  if (!(eps >= 0.f && eps < 1e30f)) return fail(GIFT_ERR_INVALID_ARG, "eps must be finite and >= 0");
  GIFT_TRY(check_vec("norm", norm));
  GIFT_TRY(check_flags(dev_flags));
  GIFT_TRY(check_ws(ws, ws_bytes, grad_ws(n)));
  return launched(launch_grad(tensors, out, n, sumsq, true, max_norm, eps, nullptr, norm, dev_flags, ws,
                              (hipStream_t)stream));
}

}  // extern "C"
