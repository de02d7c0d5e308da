// Entry points of a layer's training step in MXFP4 and of the norm
// (gift_mx_*, gift_norm_* of include/gift.h): argument validation, then the
// launchers of mx.hip and norm.hip.
#include "checks.hpp"
#include "mx.hpp"

using namespace gift;

namespace {

int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m; }

// padded elements of an operand
bool mx_size_ok(int64_t rows, int64_t k) {
  return size_ok(rows, k) && up(rows, kMxRows) * up(k, kMxStep) <= kMaxElems / (kMxRows * kMxStep);
}

gift_status check_mx(const char* name, const gift_mx* m) {
  if (!m) return fail(GIFT_ERR_INVALID_ARG, "%s is NULL", name);
  if (!mx_size_ok(m->rows, m->k))
    return fail(GIFT_ERR_UNSUPPORTED_SHAPE, "%s: %lld x %lld out of range", name, (long long)m->rows,
                (long long)m->k);
  if (!m->data || !aligned16(m->data))
    return fail(GIFT_ERR_INVALID_ARG, "%s: data is NULL or not 16-byte aligned", name);
  return GIFT_OK;
}

// Workspace of gift_mx_linear: X's operand, then the product's.
size_t linear_ws(int64_t rows, int64_t n, int64_t k) {
  if (mx_linear_cols(rows, n, k)) return 0;
  return align_up(gift_mx_bytes(rows, k)) + mx_matmul_ws(rows, n, k);
}

}  // namespace

extern "C" {

size_t gift_mx_bytes(int64_t rows, int64_t k) {
  if (!mx_size_ok(rows, k)) return 0;
  return (size_t)up(rows, kMxRows) * (size_t)up(k, kMxStep) * kMxPanel;
}

gift_status gift_mx_quantize(const void* X, int x_dtype, int64_t rows, int64_t cols, int64_t ld,
                             const gift_mx* by_row, const gift_mx* by_col, uint32_t* dev_flags,
                             void* stream) {
  GIFT_TRY(check_matrix("X", X, x_dtype, rows, cols, ld));
  if (!by_row && !by_col) return fail(GIFT_ERR_INVALID_ARG, "by_row and by_col are both NULL");
  if (by_row) {
    GIFT_TRY(check_mx("by_row", by_row));
    if (by_row->rows != rows || by_row->k != cols)
      return fail(GIFT_ERR_INVALID_ARG, "by_row is %lld x %lld, X %lld x %lld", (long long)by_row->rows,
                  (long long)by_row->k, (long long)rows, (long long)cols);
  }
  if (by_col) {
    GIFT_TRY(check_mx("by_col", by_col));
    if (by_col->rows != cols || by_col->k != rows)
      return fail(GIFT_ERR_INVALID_ARG, "by_col is %lld x %lld, the transposed X %lld x %lld",
                  (long long)by_col->rows, (long long)by_col->k, (long long)cols, (long long)rows);
  }
  if (by_row && by_col && by_row->data == by_col->data)
    return fail(GIFT_ERR_INVALID_ARG, "by_row and by_col are the same buffer");
  GIFT_TRY(check_flags(dev_flags));
  return launched(launch_mx_quantize(X, x_dtype, rows, cols, ld,
                                     by_row ? static_cast<uint8_t*>(by_row->data) : nullptr,
                                     by_col ? static_cast<uint8_t*>(by_col->data) : nullptr, dev_flags,
                                     (hipStream_t)stream));
}

gift_status gift_mx_dequantize(const gift_mx* a, void* out, int out_dtype, int64_t ld, void* stream) {
  GIFT_TRY(check_mx("operand", a));
  GIFT_TRY(check_matrix("out", out, out_dtype, a->rows, a->k, ld));
  return launched(launch_mx_dequantize(static_cast<const uint8_t*>(a->data), a->rows, a->k, out,
                                       out_dtype, ld, (hipStream_t)stream));
}

size_t gift_mx_matmul_workspace_bytes(int64_t M, int64_t N, int64_t k) {
  if (!mx_size_ok(M, k) || !mx_size_ok(N, k) || !size_ok(M, N)) return 0;
  return mx_matmul_ws(M, N, k);
}

gift_status gift_mx_matmul(const gift_mx* A, const gift_mx* B, const float* bias, void* C, int c_dtype,
                           int64_t ldc, int accumulate, void* ws, size_t ws_bytes, void* stream) {
  GIFT_TRY(check_mx("A", A));
  GIFT_TRY(check_mx("B", B));
  if (A->k != B->k)
    return fail(GIFT_ERR_INVALID_ARG, "A sums over k = %lld, B over %lld", (long long)A->k,
                (long long)B->k);
  GIFT_TRY(check_matrix("C", C, c_dtype, A->rows, B->rows, ldc));
  GIFT_TRY(check_vec("bias", bias));
  if (accumulate && (c_dtype != GIFT_DTYPE_F32 || bias))
    return fail(GIFT_ERR_INVALID_ARG, "accumulate takes an fp32 C and no bias");
  GIFT_TRY(check_ws(ws, ws_bytes, mx_matmul_ws(A->rows, B->rows, A->k)));
  return launched(launch_mx_matmul(static_cast<const uint8_t*>(A->data),
                                   static_cast<const uint8_t*>(B->data), A->rows, B->rows, A->k, bias,
                                   C, c_dtype, ldc, accumulate != 0, ws, (hipStream_t)stream));
}

size_t gift_mx_linear_workspace_bytes(int64_t rows, int64_t n, int64_t k) {
  if (!mx_size_ok(rows, k) || !mx_size_ok(n, k) || !size_ok(rows, n)) return 0;
  return linear_ws(rows, n, k);
}

gift_status gift_mx_linear(const void* X, int x_dtype, int64_t rows, int64_t ldx, const gift_mx* W,
                           const float* bias, void* Y, int y_dtype, int64_t ldy, uint32_t* dev_flags,
                           void* ws, size_t ws_bytes, void* stream) {
  GIFT_TRY(check_mx("W", W));
  GIFT_TRY(check_matrix("X", X, x_dtype, rows, W->k, ldx));
  if (!mx_size_ok(rows, W->k))
    return fail(GIFT_ERR_UNSUPPORTED_SHAPE, "X: %lld x %lld out of range", (long long)rows,
                (long long)W->k);
  GIFT_TRY(check_matrix("Y", Y, y_dtype, rows, W->rows, ldy));
  GIFT_TRY(check_vec("bias", bias));
  GIFT_TRY(check_flags(dev_flags));
  GIFT_TRY(check_ws(ws, ws_bytes, linear_ws(rows, W->rows, W->k)));
  hipStream_t st = (hipStream_t)stream;
  const uint8_t* w = static_cast<const uint8_t*>(W->data);
  if (mx_linear_cols(rows, W->rows, W->k))
    return launched(launch_mx_linear_few(X, x_dtype, rows, ldx, w, W->rows, W->k, bias, Y, y_dtype, ldy,
                                         dev_flags, st));
  uint8_t* q = static_cast<uint8_t*>(ws);
  GIFT_TRY(launched(launch_mx_quantize(X, x_dtype, rows, W->k, ldx, q, nullptr, dev_flags, st)));
  return launched(launch_mx_matmul(q, w, rows, W->rows, W->k, bias, Y, y_dtype, ldy, false,
                                   q + align_up(gift_mx_bytes(rows, W->k)), st));
}

gift_status gift_norm_forward(const void* X, int x_dtype, int64_t rows, int64_t d, int kind,
                              const float* weight, const float* bias, float eps, void* Y, float* mean,
                              float* rstd, void* stream) {
  GIFT_TRY(check_matrix("X", X, x_dtype, rows, d, d));
  GIFT_TRY(check_matrix("Y", Y, x_dtype, rows, d, d));
  if (kind != GIFT_NORM_LAYER && kind != GIFT_NORM_RMS)
    return fail(GIFT_ERR_INVALID_ARG, "unknown norm kind %d", kind);
  if (!(eps >= 0.f && eps < 1e30f)) return fail(GIFT_ERR_INVALID_ARG, "eps must be finite and >= 0");
  GIFT_TRY(check_vec("weight", weight));
  GIFT_TRY(check_vec("bias", bias));
  GIFT_TRY(check_vec("mean", mean));
  GIFT_TRY(check_vec("rstd", rstd));
  if (mean && mean == rstd) return fail(GIFT_ERR_INVALID_ARG, "mean and rstd are the same buffer");
  return launched(launch_norm_forward(X, x_dtype, rows, d, kind, weight, bias, eps, Y, mean, rstd,
                                      (hipStream_t)stream));
}

size_t gift_norm_backward_workspace_bytes(int64_t rows, int64_t d) {
  return size_ok(rows, d) ? norm_backward_ws(rows, d) : 0;
}

gift_status gift_norm_backward(const void* dY, const void* X, int x_dtype, int64_t rows, int64_t d,
                               int kind, const float* weight, const float* mean, const float* rstd,
                               void* dX, float* dweight, float* dbias, int accumulate, void* ws,
                               size_t ws_bytes, void* stream) {
  GIFT_TRY(check_matrix("X", X, x_dtype, rows, d, d));
  GIFT_TRY(check_matrix("dY", dY, x_dtype, rows, d, d));
  if (dX) GIFT_TRY(check_matrix("dX", dX, x_dtype, rows, d, d));
  if (kind != GIFT_NORM_LAYER && kind != GIFT_NORM_RMS)
    return fail(GIFT_ERR_INVALID_ARG, "unknown norm kind %d", kind);
  if (!dX && !dweight && !dbias) return fail(GIFT_ERR_INVALID_ARG, "dX, dweight and dbias are all NULL");
  if (!rstd || (kind == GIFT_NORM_LAYER && !mean))
    return fail(GIFT_ERR_INVALID_ARG, "the forward pass's statistics are NULL");
  GIFT_TRY(check_vec("weight", weight));
  GIFT_TRY(check_vec("mean", mean));
  GIFT_TRY(check_vec("rstd", rstd));
  GIFT_TRY(check_vec("dweight", dweight));
  GIFT_TRY(check_vec("dbias", dbias));
  if (dweight && dweight == dbias)
    return fail(GIFT_ERR_INVALID_ARG, "dweight and dbias are the same buffer");
  GIFT_TRY(check_ws(ws, ws_bytes, dweight || dbias ? norm_backward_ws(rows, d) : 0));
  return launched(launch_norm_backward(dY, X, x_dtype, rows, d, kind, weight, mean, rstd, dX, dweight,
                                       dbias, accumulate != 0, ws, (hipStream_t)stream));
}

}  // extern "C"
