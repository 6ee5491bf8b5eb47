// Root-mean-square norm over the rows of a matrix, with the residual's
// addition and an output in 8 bits, and its backward pass, on gfx950.
//
// Forward, for a row x of n values of type T:
//   h_i = x_i + residual_i        rounded to the residual's type S (T or
//                                 float32) and written; x_i without residual
//   rstd = 1 / sqrt(sum(h_i^2) / n + eps)
//   y_i = (h_i * rstd) * w_i      float32, rounded once to T
// or, in 8 bits, for each block of 128 values of the row (or the whole row):
//   scale = max(max|y_i| / M, 2^-126), M the type's largest value,
//   q_i = y_i * (1 / scale)       rounded once to the type
// The squares are summed in double, where the square of a float32 is exact:
// the sum neither overflows nor underflows for any finite row, and is good to
// 2^-52 log2(n), so rstd is the float32 next to the true one.
//
// Backward, with h and the rstd the forward pass wrote, g_i = dy_i * w_i:
//   xhat_i = h_i * rstd
//   dh_i = rstd * (g_i - xhat_i * c) + dsum_i,  c = sum(g xhat) / n,
// dsum the gradient of the written h (0 without one); dh is the gradient of x
// and of the residual alike, and
//   dw_j = sum over rows of dy * xhat.
//
// Every sum has one fixed order given by the shape and the types, so results
// are the same bits from run to run, and a row's y and dh do not depend on
// the other rows.
#include "sv_rms_rows.hpp"

using svh::check_device;
using svh::check_launch;
using svh::ok;

extern "C" {

sv_status sv_rms_norm(const void *x, int64_t ldx, const void *residual, int64_t ldr, int dtype, int sum_dtype,
                      int64_t rows, int64_t n, const void *weight, int param_dtype, double eps, void *y, int64_t ldy,
                      void *sum, int64_t ldsum, float *rstd, void *stream) {
  static const char who[] = "sv_rms_norm";
  sv_status st = svm::check_forward(who, x, ldx, residual, ldr, dtype, sum_dtype, rows, n, weight, param_dtype, eps,
                                    sum, ldsum);
  if (st != SV_OK) return st;
  if ((st = svr::check_matrix(who, "y", y, ldy, rows, n, svr::dtype_bytes(dtype))) != SV_OK) return st;
  if ((st = svr::check_stats(who, "rstd", rstd, rows)) != SV_OK) return st;
  if (rows == 0 || (n == 0 && !rstd)) return ok();
  if ((st = check_device()) != SV_OK) return st;
  (void)hipGetLastError();
  forward<false>(x, ldx, residual, ldr, dtype, sum_dtype, Rows{rows, (int)n, weight, param_dtype, eps, rstd}, y, ldy,
                 sum, ldsum, Out8{}, reinterpret_cast<hipStream_t>(stream));
  return check_launch(who);
}

}  // extern "C"
