// Root-mean-square norm with its output in 8 bits (the formulas and kernels of
// sv_rms.hip and sv_rms_rows.hpp).
#include "sv_rms_rows.hpp"

using svh::check_device;
using svh::check_launch;
using svh::fail;
using svh::ok;

extern "C" {

sv_status sv_rms_norm_fp8(const void *x, int64_t ldx, const void *residual, int64_t ldr, int dtype, int sum_dtype,
                          int64_t rows, int64_t n, const void *weight, int param_dtype, double eps, int out_dtype,
                          int64_t block, void *q, int64_t ldq, float *scale, void *sum, int64_t ldsum, float *rstd,
                          void *stream) {
  static const char who[] = "sv_rms_norm_fp8";
  sv_status st = svm::check_forward(who, x, ldx, residual, ldr, dtype, sum_dtype, rows, n, weight, param_dtype, eps,
                                    sum, ldsum);
  if (st != SV_OK) return st;
  if (out_dtype != SV_DTYPE_E4M3 && out_dtype != SV_DTYPE_E5M2)
    return fail(SV_ERR_INVALID_ARGUMENT, "%s: out_dtype %d must be SV_DTYPE_E4M3 or SV_DTYPE_E5M2", who, out_dtype);
  if (block != 0 && block != BLOCK)
    return fail(SV_ERR_INVALID_ARGUMENT, "%s: block = %lld must be %d, or 0 for whole rows", who, (long long)block,
                BLOCK);
  if ((st = svr::check_matrix(who, "q", q, ldq, rows, n, 1)) != SV_OK) return st;
  if ((st = svr::check_stats(who, "rstd", rstd, rows)) != SV_OK) return st;
  if (rows > 0 && (n > 0 || block == 0)) {
    if (!scale) return fail(SV_ERR_INVALID_ARGUMENT, "%s: scale is NULL", who);
    if (reinterpret_cast<uintptr_t>(scale) % sizeof(float))
      return fail(SV_ERR_INVALID_ARGUMENT, "%s: scale is not aligned to its type", who);
  }
  if (rows == 0 || (n == 0 && block != 0 && !rstd)) return ok();
  if ((st = check_device()) != SV_OK) return st;
  (void)hipGetLastError();
  forward<true>(x, ldx, residual, ldr, dtype, sum_dtype, Rows{rows, (int)n, weight, param_dtype, eps, rstd}, nullptr, 0,
                sum, ldsum, Out8{(uint8_t *)q, ldq, scale, block == 0, out_dtype == SV_DTYPE_E5M2},
                reinterpret_cast<hipStream_t>(stream));
  return check_launch(who);
}

}  // extern "C"
