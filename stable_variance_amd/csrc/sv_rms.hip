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
#include "sv_rms.hpp"

using svh::check_device;
using svh::check_launch;
using svh::fail;
using svh::ok;
using svr::Node;

namespace {

constexpr int ROW_THREADS = 512;
constexpr int64_t ROW_GRID = 8192;  // workgroups of a row launch, at most
constexpr int COL_ROWS = 64;        // rows of one partial column sum
constexpr int64_t COL_MAX_GROUPS = 512;
constexpr int BLOCK = 128;          // values that share a scale

// What a call passes on about its rows.
struct Rows {
  int64_t rows;
  int n;
  const void *w;
  int pt;
  double eps;
  float *rstd;
};

// The 8-bit output.
struct Out8 {
  uint8_t *q;
  int64_t ldq;
  float *scale;  // one for each block of 128 values, or (per_row) for each row
  bool per_row, e5m2;
};

// Rows of any length: a workgroup per row, each pass reads the row again (from
// the cache where it fits).
template <class T, class S, bool RES, bool Q>
__global__ __launch_bounds__(ROW_THREADS) void k_rms_any(const T *x, int64_t ldx, const S *res, int64_t ldr, Rows a,
                                                         T *y, int64_t ldy, S *h, int64_t ldh, Out8 o) {
  constexpr int VE = 16 / (sizeof(T) > sizeof(S) ? sizeof(T) : sizeof(S)), STEP = ROW_THREADS * VE;
  constexpr int LANES = BLOCK / VE;  // lanes that hold a block
  __shared__ double lds_sum[ROW_THREADS / 64];
  __shared__ unsigned lds_max[ROW_THREADS / 64];
  const int n = a.n, e0 = threadIdx.x * VE;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T *xr = x + r * ldx;
    double s = 0.0;
    for (int64_t e = e0; e < n; e += STEP) {
      const int count = (int)(n - e < VE ? n - e : VE);
      float f[VE];
      svm::get<T, VE>(xr + e, count, f);
      if constexpr (RES) {
        float g[VE];
        svm::get<S, VE>(res + r * ldr + e, count, g);
#pragma unroll
        for (int i = 0; i < VE; ++i) f[i] = svr::to_f(svr::from_f<S>(f[i] + g[i]));
        svm::put<S, VE>(h + r * ldh + e, count, f);
      }
      s += svr::pair_sum<0, VE>([&](int i) { return svm::square(f[i]); });
    }
    __syncthreads();  // the row before has read the sums
    const float rs = svr::rstd_of(svm::group_add<ROW_THREADS>(s, lds_sum) / (double)n + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[r] = rs;
    // the values of y in the chunk at e (a thread reads back what it wrote)
    const auto values = [&](int64_t e, int count, float(&f)[VE]) {
      float w[VE];
      if constexpr (RES) svm::get<S, VE>(h + r * ldh + e, count, f);
      else svm::get<T, VE>(xr + e, count, f);
      svm::get_weight<VE>(a.w, a.pt, e, count, w);
#pragma unroll
      for (int i = 0; i < VE; ++i) f[i] = (f[i] * rs) * w[i];
    };
    if constexpr (!Q) {
      for (int64_t e = e0; e < n; e += STEP) {
        const int count = (int)(n - e < VE ? n - e : VE);
        float f[VE];
        values(e, count, f);
        svm::put<T, VE>(y + r * ldy + e, count, f);
      }
    } else {
      const auto largest = [&](const float(&f)[VE]) {
        unsigned m = 0;
#pragma unroll
        for (int i = 0; i < VE; ++i) m = svm::umax(m, svm::abs_bits(f[i]));
        return m;
      };
      float inv = 0.0f;
      if (o.per_row) {
        unsigned m = 0;
        for (int64_t e = e0; e < n; e += STEP) {
          const int count = (int)(n - e < VE ? n - e : VE);
          float f[VE];
          values(e, count, f);
          m = svm::umax(m, largest(f));
        }
        const float scale = svm::fp8_scale(svm::group_max<ROW_THREADS>(m, lds_max), o.e5m2);
        if (threadIdx.x == 0) o.scale[r] = scale;
        inv = 1.0f / scale;
      }
      const int64_t blocks = (n + (int64_t)BLOCK - 1) / BLOCK;
      for (int64_t base = 0; base < n; base += STEP) {  // all threads, for the maxima across lanes
        const int64_t e = base + e0;
        const int count = e >= n ? 0 : (int)(n - e < VE ? n - e : VE);
        float f[VE];
        if (count) values(e, count, f);
        else
#pragma unroll
          for (int i = 0; i < VE; ++i) f[i] = 0.0f;
        if (!o.per_row) {
          const float scale = svm::fp8_scale(svm::seg_max<LANES>(largest(f)), o.e5m2);
          if (count && threadIdx.x % LANES == 0) o.scale[r * blocks + e / BLOCK] = scale;
          inv = 1.0f / scale;
        }
        if (count) svm::put_fp8<VE>(o.q + r * o.ldq + e, count, f, inv, o.e5m2);
      }
    }
    __syncthreads();  // the maxima are read
  }
}

// The rows' part of the backward pass for rows of any length.
template <class T, class S>
__global__ __launch_bounds__(ROW_THREADS) void k_rms_dh_any(const T *dy, int64_t lddy, const S *h, int64_t ldh,
                                                            const S *dsum, int64_t ldds, Rows a, S *dh, int64_t lddh,
                                                            T *dx, int64_t lddx) {
  constexpr int VE = 16 / (sizeof(T) > sizeof(S) ? sizeof(T) : sizeof(S)), STEP = ROW_THREADS * VE;
  __shared__ double lds[ROW_THREADS / 64];
  const int n = a.n, e0 = threadIdx.x * VE;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const float rs = a.rstd[r];
    // xhat and g of the chunk at e
    const auto values = [&](int64_t e, int count, float(&xh)[VE], float(&g)[VE]) {
      float w[VE];
      svm::get<S, VE>(h + r * ldh + e, count, xh);
      svm::get<T, VE>(dy + r * lddy + e, count, g);
      svm::get_weight<VE>(a.w, a.pt, e, count, w);
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        xh[i] = xh[i] * rs;
        g[i] = g[i] * w[i];
      }
    };
    double s = 0.0;
    for (int64_t e = e0; e < n; e += STEP) {
      const int count = (int)(n - e < VE ? n - e : VE);
      float xh[VE], g[VE];
      values(e, count, xh, g);
      s += (double)svr::pair_sum<0, VE>([&](int i) { return i < count ? g[i] * xh[i] : 0.0f; });
    }
    __syncthreads();
    const float c = (float)(svm::group_add<ROW_THREADS>(s, lds) / (double)n);
    for (int64_t e = e0; e < n; e += STEP) {
      const int count = (int)(n - e < VE ? n - e : VE);
      float xh[VE], g[VE];
      values(e, count, xh, g);
#pragma unroll
      for (int i = 0; i < VE; ++i) g[i] = rs * (g[i] - xh[i] * c);
      if (dsum) {
        float d[VE];
        svm::get<S, VE>(dsum + r * ldds + e, count, d);
#pragma unroll
        for (int i = 0; i < VE; ++i) g[i] = g[i] + d[i];
      }
      if (dh) svm::put<S, VE>(dh + r * lddh + e, count, g);
      if (dx) svm::put<T, VE>(dx + r * lddx + e, count, g);
    }
  }
}

// The columns' part for rows of any length: group q of the rows (row r belongs
// to group r mod groups) and 64 chunks of columns per workgroup; each wave
// takes every fourth row of the group.  part is [groups][n].
constexpr int COL_WAVES = 4;
template <class T, class S>
__global__ __launch_bounds__(64 * COL_WAVES) void k_rms_dw_any(const T *dy, int64_t lddy, const S *h, int64_t ldh,
                                                               Rows a, int groups, int ctiles, Node *part) {
  constexpr int VE = 16 / (sizeof(T) > sizeof(S) ? sizeof(T) : sizeof(S));
  __shared__ Node lds[COL_WAVES][64][VE];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = a.n;
  const int q = blockIdx.x / ctiles;
  const int64_t j = ((int64_t)(blockIdx.x % ctiles) * 64 + lane) * VE;
  const int count = j >= n ? 0 : (int)(n - j < VE ? n - j : VE);
  Node dw[VE];
#pragma unroll
  for (int i = 0; i < VE; ++i) dw[i] = sv::zero_node();
  if (count) {
    for (int64_t r = q + (int64_t)wave * groups; r < a.rows; r += COL_WAVES * (int64_t)groups) {
      const float rs = a.rstd[r];
      float g[VE], x[VE];
      svm::get<T, VE>(dy + r * lddy + j, count, g);
      svm::get<S, VE>(h + r * ldh + j, count, x);
#pragma unroll
      for (int i = 0; i < VE; ++i) svr::add_to(dw[i], g[i] * (x[i] * rs));
    }
  }
#pragma unroll
  for (int i = 0; i < VE; ++i) lds[wave][lane][i] = dw[i];
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      Node t[COL_WAVES];
#pragma unroll
      for (int v = 0; v < COL_WAVES; ++v) t[v] = lds[v][lane][i];
      if (i < count) part[(int64_t)q * n + j + i] = sv::node_tree<0, COL_WAVES, COL_WAVES>(t);
    }
  }
}

// Joins the partial sums part[groups][n] of 64 columns: wave i adds up groups
// i, i + 16, .. in order, then the waves are joined pairwise.  The launch
// starts at block b0.
constexpr int JOIN_WAVES = 16;
__global__ __launch_bounds__(64 * JOIN_WAVES) void k_rms_join(const Node *part, int groups, int n, int b0, void *dw,
                                                              int pt) {
  __shared__ Node lds[JOIN_WAVES][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t j = ((int64_t)b0 + blockIdx.x) * 64 + lane;
  Node s = sv::zero_node();
  if (j < n) {
#pragma unroll 8
    for (int q = wave; q < groups; q += JOIN_WAVES) s = sv::combine(s, part[(int64_t)q * n + j]);
  }
  lds[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && j < n) {
    Node t[JOIN_WAVES];
#pragma unroll
    for (int i = 0; i < JOIN_WAVES; ++i) t[i] = lds[i][lane];
    svr::store_as(dw, j, pt, sv::root_value(sv::node_tree<0, JOIN_WAVES, JOIN_WAVES>(t)));
  }
}

// Workgroups of k_rms_dw_any across a row.
int64_t col_tiles(int dtype, int sum_dtype, int64_t n) {
  const int64_t widest = dtype == SV_DTYPE_F32 || sum_dtype == SV_DTYPE_F32 ? 4 : 2, values = 64 * (16 / widest);
  return (n + values - 1) / values;
}

// Groups of rows: 64 rows each or more, at most 512 and at most 2^22
// workgroups in all (2^30 work-items, within HIP's grid limit).
int64_t col_groups(int dtype, int sum_dtype, int64_t rows, int64_t n) {
  const int64_t ctiles = col_tiles(dtype, sum_dtype, n);
  int64_t g = (rows + COL_ROWS - 1) / COL_ROWS;
  if (g > COL_MAX_GROUPS) g = COL_MAX_GROUPS;
  if (g > ((int64_t)1 << 22) / ctiles) g = ((int64_t)1 << 22) / ctiles;
  return g < 1 ? 1 : g;
}

// Checks that the calls share; SV_OK without touching the message.
sv_status check_rows(const char *who, int dtype, int sum_dtype, int64_t rows, int64_t n, int param_dtype) {
  if (!svr::dtype_bytes(dtype)) return fail(SV_ERR_INVALID_ARGUMENT, "%s: dtype %d is not a type code", who, dtype);
  if (sum_dtype != dtype && sum_dtype != SV_DTYPE_F32)
    return fail(SV_ERR_INVALID_ARGUMENT, "%s: sum_dtype %d must be dtype or SV_DTYPE_F32", who, sum_dtype);
  if (param_dtype != dtype && param_dtype != SV_DTYPE_F32)
    return fail(SV_ERR_INVALID_ARGUMENT, "%s: param_dtype %d must be the rows' type or SV_DTYPE_F32", who,
                param_dtype);
  if (rows < 0 || n < 0)
    return fail(SV_ERR_INVALID_ARGUMENT, "%s: rows = %lld, n = %lld must be >= 0", who, (long long)rows,
                (long long)n);
  if (n > svr::MAX_N) return fail(SV_ERR_UNSUPPORTED, "%s: rows of %lld values exceed 2^27", who, (long long)n);
  if (n > 0 && rows > svr::MAX_VALUES / n)
    return fail(SV_ERR_UNSUPPORTED, "%s: %lld x %lld values exceed 2^36", who, (long long)rows, (long long)n);
  if (rows > svr::MAX_VALUES) return fail(SV_ERR_UNSUPPORTED, "%s: %lld rows exceed 2^36", who, (long long)rows);
  return SV_OK;
}

// Checks of the forward calls.
sv_status check_forward(const char *who, const void *x, int64_t ldx, const void *residual, int64_t ldr, int dtype,
                        int sum_dtype, int64_t rows, int64_t n, const void *weight, int param_dtype, double eps,
                        const void *sum, int64_t ldsum) {
  sv_status st = check_rows(who, dtype, sum_dtype, rows, n, param_dtype);
  if (st != SV_OK) return st;
  if (!(eps >= 0.0) || eps > 3.0e38) return fail(SV_ERR_INVALID_ARGUMENT, "%s: eps must be >= 0 and finite", who);
  const size_t e = svr::dtype_bytes(dtype), se = svr::dtype_bytes(sum_dtype);
  if ((st = svr::check_matrix(who, "x", x, ldx, rows, n, e)) != SV_OK) return st;
  if (residual || sum) {
    if ((st = svr::check_matrix(who, "residual", residual, ldr, rows, n, se)) != SV_OK) return st;
    if ((st = svr::check_matrix(who, "sum", sum, ldsum, rows, n, se)) != SV_OK) return st;
  } else if (sum_dtype != dtype) {
    return fail(SV_ERR_INVALID_ARGUMENT, "%s: sum_dtype %d without a residual must be dtype", who, sum_dtype);
  }
  if (weight && (st = svr::check_matrix(who, "weight", weight, n, 1, n, svr::dtype_bytes(param_dtype))) != SV_OK)
    return st;
  return SV_OK;
}

unsigned row_grid(int64_t rows) { return (unsigned)(rows < ROW_GRID ? rows : ROW_GRID); }

// The launch of a forward call: with (Q) the output in 8 bits.
template <bool Q>
void forward(const void *x, int64_t ldx, const void *residual, int64_t ldr, int dtype, int sum_dtype, const Rows &a,
             void *y, int64_t ldy, void *sum, int64_t ldsum, const Out8 &o, hipStream_t s) {
  svm::with_types(dtype, sum_dtype, [&](auto t, auto u) {
    using T = decltype(t);
    using S = decltype(u);
    if (residual)
      k_rms_any<T, S, true, Q><<<row_grid(a.rows), ROW_THREADS, 0, s>>>((const T *)x, ldx, (const S *)residual, ldr, a,
                                                                       (T *)y, ldy, (S *)sum, ldsum, o);
    else
      k_rms_any<T, T, false, Q><<<row_grid(a.rows), ROW_THREADS, 0, s>>>((const T *)x, ldx, nullptr, 0, a, (T *)y, ldy,
                                                                        nullptr, 0, o);
  });
}

}  // namespace

extern "C" {

sv_status sv_rms_norm(const void *x, int64_t ldx, const void *residual, int64_t ldr, int dtype, int sum_dtype,
                      int64_t rows, int64_t n, const void *weight, int param_dtype, double eps, void *y, int64_t ldy,
                      void *sum, int64_t ldsum, float *rstd, void *stream) {
  static const char who[] = "sv_rms_norm";
  sv_status st = check_forward(who, x, ldx, residual, ldr, dtype, sum_dtype, rows, n, weight, param_dtype, eps, sum,
                               ldsum);
  if (st != SV_OK) return st;
  if ((st = svr::check_matrix(who, "y", y, ldy, rows, n, svr::dtype_bytes(dtype))) != SV_OK) return st;
  if (rows == 0 || (n == 0 && !rstd)) return ok();
  if ((st = check_device()) != SV_OK) return st;
  (void)hipGetLastError();
  forward<false>(x, ldx, residual, ldr, dtype, sum_dtype, Rows{rows, (int)n, weight, param_dtype, eps, rstd}, y, ldy,
                 sum, ldsum, Out8{}, reinterpret_cast<hipStream_t>(stream));
  return check_launch(who);
}

sv_status sv_rms_norm_fp8(const void *x, int64_t ldx, const void *residual, int64_t ldr, int dtype, int sum_dtype,
                          int64_t rows, int64_t n, const void *weight, int param_dtype, double eps, int out_dtype,
                          int64_t block, void *q, int64_t ldq, float *scale, void *sum, int64_t ldsum, float *rstd,
                          void *stream) {
  static const char who[] = "sv_rms_norm_fp8";
  sv_status st = check_forward(who, x, ldx, residual, ldr, dtype, sum_dtype, rows, n, weight, param_dtype, eps, sum,
                               ldsum);
  if (st != SV_OK) return st;
  if (out_dtype != SV_DTYPE_E4M3 && out_dtype != SV_DTYPE_E5M2)
    return fail(SV_ERR_INVALID_ARGUMENT, "%s: out_dtype %d must be SV_DTYPE_E4M3 or SV_DTYPE_E5M2", who, out_dtype);
  if (block != 0 && block != BLOCK)
    return fail(SV_ERR_INVALID_ARGUMENT, "%s: block = %lld must be %d, or 0 for whole rows", who, (long long)block,
                BLOCK);
  if ((st = svr::check_matrix(who, "q", q, ldq, rows, n, 1)) != SV_OK) return st;
  if (rows > 0 && (n > 0 || block == 0)) {
    if (!scale) return fail(SV_ERR_INVALID_ARGUMENT, "%s: scale is NULL", who);
    if (reinterpret_cast<uintptr_t>(scale) % sizeof(float))
      return fail(SV_ERR_INVALID_ARGUMENT, "%s: scale is not aligned to its type", who);
  }
  if (rows == 0) return ok();
  if ((st = check_device()) != SV_OK) return st;
  (void)hipGetLastError();
  forward<true>(x, ldx, residual, ldr, dtype, sum_dtype, Rows{rows, (int)n, weight, param_dtype, eps, rstd}, nullptr, 0,
                sum, ldsum, Out8{(uint8_t *)q, ldq, scale, block == 0, out_dtype == SV_DTYPE_E5M2},
                reinterpret_cast<hipStream_t>(stream));
  return check_launch(who);
}

size_t sv_rms_norm_backward_workspace_size(int64_t rows, int64_t n, int dtype, int sum_dtype) {
  if (!svr::dtype_bytes(dtype) || (sum_dtype != dtype && sum_dtype != SV_DTYPE_F32) || rows < 0 || n < 0 ||
      n > svr::MAX_N || rows > svr::MAX_VALUES || (n > 0 && rows > svr::MAX_VALUES / n))
    return (size_t)-1;
  if (n == 0) return 0;
  return svr::round256((size_t)col_groups(dtype, sum_dtype, rows, n) * (size_t)n * sizeof(Node));
}

sv_status sv_rms_norm_backward(const void *dy, int64_t lddy, const void *h, int64_t ldh, const void *dsum,
                               int64_t lddsum, int dtype, int sum_dtype, int64_t rows, int64_t n, const void *weight,
                               int param_dtype, const float *rstd, void *dh, int64_t lddh, void *dx, int64_t lddx,
                               void *dweight, void *workspace, size_t workspace_bytes, void *stream) {
  static const char who[] = "sv_rms_norm_backward";
  sv_status st = check_rows(who, dtype, sum_dtype, rows, n, param_dtype);
  if (st != SV_OK) return st;
  const size_t e = svr::dtype_bytes(dtype), se = svr::dtype_bytes(sum_dtype), pe = svr::dtype_bytes(param_dtype);
  if ((st = svr::check_matrix(who, "dy", dy, lddy, rows, n, e)) != SV_OK) return st;
  if ((st = svr::check_matrix(who, "h", h, ldh, rows, n, se)) != SV_OK) return st;
  if (dsum && (st = svr::check_matrix(who, "dsum", dsum, lddsum, rows, n, se)) != SV_OK) return st;
  if (weight && (st = svr::check_matrix(who, "weight", weight, n, 1, n, pe)) != SV_OK) return st;
  if (dh && (st = svr::check_matrix(who, "dh", dh, lddh, rows, n, se)) != SV_OK) return st;
  if (dx && (st = svr::check_matrix(who, "dx", dx, lddx, rows, n, e)) != SV_OK) return st;
  if (dweight && (st = svr::check_matrix(who, "dweight", dweight, n, 1, n, pe)) != SV_OK) return st;
  if (rows > 0 && n > 0 && !rstd) return fail(SV_ERR_INVALID_ARGUMENT, "%s: rstd is NULL", who);
  if (n == 0 || (!dh && !dx && !dweight) || (rows == 0 && !dweight)) return ok();
  const size_t need = sv_rms_norm_backward_workspace_size(rows, n, dtype, sum_dtype);
  if (dweight) {
    if (!workspace) return fail(SV_ERR_WORKSPACE, "%s: workspace is NULL (%zu bytes needed)", who, need);
    if (workspace_bytes < need)
      return fail(SV_ERR_WORKSPACE, "%s: workspace has %zu bytes, %zu needed", who, workspace_bytes, need);
    if (!svh::aligned256(workspace)) return fail(SV_ERR_WORKSPACE, "%s: workspace is not 256-byte aligned", who);
  }
  if ((st = check_device()) != SV_OK) return st;
  (void)hipGetLastError();
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const Rows a{rows, (int)n, weight, param_dtype, 0.0, const_cast<float *>(rstd)};
  const int64_t groups = col_groups(dtype, sum_dtype, rows, n), ctiles = col_tiles(dtype, sum_dtype, n);
  Node *part = reinterpret_cast<Node *>(workspace);
  svm::with_types(dtype, sum_dtype, [&](auto t, auto u) {
    using T = decltype(t);
    using S = decltype(u);
    if (rows > 0 && (dh || dx))
      k_rms_dh_any<T, S><<<row_grid(rows), ROW_THREADS, 0, s>>>((const T *)dy, lddy, (const S *)h, ldh, (const S *)dsum,
                                                                lddsum, a, (S *)dh, lddh, (T *)dx, lddx);
    if (dweight)
      k_rms_dw_any<T, S><<<(unsigned)(groups * ctiles), 64 * COL_WAVES, 0, s>>>((const T *)dy, lddy, (const S *)h, ldh,
                                                                               a, (int)groups, (int)ctiles, part);
  });
  if (dweight)
    svh::in_batches((n + 63) / 64, 1, 64 * JOIN_WAVES, [&](int64_t b0, int64_t blocks) {
      k_rms_join<<<(unsigned)blocks, 64 * JOIN_WAVES, 0, s>>>(part, (int)groups, (int)n, (int)b0, dweight, param_dtype);
    });
  return check_launch(who);
}

}  // extern "C"
