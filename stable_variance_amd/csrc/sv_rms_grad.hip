// Backward pass of the root-mean-square norm (the formulas are at the head of
// sv_rms.hip).
#include "sv_rms.hpp"

using svh::check_device;
using svh::check_launch;
using svh::fail;
using svh::ok;
using svm::ROW_THREADS;
using svm::Rows;
using svr::Node;

namespace {

constexpr int COL_ROWS = 64;  // rows of one partial column sum
constexpr int64_t COL_MAX_GROUPS = 512;

// The rows' part of the backward pass for rows of any length.
template <class T, class S>
__global__ __launch_bounds__(ROW_THREADS) void k_rms_dh_any(const T *dy, int64_t lddy, const S *h, int64_t ldh,
                                                            const S *dsum, int64_t ldds, Rows a, S *dh, int64_t lddh,
                                                            T *dx, int64_t lddx) {
  constexpr int VE = svm::chunk_values<T, S>(), STEP = ROW_THREADS * VE;
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
  constexpr int VE = svm::chunk_values<T, S>();
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

}  // namespace

extern "C" {

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
  sv_status st = svm::check_rows(who, dtype, sum_dtype, rows, n, param_dtype);
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
      k_rms_dh_any<T, S><<<svm::row_grid(rows), ROW_THREADS, 0, s>>>((const T *)dy, lddy, (const S *)h, ldh, (const S *)dsum,
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
