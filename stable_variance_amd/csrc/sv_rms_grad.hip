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

// ---------------------------------------------------------------- rows in registers

// Threads of a workgroup of the backward pass: one workgroup per CU with as
// many waves as the registers of E values allow, since every workgroup leaves
// one partial column sum.
constexpr int grad_tpb(int L, int E, int VE) {
  return (E <= 8 || L > 512 ? 1024 : E <= 16 && VE == 8 && L <= 256 ? 768 : 512) / L * L;
}
constexpr int64_t GRAD_BLOCKS = 256;  // one workgroup per CU
// Rows that one thread adds up in plain float32 for the columns' sums; the
// workgroup's groups and then the workgroups are joined with compensation.
constexpr int64_t GRAD_RUN = 32;

// The backward pass of rows that a group of L threads holds in registers, K
// chunks per thread: dy, h and (SUM) dsum are read once, one cross-thread sum
// per row gives c.  The column sums of the rows a group passes stay in
// registers; at the end the workgroup's groups are added up through LDS into
// its row of `part`, [gridDim.x][n], or, by a single workgroup, to dw (part ==
// nullptr: not asked for).
// STREAM: what is read is loaded non-temporal, which leaves the last-level
// cache to dh and its reader.  Measured between kernels that write dsum and dy
// (with 256 MB of other stores between) and one that reads dh, n = 4096 bf16,
// all of it in us, with plain loads and so: 4096 rows (96 MB in) 118 and 115,
// 8192 rows (192 MB) 178 and 168, 10923 rows (256 MB) 224 and 208.  The call by
// itself, whose inputs the cache may hold from before: 28 and 31, 46 and 52, 74
// and 64, for 16384 rows 101 and 94.  So it is taken above 192 MB: up to there
// one of the two gains what the other loses, and at 256 MB both gain.
// Bound by the three or four streams: 16384 x 4096 bf16 with dsum 89 us and 5
// for the join, 6.1 TB/s; 200000 x 128 bf16 33 us, with dsum 43 (4.7 TB/s).  5003
// x 1531 f16 16 us, 3.0 TB/s: 2.4 rounds of rows over the chip, two waves per
// SIMD.
template <class T, class S, bool SUM, bool STREAM, int L, int K, int FIT>
__global__ __launch_bounds__(grad_tpb(L, K * svm::chunk_values<T, S>(), svm::chunk_values<T, S>())) void k_rms_grad(
    const T *__restrict__ dy, int64_t lddy, const S *__restrict__ h, int64_t ldh, const S *__restrict__ dsum,
    int64_t ldds, Rows a, S *__restrict__ dh, int64_t lddh, T *__restrict__ dx, int64_t lddx,
    float *__restrict__ part, void *__restrict__ dw) {
  constexpr int VE = svm::chunk_values<T, S>(), E = K * VE, TPB = grad_tpb(L, E, VE), R = TPB / L;
  using TT = svr::RowTile<T, L, K, FIT, VE>;
  using TS = svr::RowTile<S, L, K, FIT, VE>;
  // 1024 threads leave 128 registers each: the weight then waits in LDS (a
  // thread reads back what it wrote) and the next row is loaded after this one
  constexpr bool FEW = L > 512;
  __shared__ float wlds[FEW ? TPB * E : 1];
  __shared__ float lds[2][TPB / 64];
  __shared__ float cols[TPB * E];
  const int64_t rows = a.rows;
  const int n = a.n, g = svr::group_of<L>(), l0 = threadIdx.x % L;
  const float inv_n = 1.0f / (float)n;
  float wv[FEW ? 1 : K][VE], aw[E];
#pragma unroll
  for (int i = 0; i < E; ++i) aw[i] = 0.0f;
  const int64_t step = (int64_t)gridDim.x * R;
  typename TS::Vec rh[K], rd[SUM ? K : 1];
  typename TT::Vec rg[K];
  int64_t r = (int64_t)blockIdx.x * R + g;
  int64_t rl = R == 1 || r < rows ? r : rows - 1;  // the row that is loaded
  float rs_next;
  const auto load = [&](int l) {
    TS::template load<STREAM>(h + rl * ldh, n, TS::avail(rows, rl, ldh, n), l, rh);
    TT::template load<STREAM>(dy + rl * lddy, n, TT::avail(rows, rl, lddy, n), l, rg);
    if constexpr (SUM) TS::template load<STREAM>(dsum + rl * ldds, n, TS::avail(rows, rl, ldds, n), l, rd);
    rs_next = a.rstd[rl];
  };
  const auto arrived = [&] {
    TS::arrived(rh, rs_next);
    TT::arrived(rg);
    if constexpr (SUM) TS::arrived(rd);
  };
  load(l0);
#pragma unroll
  for (int k = 0; k < K; ++k) {  // in flight beside the first row
    const int e = TT::first(l0, k), left = n - e;
    svm::get_weight<T, VE, FIT != svr::FIT_CHUNKS>(a.w, a.pt, e, left < 0 ? 0 : left, wv[FEW ? 0 : k]);
    if constexpr (FEW) {
#pragma unroll
      for (int i = 0; i < VE; ++i) wlds[e + i] = wv[0][i];
    }
  }
  if constexpr (!FEW) arrived();
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * R; r0 < rows; r0 += step, r += step, turn ^= 1) {
    int l = l0;  // opaque, so that the addresses of all chunks are not kept in registers across rows
    asm volatile("" : "+v"(l));
    float x[E], v[E], d[SUM ? E : 1];
    TS::unpack(rh, x);
    TT::unpack(rg, v);
    TS::load_rest(h + rl * ldh, n, TS::avail(rows, rl, ldh, n), l, x);
    TT::load_rest(dy + rl * lddy, n, TT::avail(rows, rl, lddy, n), l, v);
    if constexpr (SUM) {
      TS::unpack(rd, d);
      TS::load_rest(dsum + rl * ldds, n, TS::avail(rows, rl, ldds, n), l, d);
    }
    const float rs = rs_next;
    rl = r + step < rows ? r + step : rows - 1;
    if constexpr (!FEW) load(l);
    TS::set_rest(n, l, 0.0f, x);
    TT::set_rest(n, l, 0.0f, v);
    const auto weight = [&](int i) { return FEW ? wlds[TT::first(l, i / VE) + i % VE] : wv[FEW ? 0 : i / VE][i % VE]; };
    const bool own = R == 1 || r < rows;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      x[i] = x[i] * rs;
      if (own) aw[i] = aw[i] + v[i] * x[i];
      v[i] = v[i] * weight(i);
    }
    float s[1] = {TT::sum(n, l, [&](int i) { return v[i] * x[i]; })};
    svr::group_sum<L, 1>(s, lds[turn]);
    const float c = s[0] * inv_n;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      v[i] = rs * (v[i] - x[i] * c);
      if constexpr (SUM) v[i] = v[i] + d[i];
    }
    if constexpr (!FEW) arrived();
    if (own && dh) {
#pragma unroll
      for (int k = 0; k < K; ++k) TS::store_chunk(dh + r * lddh, n, l, k, v);
    }
    if (own && dx) {
#pragma unroll
      for (int k = 0; k < K; ++k) TT::store_chunk(dx + r * lddx, n, l, k, v);
    }
    if constexpr (FEW) {
      __builtin_amdgcn_sched_barrier(0);
      load(l);
    }
  }
  if (!part) return;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < VE; ++i) cols[g * (L * E) + TT::first(l0, k) + i] = aw[k * VE + i];
  __syncthreads();
  float *out = part + (int64_t)blockIdx.x * n;
  for (int j = threadIdx.x; j < n; j += TPB) {
    Node t = sv::zero_node();
    for (int q = 0; q < R; ++q) svr::add_to(t, cols[q * (L * E) + j]);
    if (gridDim.x == 1) svr::store_as(dw, j, a.pt, sv::root_value(t));
    else out[j] = sv::root_value(t);
  }
}

// Calls fn(L, K, FIT) (integral constants) with the smallest tile of VE-value
// chunks that holds n values; false when none does.  Rows of whole chunks have
// kernels of their own only for 1024 threads, where no register is left for the
// others, and (`whole`) for inputs that are loaded non-temporal: elsewhere they
// gain up to 4% (4096 x 4096 bf16 22.6 against 23.6 us) and with the forward
// pass's that would be a third of the library.
template <int VE, class Fn>
bool with_tile(int64_t n, bool whole, Fn &&fn) {
  if (n < 1) return false;
  const auto tile = [&](auto tl, auto tk) {
    constexpr int L = decltype(tl)::value, K = decltype(tk)::value;
    if constexpr (L == 1) {
      if (n < VE) {
        fn(tl, tk, std::integral_constant<int, svr::FIT_SMALL>{});
        return true;
      }
    }
    if (n > (int64_t)L * K * VE) return false;
    if constexpr (L >= 128) {
      if (n % VE == 0 && (L > 512 || whole)) {
        fn(tl, tk, std::integral_constant<int, svr::FIT_CHUNKS>{});
        return true;
      }
    }
    if constexpr (L <= 512) fn(tl, tk, std::integral_constant<int, svr::FIT_ANY>{});
    return L <= 512;
  };
#define SV_TILE(L, V) \
  if (tile(std::integral_constant<int, L>{}, std::integral_constant<int, (V) / VE>{})) return true;
  SV_TILE(1, 8) SV_TILE(4, 8) SV_TILE(8, 8) SV_TILE(8, 16)
  SV_TILE(16, 16) SV_TILE(32, 16) SV_TILE(64, 16) SV_TILE(64, 24)
  SV_TILE(128, 16) SV_TILE(256, 16) SV_TILE(256, 24) SV_TILE(512, 16) SV_TILE(512, 24)
  SV_TILE(1024, 16)
#undef SV_TILE
  return false;
}

// Workgroups of k_rms_grad (0: the rows are too long for it).  Every group of
// a workgroup passes at most GRAD_RUN rows.
int64_t grad_blocks(int dtype, int sum_dtype, int64_t rows, int64_t n) {
  int64_t blocks = 0;
  svm::with_types(dtype, sum_dtype, [&](auto t, auto u) {
    constexpr int VE = svm::chunk_values<decltype(t), decltype(u)>();
    with_tile<VE>(n, false, [&](auto tl, auto tk, auto) {
      constexpr int L = decltype(tl)::value, E = decltype(tk)::value * VE;
      constexpr int64_t R = grad_tpb(L, E, VE) / L;
      const int64_t all = (rows + R - 1) / R;
      const int64_t rounds = (all + GRAD_RUN * GRAD_BLOCKS - 1) / (GRAD_RUN * GRAD_BLOCKS);
      blocks = all < GRAD_BLOCKS ? all : rounds * GRAD_BLOCKS;  // whole rounds of the chip
      if (blocks < 1) blocks = 1;
    });
  });
  return blocks;
}

// ---------------------------------------------------------------- longer rows

// The rows' part of the backward pass for rows of any length: dy and h are read
// twice here and once more for the columns.  Both parts and the join: 2000 x
// 12291 bf16 94 us, 2000 x 20000 104 us (2.3 TB/s of what is read and written
// once), in float32 118 and 186, where 2000 x 12288 bf16 held in registers take 35.
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
      svm::get_weight<T, VE>(a.w, a.pt, e, count, w);
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
__device__ __forceinline__ Node node_of(float v) { return {v, 0.0f}; }
__device__ __forceinline__ Node node_of(Node v) { return v; }

constexpr int JOIN_WAVES = 16;
template <class P>
__global__ __launch_bounds__(64 * JOIN_WAVES) void k_rms_join(const P *part, int groups, int n, int b0, void *dw,
                                                              int pt) {
  __shared__ Node lds[JOIN_WAVES][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t j = ((int64_t)b0 + blockIdx.x) * 64 + lane;
  Node s = sv::zero_node();
  if (j < n) {
#pragma unroll 8
    for (int q = wave; q < groups; q += JOIN_WAVES) s = sv::combine(s, node_of(part[(int64_t)q * n + j]));
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

// k_rms_join over all columns, in launches within HIP's limit.
template <class P>
void join_columns(const P *part, int64_t groups, int64_t n, void *dw, int pt, hipStream_t s) {
  svh::in_batches((n + 63) / 64, 1, 64 * JOIN_WAVES, [&](int64_t b0, int64_t blocks) {
    k_rms_join<P><<<(unsigned)blocks, 64 * JOIN_WAVES, 0, s>>>(part, (int)groups, (int)n, (int)b0, dw, pt);
  });
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
  const int64_t blocks = grad_blocks(dtype, sum_dtype, rows, n);
  if (blocks) return svr::round256((size_t)blocks * (size_t)n * sizeof(float));
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
  if ((st = svr::check_stats(who, "rstd", rstd, rows)) != SV_OK) return st;
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
  const int64_t blocks = grad_blocks(dtype, sum_dtype, rows, n);
  const int64_t groups = col_groups(dtype, sum_dtype, rows, n), ctiles = col_tiles(dtype, sum_dtype, n);
  svm::with_types(dtype, sum_dtype, [&](auto t, auto u) {
    using T = decltype(t);
    using S = decltype(u);
    constexpr int VE = svm::chunk_values<T, S>();
    const T *g = (const T *)dy;
    const S *x = (const S *)h, *d = (const S *)dsum;
    if (blocks) {
      float *part = dweight ? reinterpret_cast<float *>(workspace) : nullptr;
      const bool stream = rows * n * (int64_t)(sizeof(T) + (d ? 2 : 1) * sizeof(S)) > svm::LAST_LEVEL / 4 * 3;
      if (rows > 0)
        with_tile<VE>(n, stream, [&](auto tl, auto tk, auto tf) {
          constexpr int L = decltype(tl)::value, K = decltype(tk)::value, FIT = decltype(tf)::value;
          const auto rows_of = [&](auto sum, auto st) {
            k_rms_grad<T, S, decltype(sum)::value, decltype(st)::value, L, K, FIT>
                <<<(unsigned)blocks, grad_tpb(L, K * VE, VE), 0, s>>>(g, lddy, x, ldh, d, lddsum, a, (S *)dh, lddh,
                                                                      (T *)dx, lddx, part, dweight);
          };
          const auto launch = [&](auto st) {
            if (dsum) rows_of(std::true_type{}, st);
            else rows_of(std::false_type{}, st);
          };
          if constexpr (FIT == svr::FIT_CHUNKS) {
            if (stream) return launch(std::true_type{});
          }
          if constexpr (FIT != svr::FIT_CHUNKS || L > 512) launch(std::false_type{});
        });
      if (dweight && (rows == 0 || blocks > 1)) join_columns(part, rows > 0 ? blocks : 0, n, dweight, param_dtype, s);
      return;
    }
    Node *part = reinterpret_cast<Node *>(workspace);
    if (rows > 0 && (dh || dx))
      k_rms_dh_any<T, S><<<svm::row_grid(rows), ROW_THREADS, 0, s>>>(g, lddy, x, ldh, d, lddsum, a, (S *)dh, lddh,
                                                                     (T *)dx, lddx);
    if (dweight) {
      k_rms_dw_any<T, S><<<(unsigned)(groups * ctiles), 64 * COL_WAVES, 0, s>>>(g, lddy, x, ldh, a, (int)groups,
                                                                               (int)ctiles, part);
      join_columns(part, groups, n, dweight, param_dtype, s);
    }
  });
  return check_launch(who);
}

}  // extern "C"
