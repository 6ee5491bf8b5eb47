// Layer norm over the rows of a matrix, forward and backward, on gfx950.
//
// Forward, for a row x of n values (all in float32):
//   m1  = fl(x_0 + sum(x_i - x_0) / n)          shift by the first value
//   d_i = x_i - m1,  b = sum(d_i) / n           local centring; b is what m1
//                                               is off by
//   var = max(sum(d_i^2) / n - b^2, 0)          two-term correction
//   mean = m1 + b,  rstd = 1 / sqrt(var + eps)
//   y_i = (d_i - b) * rstd * w_i + bias_i       rounded once to x's type
// the shift, centring and correction of the variance in sv_lib.hip: a row of
// equal values has d = 0 exactly, and a mean far from zero cancels before
// anything is squared.
//
// Backward, with the mean and rstd the forward pass wrote, d_i = x_i - mean,
// b = sum(d) / n (what the float32 mean is off by), g_i = dy_i * w_i:
//   xhat_i = (d_i - b) * rstd
//   dx_i = rstd * ((g_i - sum(g) / n) - xhat_i * c),
//          c = rstd * (sum(g d) - b * sum(g)) / n  ( = sum(g xhat) / n )
//   dw_j = sum over rows of dy * xhat,  dbias_j = sum over rows of dy.
//
// Every sum has one fixed order given by the shape and the type, so results
// are the same bits from run to run, and a row's y and dx do not depend on
// the other rows.
#include "sv_rows.hpp"

using svh::check_device;
using svh::check_launch;
using svh::fail;
using svh::ok;
using svr::Node;

namespace {

constexpr int ROW_THREADS = 512;
constexpr int64_t ROW_GRID = 8192;     // workgroups of a row launch, at most
constexpr int COL_ROWS = 64;           // rows of one partial column sum
constexpr int64_t COL_MAX_GROUPS = 512;

// 1 / sqrt(v) in double (one Newton step from the hardware's estimate, about
// 2^-46), so that the float32 value is the rounded one; 0, Inf and NaN as
// the estimate gives them.  Above float32's range (var = 0 and eps below
// 8.6e-78) it is the largest finite value: with Inf, equal values would give
// 0 * Inf = NaN in place of the bias, and NaN gradients.
__device__ __forceinline__ float rstd_of(float var, double eps) {
  const double v = (double)var + eps;
  const double r = __builtin_amdgcn_rsq(v);
  const double e = 1.0 - v * r * r;
  const double s = r + 0.5 * r * e;
  const float f = (float)(__builtin_isfinite(e) ? s : r);
  return v > 0.0 && f > __FLT_MAX__ ? __FLT_MAX__ : f;
}

// Sum of one node per thread over the workgroup, in a fixed order; every
// thread gets the root's value.  `lds` holds a node per wave.
template <int WAVES>
__device__ __forceinline__ float block_sum(Node n, Node *lds) {
  n = sv::wave_tree<sv::NODE_TWOSUM>(n);
  if constexpr (WAVES > 1) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = n;
    __syncthreads();
    Node w[WAVES];
#pragma unroll
    for (int i = 0; i < WAVES; ++i) w[i] = lds[i];
    n = sv::node_tree<0, WAVES, WAVES>(w);
  }
  return sv::root_value(n);
}

// Threads of a workgroup whose groups of L threads hold a row each.
constexpr int tpb(int L) { return L <= 128 ? 256 : L; }

// Rows that a group of L threads holds in registers, K chunks of 16 bytes per
// thread: the row is read once, and the group's R - 1 neighbours in the
// workgroup hold other rows.  The next row's loads are in flight while a row
// is summed (waited for before this row's stores, so that no store is ever
// waited for), and up to 24 values' parameters stay in registers across rows.
// Plain pairwise sums: with the shift and the second centring each is a sum
// of values of the size of the spread.  Up to 15 levels of additions (32768
// values) round by at most 15 u of it, u = 2^-24: far below the rounding of a
// 16-bit result (2^-8 or 2^-11 of it), a few steps of a float32 one.
// Bound by the read and the write: 16384 x 4096 bf16 51-54 us, 5.0-5.3 TB/s,
// 4096 x 4096 float32 24-26 us; a large copy runs at 4.9-5.3 TB/s.  Next to
// that is the vector unit (about 265 instructions per row and wave at 16 values
// a thread, three quarters of the time).  Lengths that end inside a chunk: 43833
// x 1531 bf16 64-67 us, 4.1 TB/s.
template <class T, int L, int K, int FIT>
__global__ __launch_bounds__(tpb(L)) void k_norm_rows(
    const T *__restrict__ x, int64_t rows, int n, int64_t ldx, const void *__restrict__ w,
    const void *__restrict__ bias, int pt, double eps, T *__restrict__ y, int64_t ldy, float *__restrict__ mean,
    float *__restrict__ rstd) {
  using Tile = svr::RowTile<T, L, K, FIT>;
  constexpr int E = Tile::E, TPB = tpb(L), R = TPB / L;
  constexpr bool HOLD = E <= 24;
  __shared__ float lds_a[TPB / 64], lds_b[2 * TPB / 64];
  const int g = svr::group_of<L>(), l0 = threadIdx.x % L;
  const float inv_n = 1.0f / (float)n;
  constexpr int VE = Tile::VE;
  float wv[HOLD ? E : 1], bv[HOLD ? E : 1];
  if constexpr (HOLD) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      svr::load_param<T, L>(w, pt, n, l0, k, 1.0f, wv + k * VE);
      svr::load_param<T, L>(bias, pt, n, l0, k, 0.0f, bv + k * VE);
    }
  }
  const int64_t step = (int64_t)gridDim.x * R;
  typename Tile::Vec raw[K];
  int64_t r = (int64_t)blockIdx.x * R + g;
  int64_t rl = R == 1 || r < rows ? r : rows - 1;  // the row that is loaded
  Tile::load(x + rl * ldx, n, Tile::avail(rows, rl, ldx, n), l0, raw);
  T first = x[rl * ldx];
  if constexpr (HOLD) Tile::arrived(raw, first);
  for (int64_t r0 = (int64_t)blockIdx.x * R; r0 < rows; r0 += step, r += step) {
    int l = l0;  // opaque, so that the addresses of all chunks are not kept in registers across rows
    asm volatile("" : "+v"(l));
    float f[E];
    Tile::unpack(raw, f);
    Tile::load_rest(x + rl * ldx, n, Tile::avail(rows, rl, ldx, n), l, f);
    const float x0 = svr::to_f(first);
    rl = r + step < rows ? r + step : rows - 1;
    if constexpr (HOLD) {
      Tile::load(x + rl * ldx, n, Tile::avail(rows, rl, ldx, n), l, raw);
      first = x[rl * ldx];
    }
    Tile::set_rest(n, l, x0, f);
    float a[1] = {Tile::sum(n, l, [&](int i) { return f[i] - x0; })};
    svr::group_sum<L, 1>(a, lds_a);
    const float m1 = x0 + a[0] * inv_n;
    Tile::set_rest(n, l, m1, f);
#pragma unroll
    for (int i = 0; i < E; ++i) f[i] = f[i] - m1;
    float s[2] = {Tile::sum(n, l, [&](int i) { return f[i]; }), Tile::sum(n, l, [&](int i) { return f[i] * f[i]; })};
    svr::group_sum<L, 2>(s, lds_b);
    const float b = s[0] * inv_n;
    const float q = s[1] * inv_n - b * b;
    const float rs = rstd_of(q <= 0.0f ? 0.0f : q, eps);  // a NaN stays
    if (R == 1 || r < rows) {
      if (l == 0) {
        if (mean) mean[r] = m1 + b;
        if (rstd) rstd[r] = rs;
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float wk[VE], bk[VE];
        if constexpr (!HOLD) {
          svr::load_param<T, L>(w, pt, n, l, k, 1.0f, wk);
          svr::load_param<T, L>(bias, pt, n, l, k, 0.0f, bk);
        }
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          const float ww = HOLD ? wv[HOLD ? k * VE + i : 0] : wk[i], bb = HOLD ? bv[HOLD ? k * VE + i : 0] : bk[i];
          f[k * VE + i] = ((f[k * VE + i] - b) * rs) * ww + bb;
        }
        if constexpr (!HOLD) {
          Tile::store_chunk(y + r * ldy, n, l, k, f);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    if constexpr (HOLD) {
      Tile::arrived(raw, first);
      if (R == 1 || r < rows) {
#pragma unroll
        for (int k = 0; k < K; ++k) Tile::store_chunk(y + r * ldy, n, l, k, f);
      }
    }
    if constexpr (!HOLD) {
      Tile::load(x + rl * ldx, n, Tile::avail(rows, rl, ldx, n), l, raw);
      first = x[rl * ldx];
    }
  }
}

// The backward pass's tiles: up to 24 values on 512 threads and 16 on 1024 (their
// registers also hold the column sums), and 16 values for the shorter float32 rows
// (446666 x 150: 205 us with 24 values, 170 with 16; bfloat16 is the other way
// round, 43762 x 1531: 82 us with 24, 108 with 16).
constexpr bool grad_tile(int L, int E, int VE) {
  return (L <= 512 ? E <= 24 : E <= 16) && !(VE == 4 && E == 24 && L <= 64);
}

// Calls fn(L, K, FIT) (integral constants) with the smallest tile of the
// forward (GRAD: backward) pass that holds n values of T; false when none
// does.  The choice follows from n and the type alone.
template <class T, bool GRAD, class Fn>
bool with_tile(int64_t n, Fn &&fn) {
  constexpr int VE = svr::Chunk<T>::VE;
  if (n < 1) return false;
  const auto tile = [&](auto tl, auto tk) {
    constexpr int L = decltype(tl)::value, K = decltype(tk)::value;
    if constexpr (!GRAD || grad_tile(L, K * VE, VE)) {
      if (n > (int64_t)L * K * VE) return false;
      if constexpr (L == 1) {
        if (n < VE) {
          fn(tl, tk, std::integral_constant<int, svr::FIT_SMALL>{});
          return true;
        }
      }
      constexpr bool WHOLE = GRAD && L > 512;  // whole chunks only: no register is left for the others
      if (WHOLE && n % VE != 0) return false;
      if (n == (int64_t)L * K * VE) fn(tl, tk, std::integral_constant<int, svr::FIT_FULL>{});
      else if (n % VE == 0) fn(tl, tk, std::integral_constant<int, svr::FIT_CHUNKS>{});
      else if constexpr (!WHOLE) fn(tl, tk, std::integral_constant<int, svr::FIT_ANY>{});
      return true;
    }
    return false;
  };
#define SV_TILE(L, V) \
  if (tile(std::integral_constant<int, L>{}, std::integral_constant<int, (V) / VE>{})) return true;
  // Up to 64 values: 8 per thread, so that a row's lanes read whole cache
  // lines together; then 16 (half the cost per value of the cross-lane sums),
  // or 24 where that leaves fewer threads idle; 32 for the longest rows.
  SV_TILE(1, 8) SV_TILE(2, 8) SV_TILE(4, 8) SV_TILE(8, 8) SV_TILE(8, 16) SV_TILE(8, 24)
  SV_TILE(16, 16) SV_TILE(16, 24) SV_TILE(32, 16) SV_TILE(32, 24) SV_TILE(64, 16) SV_TILE(64, 24)
  SV_TILE(128, 16) SV_TILE(256, 16) SV_TILE(256, 24) SV_TILE(512, 16) SV_TILE(512, 24)
  SV_TILE(1024, 16) SV_TILE(1024, 32)
#undef SV_TILE
  return false;
}

// Rows of any length: a workgroup per row, each pass reads the row again (from
// the cache where it fits).  Compensated sums, as a thread adds up a long run
// of chunks one by one.  335 x 200000 bf16: 151 us, 1.8 TB/s (a row's two later
// passes and the parameters come from the cache).
template <class T>
__global__ __launch_bounds__(ROW_THREADS) void k_norm_any(const T *__restrict__ x, int64_t rows, int n, int64_t ldx,
                                                          const void *__restrict__ w, const void *__restrict__ bias,
                                                          int pt, double eps, T *__restrict__ y, int64_t ldy,
                                                          float *__restrict__ mean, float *__restrict__ rstd) {
  constexpr int VE = svr::Chunk<T>::VE;
  __shared__ Node lds[ROW_THREADS / 64];
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const T *xr = x + r * ldx;
    const float fn = (float)n;
    const float x0 = n > 0 ? svr::to_f(xr[0]) : 0.0f;
    Node a = sv::zero_node();
    svr::for_chunks(xr, n, threadIdx.x, ROW_THREADS, [&](int, const float *f, int count) {
      svr::add_to(a, svr::pair_sum<0, VE>([&](int i) { return i < count ? f[i] - x0 : 0.0f; }));
    });
    const float m1 = x0 + block_sum<ROW_THREADS / 64>(a, lds) / fn;
    Node s1 = sv::zero_node(), s2 = sv::zero_node();
    svr::for_chunks(xr, n, threadIdx.x, ROW_THREADS, [&](int, float *f, int count) {
#pragma unroll
      for (int i = 0; i < VE; ++i) f[i] = i < count ? f[i] - m1 : 0.0f;
      svr::add_to(s1, svr::pair_sum<0, VE>([&](int i) { return f[i]; }));
      svr::add_to(s2, svr::pair_sum<0, VE>([&](int i) { return f[i] * f[i]; }));
    });
    const float b = block_sum<ROW_THREADS / 64>(s1, lds) / fn;
    const float q = block_sum<ROW_THREADS / 64>(s2, lds) / fn - b * b;
    const float var = q <= 0.0f ? 0.0f : q;  // a NaN stays
    const float rs = rstd_of(var, eps);
    if (threadIdx.x == 0) {
      if (mean) mean[r] = m1 + b;
      if (rstd) rstd[r] = rs;
    }
    T *yr = y + r * ldy;
    svr::for_chunks(xr, n, threadIdx.x, ROW_THREADS, [&](int e, float *f, int count) {
      float wv[VE], bv[VE];
      svr::load_param<T, 1>(w, pt, n, 0, e / VE, 1.0f, wv);
      svr::load_param<T, 1>(bias, pt, n, 0, e / VE, 0.0f, bv);
#pragma unroll
      for (int i = 0; i < VE; ++i) f[i] = (((f[i] - m1) - b) * rs) * wv[i] + bv[i];
      svr::put_chunk(yr, e, count, f);
    });
  }
}

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

// The backward pass of rows that L threads hold (see k_norm_rows): x and dy
// are read once.  One cross-thread sum per row gives sum(d), sum(g) and
// sum(g d).  The column sums of the rows a group passes stay in registers;
// at the end the workgroup's groups are added up through LDS into its row
// of `part`, [gridDim.x][2][n] (part == nullptr: not asked for).  dx is stored
// non-temporal (16384 x 4096 bf16: 82 us plain, 76-80 so); the forward pass
// keeps plain stores, whose result is read next and gains from the cache (48
// us plain, 53 non-temporal).
// Bound by the three streams: 16384 x 4096 bf16 80 us with the join, 5.1 TB/s;
// the same size in float32 152 us, 5.3 TB/s.
template <class T, int L, int K, int FIT>
__global__ __launch_bounds__(grad_tpb(L, K * svr::Chunk<T>::VE, svr::Chunk<T>::VE)) void k_norm_grad(
    const T *__restrict__ dy, int64_t lddy, const T *__restrict__ x, int64_t ldx, int64_t rows, int n,
    const void *__restrict__ w, int pt, const float *__restrict__ mean, const float *__restrict__ rstd,
    T *__restrict__ dx, int64_t lddx, float *__restrict__ part) {
  using Tile = svr::RowTile<T, L, K, FIT>;
  constexpr int E = Tile::E, VE = Tile::VE, TPB = grad_tpb(L, E, VE), R = TPB / L;
  // 1024 threads leave 128 registers each: the weight then waits in LDS (a
  // thread reads back what it wrote) and the next row is loaded after this one
  constexpr bool FEW = L > 512;
  constexpr bool AHEAD = !FEW && !(VE == 4 && E > 16 && L > 256 && FIT == svr::FIT_ANY);
  __shared__ float wlds[FEW ? TPB * E : 1];
  __shared__ float lds[2][3 * TPB / 64];
  __shared__ float cols[TPB * E];
  const int g = svr::group_of<L>(), l0 = threadIdx.x % L;
  const float inv_n = 1.0f / (float)n;
  float wv[FEW ? VE : E], aw[E], ab[E];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    svr::load_param<T, L>(w, pt, n, l0, k, 1.0f, wv + (FEW ? 0 : k * VE));
    if constexpr (FEW) {
#pragma unroll
      for (int i = 0; i < VE; ++i) wlds[Tile::first(l0, k) + i] = wv[i];
    }
  }
#pragma unroll
  for (int i = 0; i < E; ++i) aw[i] = ab[i] = 0.0f;
  const int64_t step = (int64_t)gridDim.x * R;
  typename Tile::Vec rx[K], rg[K];
  int64_t r = (int64_t)blockIdx.x * R + g;
  int64_t rl = R == 1 || r < rows ? r : rows - 1;  // the row that is loaded
  Tile::load(x + rl * ldx, n, Tile::avail(rows, rl, ldx, n), l0, rx);
  Tile::load(dy + rl * lddy, n, Tile::avail(rows, rl, lddy, n), l0, rg);
  float m = mean[rl], rs = rstd[rl];
  if constexpr (AHEAD) {
    Tile::arrived(rx, m);
    Tile::arrived(rg, rs);
  }
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * R; r0 < rows; r0 += step, r += step, turn ^= 1) {
    int l = l0;  // opaque, as in k_norm_rows
    asm volatile("" : "+v"(l));
    float d[E], gy[E];
    Tile::unpack(rx, d);
    Tile::unpack(rg, gy);
    Tile::load_rest(x + rl * ldx, n, Tile::avail(rows, rl, ldx, n), l, d);
    Tile::load_rest(dy + rl * lddy, n, Tile::avail(rows, rl, lddy, n), l, gy);
    const float mu = m, rr = rs;
    rl = r + step < rows ? r + step : rows - 1;
    const auto load_next = [&] {
      Tile::load(x + rl * ldx, n, Tile::avail(rows, rl, ldx, n), l, rx);
      Tile::load(dy + rl * lddy, n, Tile::avail(rows, rl, lddy, n), l, rg);
      m = mean[rl];
      rs = rstd[rl];
    };
    if constexpr (AHEAD) load_next();
    Tile::set_rest(n, l, mu, d);
    Tile::set_rest(n, l, 0.0f, gy);
#pragma unroll
    for (int i = 0; i < E; ++i) d[i] = d[i] - mu;
    const auto weight = [&](int i) { return FEW ? wlds[Tile::first(l, i / VE) + i % VE] : wv[FEW ? 0 : i]; };
    float s[3] = {Tile::sum(n, l, [&](int i) { return d[i]; }),
                  Tile::sum(n, l, [&](int i) { return gy[i] * weight(i); }),
                  Tile::sum(n, l, [&](int i) { return (gy[i] * weight(i)) * d[i]; })};
    svr::group_sum<L, 3>(s, lds[turn]);
    const float b = s[0] * inv_n, a = s[1] * inv_n;
    const float c = rr * ((s[2] - b * s[1]) * inv_n);
    const bool own = R == 1 || r < rows;
    // keeps the compiler from spreading a step's values over the next
    const auto step_done = [] {
      if constexpr (FEW) __builtin_amdgcn_sched_barrier(0);
    };
    step_done();
#pragma unroll
    for (int i = 0; i < E; ++i) {
      if (i % VE == 0) step_done();
      const float xh = (d[i] - b) * rr;
      if (own) {
        aw[i] = aw[i] + gy[i] * xh;
        ab[i] = ab[i] + gy[i];
      }
      d[i] = rr * ((gy[i] * weight(i) - a) - xh * c);
    }
    step_done();
    if constexpr (AHEAD) {
      Tile::arrived(rx, m);
      Tile::arrived(rg, rs);
    }
    if (own && dx) {
#pragma unroll
      for (int k = 0; k < K; ++k) Tile::template store_chunk<true>(dx + r * lddx, n, l, k, d);
    }
    step_done();
    if constexpr (!AHEAD) load_next();
  }
  if (!part) return;
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < VE; ++i)
        cols[g * (L * E) + Tile::first(l0, k) + i] = which ? ab[k * VE + i] : aw[k * VE + i];
    __syncthreads();
    float *out = part + ((int64_t)blockIdx.x * 2 + which) * n;
    for (int j = threadIdx.x; j < n; j += TPB) {
      Node t = sv::zero_node();
      for (int q = 0; q < R; ++q) svr::add_to(t, cols[q * (L * E) + j]);
      out[j] = sv::root_value(t);
    }
  }
}

// The rows' part of the backward pass for longer rows, whose column sums no
// workgroup's registers hold (more than 16384 values, or more than 12288 that
// end inside a chunk): dx and, for the column sums, b.  With k_norm_dw_any x and dy are read from memory twice: 3355 x
// 20000 bf16 178 us, 2.3 TB/s of the call's own bytes.
template <class T>
__global__ __launch_bounds__(ROW_THREADS) void k_norm_dx_any(
    const T *__restrict__ dy, int64_t lddy, const T *__restrict__ x, int64_t ldx, int64_t rows, int n,
    const void *__restrict__ w, int pt, const float *__restrict__ mean, const float *__restrict__ rstd,
    T *__restrict__ dx, int64_t lddx, float *__restrict__ off) {
  constexpr int VE = svr::Chunk<T>::VE;
  __shared__ Node lds[ROW_THREADS / 64];
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const T *xr = x + r * ldx, *gr = dy + r * lddy;
    const float fn = (float)n, m = mean[r], rs = rstd[r];
    // fn(e, d, g, count) over the row's chunks
    const auto chunks = [&](auto &&fn2) {
      svr::for_chunks(xr, n, threadIdx.x, ROW_THREADS, [&](int e, float *d, int count) {
        float wv[VE];
        svr::load_param<T, 1>(w, pt, n, 0, e / VE, 1.0f, wv);
        svr::for_chunks(gr + e, count, 0, 1, [&](int, float *g, int) {
#pragma unroll
          for (int i = 0; i < VE; ++i) {
            d[i] = i < count ? d[i] - m : 0.0f;
            g[i] = g[i] * wv[i];  // past the row 0 * 1
          }
          fn2(e, d, g, count);
        });
      });
    };
    Node sd = sv::zero_node(), sg = sv::zero_node(), sgd = sv::zero_node();
    chunks([&](int, const float *d, const float *g, int) {
      svr::add_to(sd, svr::pair_sum<0, VE>([&](int i) { return d[i]; }));
      svr::add_to(sg, svr::pair_sum<0, VE>([&](int i) { return g[i]; }));
      svr::add_to(sgd, svr::pair_sum<0, VE>([&](int i) { return g[i] * d[i]; }));
    });
    const float b = block_sum<ROW_THREADS / 64>(sd, lds) / fn;
    const float sumg = block_sum<ROW_THREADS / 64>(sg, lds);
    const float sumgd = block_sum<ROW_THREADS / 64>(sgd, lds);
    const float a = sumg / fn;
    const float c = rs * ((sumgd - b * sumg) / fn);
    if (off && threadIdx.x == 0) off[r] = b;
    if (dx) {
      T *dr = dx + r * lddx;
      chunks([&](int e, const float *d, const float *g, int count) {
        float v[VE];
#pragma unroll
        for (int i = 0; i < VE; ++i) v[i] = rs * ((g[i] - a) - ((d[i] - b) * rs) * c);
        svr::put_chunk(dr, e, count, v);
      });
    }
  }
}

// The columns' part for longer rows: group q of the rows (row r belongs to
// group r mod groups) and 64 chunks of columns per workgroup; each wave takes
// every fourth row of the group.
constexpr int COL_WAVES = 4;
template <class T>
__global__ __launch_bounds__(64 * COL_WAVES) void k_norm_dw_any(
    const T *__restrict__ dy, int64_t lddy, const T *__restrict__ x, int64_t ldx, int64_t rows, int n,
    const float *__restrict__ mean, const float *__restrict__ rstd, const float *__restrict__ off, int groups,
    int ctiles, Node *__restrict__ part) {
  constexpr int VE = svr::Chunk<T>::VE;
  __shared__ Node lds[COL_WAVES][64][VE];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int q = blockIdx.x / ctiles;
  // the last chunk ends with the row and repeats some of the one before (n >= VE)
  const int chunk = (blockIdx.x % ctiles) * 64 + lane;
  const bool in = (int64_t)chunk * VE < n;
  const int j = !in ? 0 : chunk * VE + VE <= n ? chunk * VE : n - VE;
  Node dw[VE], db[VE];
#pragma unroll
  for (int i = 0; i < VE; ++i) dw[i] = db[i] = sv::zero_node();
#pragma unroll 2
  for (int64_t r = q + (int64_t)wave * groups; r < rows; r += COL_WAVES * (int64_t)groups) {
    const float m = mean[r], b = off[r], rs = rstd[r];
    typename svr::Chunk<T>::Vec gv, xv;
    __builtin_memcpy(&gv, dy + r * lddy + j, 16);
    __builtin_memcpy(&xv, x + r * ldx + j, 16);
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const float g = svr::to_f<T>(gv[i]);
      svr::add_to(dw[i], g * (((svr::to_f<T>(xv[i]) - m) - b) * rs));
      svr::add_to(db[i], g);
    }
  }
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < VE; ++i) lds[wave][lane][i] = which ? db[i] : dw[i];
    __syncthreads();
    if (wave == 0 && in) {
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        Node t[COL_WAVES];
#pragma unroll
        for (int v = 0; v < COL_WAVES; ++v) t[v] = lds[v][lane][i];
        part[((int64_t)q * 2 + which) * n + j + i] = sv::node_tree<0, COL_WAVES, COL_WAVES>(t);
      }
    }
  }
}

__device__ __forceinline__ Node node_of(float v) { return {v, 0.0f}; }
__device__ __forceinline__ Node node_of(Node v) { return v; }

// Joins the partial sums part[groups][2][n] of 64 columns of dw (blocks [0,
// ctiles)) or dbias (blocks [ctiles, 2 ctiles)): wave i adds up groups i,
// i + 16, .. in order, then the waves are joined pairwise.  The launch starts
// at block b0.
constexpr int JOIN_WAVES = 16;
template <class P>
__global__ __launch_bounds__(64 * JOIN_WAVES) void k_norm_join(const P *__restrict__ part, int groups, int n, int b0,
                                                               int ctiles, void *__restrict__ dw,
                                                               void *__restrict__ db, int pt) {
  __shared__ Node lds[JOIN_WAVES][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, block = b0 + (int)blockIdx.x;
  const int which = block >= ctiles, j = (block - which * ctiles) * 64 + lane;
  void *out = which ? db : dw;
  if (!out) return;
  Node s = sv::zero_node();
  if (j < n) {
#pragma unroll 8
    for (int q = wave; q < groups; q += JOIN_WAVES) s = sv::combine(s, node_of(part[((int64_t)q * 2 + which) * n + j]));
  }
  lds[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && j < n) {
    Node t[JOIN_WAVES];
#pragma unroll
    for (int i = 0; i < JOIN_WAVES; ++i) t[i] = lds[i][lane];
    svr::store_as(out, j, pt, sv::root_value(sv::node_tree<0, JOIN_WAVES, JOIN_WAVES>(t)));
  }
}

// k_norm_join over all columns, in launches within HIP's limit (the longest
// rows have 2^22 tiles for dw and dbias, 2^32 work-items).
template <class P>
void join_columns(const P *part, int64_t groups, int64_t n, void *dw, void *db, int pt, hipStream_t s) {
  const int64_t ctiles = (n + 63) / 64;
  svh::in_batches(2 * ctiles, 1, 64 * JOIN_WAVES, [&](int64_t b0, int64_t blocks) {
    k_norm_join<P><<<(unsigned)blocks, 64 * JOIN_WAVES, 0, s>>>(part, (int)groups, (int)n, (int)b0, (int)ctiles, dw,
                                                                db, pt);
  });
}

// Workgroups of k_norm_dw_any across a row.
int64_t col_tiles(int dtype, int64_t n) {
  const int64_t values = 64 * (16 / (int64_t)svr::dtype_bytes(dtype));
  return (n + values - 1) / values;
}

// Groups of rows: 64 rows each or more, at most 512 and at most 2^22
// workgroups in all (2^30 work-items, within HIP's grid limit).
int64_t col_groups(int dtype, int64_t rows, int64_t n) {
  const int64_t ctiles = col_tiles(dtype, n);
  int64_t g = (rows + COL_ROWS - 1) / COL_ROWS;
  if (g > COL_MAX_GROUPS) g = COL_MAX_GROUPS;
  if (g > ((int64_t)1 << 22) / ctiles) g = ((int64_t)1 << 22) / ctiles;
  return g < 1 ? 1 : g;
}

// Workgroups of k_norm_grad (0: the rows are too long for it).  Every group
// of a workgroup passes at most GRAD_RUN rows.
int64_t grad_blocks(int dtype, int64_t rows, int64_t n) {
  int64_t blocks = 0;
  svr::with_type(dtype, [&](auto t) {
    with_tile<decltype(t), true>(n, [&](auto tl, auto tk, auto) {
      constexpr int L = decltype(tl)::value, E = decltype(tk)::value * svr::Chunk<decltype(t)>::VE;
      constexpr int64_t R = grad_tpb(L, E, svr::Chunk<decltype(t)>::VE) / L;
      const int64_t all = (rows + R - 1) / R;
      const int64_t rounds = (all + GRAD_RUN * GRAD_BLOCKS - 1) / (GRAD_RUN * GRAD_BLOCKS);
      blocks = all < GRAD_BLOCKS ? all : rounds * GRAD_BLOCKS;  // whole rounds of the chip
      if (blocks < 1) blocks = 1;
    });
  });
  return blocks;
}

// Checks that the two calls share; SV_OK without touching the message.
sv_status check_rows(const char *who, int dtype, int64_t rows, int64_t n, int param_dtype) {
  if (!svr::dtype_bytes(dtype)) return fail(SV_ERR_INVALID_ARGUMENT, "%s: dtype %d is not a type code", who, dtype);
  if (param_dtype != dtype && param_dtype != SV_DTYPE_F32)
    return fail(SV_ERR_INVALID_ARGUMENT, "%s: param_dtype %d must be the rows' type or SV_DTYPE_F32", who,
                param_dtype);
  if (rows < 0 || n < 0)
    return fail(SV_ERR_INVALID_ARGUMENT, "%s: rows = %lld, n = %lld must be >= 0", who, (long long)rows,
                (long long)n);
  if (n > svr::MAX_N) return fail(SV_ERR_UNSUPPORTED, "%s: rows of %lld values exceed 2^27", who, (long long)n);
  if (n > 0 && rows > svr::MAX_VALUES / n)
    return fail(SV_ERR_UNSUPPORTED, "%s: %lld x %lld values exceed 2^36", who, (long long)rows, (long long)n);
  if (rows > svr::MAX_VALUES)
    return fail(SV_ERR_UNSUPPORTED, "%s: %lld rows exceed 2^36", who, (long long)rows);
  return SV_OK;
}

unsigned row_grid(int64_t rows) { return (unsigned)(rows < ROW_GRID ? rows : ROW_GRID); }

}  // namespace

extern "C" {

sv_status sv_layer_norm(const void *x, int dtype, int64_t rows, int64_t n, int64_t ldx, const void *weight,
                        const void *bias, int param_dtype, double eps, void *y, int64_t ldy, float *mean, float *rstd,
                        void *stream) {
  static const char who[] = "sv_layer_norm";
  sv_status st = check_rows(who, dtype, rows, n, param_dtype);
  if (st != SV_OK) return st;
  if (!(eps >= 0.0) || eps > 3.0e38) return fail(SV_ERR_INVALID_ARGUMENT, "%s: eps must be >= 0 and finite", who);
  const size_t e = svr::dtype_bytes(dtype);
  if ((st = svr::check_matrix(who, "x", x, ldx, rows, n, e)) != SV_OK) return st;
  if ((st = svr::check_matrix(who, "y", y, ldy, rows, n, e)) != SV_OK) return st;
  const size_t pe = svr::dtype_bytes(param_dtype);
  if (weight && (st = svr::check_matrix(who, "weight", weight, n, 1, n, pe)) != SV_OK) return st;
  if (bias && (st = svr::check_matrix(who, "bias", bias, n, 1, n, pe)) != SV_OK) return st;
  if (rows == 0) return ok();
  if ((st = check_device()) != SV_OK) return st;
  (void)hipGetLastError();
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  svr::with_type(dtype, [&](auto t) {
    using T = decltype(t);
    const bool held = with_tile<T, false>(n, [&](auto tl, auto tk, auto tf) {
      constexpr int L = decltype(tl)::value, K = decltype(tk)::value, TPB = tpb(L), R = TPB / L;
      const int64_t blocks = (rows + R - 1) / R, most = 256 * (2048 / TPB);
      k_norm_rows<T, L, K, decltype(tf)::value><<<(unsigned)(blocks < most ? blocks : most), TPB, 0, s>>>(
          (const T *)x, rows, (int)n, ldx, weight, bias, param_dtype, eps, (T *)y, ldy, mean, rstd);
    });
    if (held) return;
    k_norm_any<T><<<row_grid(rows), ROW_THREADS, 0, s>>>((const T *)x, rows, (int)n, ldx, weight, bias, param_dtype,
                                                         eps, (T *)y, ldy, mean, rstd);
  });
  return check_launch(who);
}

size_t sv_layer_norm_backward_workspace_size(int64_t rows, int64_t n, int dtype) {
  if (!svr::dtype_bytes(dtype) || rows < 0 || n < 0 || n > svr::MAX_N || rows > svr::MAX_VALUES ||
      (n > 0 && rows > svr::MAX_VALUES / n))
    return (size_t)-1;
  if (n == 0) return 0;
  const int64_t blocks = grad_blocks(dtype, rows, n);
  if (blocks) return svr::round256((size_t)blocks * 2 * (size_t)n * sizeof(float));
  return svr::round256((size_t)rows * 4) + (size_t)col_groups(dtype, rows, n) * 2 * (size_t)n * sizeof(Node);
}

sv_status sv_layer_norm_backward(const void *dy, int64_t lddy, const void *x, int64_t ldx, int dtype, int64_t rows,
                                 int64_t n, const void *weight, int param_dtype, const float *mean, const float *rstd,
                                 void *dx, int64_t lddx, void *dweight, void *dbias, void *workspace,
                                 size_t workspace_bytes, void *stream) {
  static const char who[] = "sv_layer_norm_backward";
  sv_status st = check_rows(who, dtype, rows, n, param_dtype);
  if (st != SV_OK) return st;
  const size_t e = svr::dtype_bytes(dtype);
  if ((st = svr::check_matrix(who, "dy", dy, lddy, rows, n, e)) != SV_OK) return st;
  if ((st = svr::check_matrix(who, "x", x, ldx, rows, n, e)) != SV_OK) return st;
  const size_t pe = svr::dtype_bytes(param_dtype);
  if (weight && (st = svr::check_matrix(who, "weight", weight, n, 1, n, pe)) != SV_OK) return st;
  if (dweight && (st = svr::check_matrix(who, "dweight", dweight, n, 1, n, pe)) != SV_OK) return st;
  if (dbias && (st = svr::check_matrix(who, "dbias", dbias, n, 1, n, pe)) != SV_OK) return st;
  if (dx && (st = svr::check_matrix(who, "dx", dx, lddx, rows, n, e)) != SV_OK) return st;
  if (rows > 0 && n > 0 && (!mean || !rstd))
    return fail(SV_ERR_INVALID_ARGUMENT, "%s: mean or rstd is NULL", who);
  if (n == 0 || (!dx && !dweight && !dbias)) return ok();
  const bool cols = dweight || dbias;
  if (!cols && rows == 0) return ok();
  const size_t need = sv_layer_norm_backward_workspace_size(rows, n, dtype);
  if (cols) {
    if (!workspace) return fail(SV_ERR_WORKSPACE, "%s: workspace is NULL (%zu bytes needed)", who, need);
    if (workspace_bytes < need)
      return fail(SV_ERR_WORKSPACE, "%s: workspace has %zu bytes, %zu needed", who, workspace_bytes, need);
    if (!svh::aligned256(workspace)) return fail(SV_ERR_WORKSPACE, "%s: workspace is not 256-byte aligned", who);
  }
  if ((st = check_device()) != SV_OK) return st;
  (void)hipGetLastError();
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const int64_t blocks = grad_blocks(dtype, rows, n);
  if (blocks) {
    float *part = cols ? reinterpret_cast<float *>(workspace) : nullptr;
    if (rows > 0)
      svr::with_type(dtype, [&](auto t) {
        using T = decltype(t);
        with_tile<T, true>(n, [&](auto tl, auto tk, auto tf) {
          constexpr int L = decltype(tl)::value, K = decltype(tk)::value, VE = svr::Chunk<T>::VE;
          k_norm_grad<T, L, K, decltype(tf)::value><<<(unsigned)blocks, grad_tpb(L, K * VE, VE), 0, s>>>(
              (const T *)dy, lddy, (const T *)x, ldx, rows, (int)n, weight, param_dtype, mean, rstd, (T *)dx, lddx,
              part);
        });
      });
    if (cols) join_columns(part, rows > 0 ? blocks : 0, n, dweight, dbias, param_dtype, s);
    return check_launch(who);
  }
  float *off = cols ? reinterpret_cast<float *>(workspace) : nullptr;
  Node *part = cols ? reinterpret_cast<Node *>((char *)workspace + svr::round256((size_t)rows * 4)) : nullptr;
  const int groups = (int)col_groups(dtype, rows, n), wtiles = (int)col_tiles(dtype, n);
  svr::with_type(dtype, [&](auto t) {
    using T = decltype(t);
    const T *g = (const T *)dy, *xx = (const T *)x;
    if (rows > 0)
      k_norm_dx_any<T><<<row_grid(rows), ROW_THREADS, 0, s>>>(g, lddy, xx, ldx, rows, (int)n, weight, param_dtype,
                                                              mean, rstd, (T *)dx, lddx, off);
    if (cols)
      k_norm_dw_any<T><<<(unsigned)(groups * wtiles), 64 * COL_WAVES, 0, s>>>(g, lddy, xx, ldx, rows, (int)n, mean,
                                                                              rstd, off, groups, wtiles, part);
  });
  if (cols) join_columns(part, groups, n, dweight, dbias, param_dtype, s);
  return check_launch(who);
}

}  // extern "C"
