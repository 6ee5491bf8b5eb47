// The root-mean-square norm's forward kernels and their launch, for the
// output in the rows' type (sv_rms.hip) and in 8 bits (sv_rms_fp8.hip).
#pragma once

#include "sv_rms.hpp"

namespace {

using svm::BLOCK;
using svm::Out8;
using svm::ROW_THREADS;
using svm::Rows;

// Rows of any length: a workgroup per row, each pass reads the row again (from
// the cache where it fits).  2000 x 40000 bf16 89 us, 3.6 TB/s of what is read
// and written once (float32 184 us, to 8 bits 83), where 2000 x 32768 held in
// registers take 59.
template <class T, class S, bool RES, bool Q>
__global__ __launch_bounds__(ROW_THREADS) void k_rms_any(const T *x, int64_t ldx, const S *res, int64_t ldr, Rows a,
                                                         T *y, int64_t ldy, S *h, int64_t ldh, Out8 o) {
  constexpr int VE = svm::chunk_values<T, S>(), STEP = ROW_THREADS * VE;
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
      svm::get_weight<T, VE>(a.w, a.pt, e, count, w);
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

// ---------------------------------------------------------------- rows in registers

// Threads of a workgroup whose groups of L threads hold a row each.
constexpr int tpb(int L) { return L <= 128 ? 256 : L; }

// Rows that a group of L threads holds in registers, K chunks per thread: x
// (and the residual) is read once, and the group's R - 1 neighbours in the
// workgroup hold other rows.  The next row's loads are in flight while a row
// is summed (waited for before this row's stores, so that no store is ever
// waited for), and up to 24 values' weights stay in registers across rows.
// One sum of squares in double across the group's threads per row.
// What is read next, y or q, is stored as it comes, so that the last-level
// cache (256 MB) can serve its reader.  The sum h, which is read only behind
// the next products, is stored non-temporal, and inputs that are no smaller
// than the cache (STREAM), of which it holds little, are loaded so.  Measured
// between a kernel that writes x and one that reads y, with h read after 256
// MB of other stores, n = 4096 bf16, all of it in us, with h stored plainly,
// then non-temporal, then the loads so too: 4096 rows 96.7, 96.1, 98.7; 16384
// rows (256 MB in) 241, 236, 229; 32768 rows 443, 434, 398.  With h read as well,
// plain loads and others: 8192 rows 172 and 174, 12288 rows 230 and 231, 16384
// rows 299 and 299 (the kernel by itself 99 and 86).
// Bound by the read and the write: 16384 x 8192 bf16 with a residual to 8 bits
// 147 us, 6.4 TB/s, 200000 x 128 bf16 17.6 us, 5.8 TB/s (a copy in torch runs
// at 4.9-5.4).  Short of that, few rows: 5003 x 1531 f16 to 8 bits 9.8 us, 2.3
// TB/s, where every wave has one row, whose loads, sums and stores follow each
// other; one row of 4096 takes 2.8 us.
template <class T, class S, bool RES, bool Q, bool STREAM, int L, int K, int FIT>
__global__ __launch_bounds__(tpb(L)) void k_rms_rows(const T *__restrict__ x, int64_t ldx, const S *__restrict__ res,
                                                     int64_t ldr, Rows a, T *__restrict__ y, int64_t ldy,
                                                     S *__restrict__ h, int64_t ldh, Out8 o) {
  constexpr int VE = svm::chunk_values<T, S>(), E = K * VE, TPB = tpb(L), R = TPB / L;
  constexpr bool HOLD = E <= 24, TAIL = FIT != svr::FIT_CHUNKS;
  using TX = svr::RowTile<T, L, K, FIT, VE>;
  using TS = svr::RowTile<S, L, K, FIT, VE>;
  __shared__ double lds_sum[2][TPB / 64];
  __shared__ unsigned lds_max[TPB / 64];
  const int64_t rows = a.rows;
  const int n = a.n, g = svr::group_of<L>(), l0 = threadIdx.x % L;
  const double inv_n = 1.0 / (double)n;
  float wv[HOLD ? K : 1][VE];
  const auto weight = [&](int l, int k, float(&w)[VE]) {
    const int e = TX::first(l, k), left = n - e;
    svm::get_weight<T, VE, TAIL>(a.w, a.pt, e, left < 0 ? 0 : left, w);
  };
  const int64_t step = (int64_t)gridDim.x * R;
  typename TX::Vec rx[K];
  typename TS::Vec rr[RES ? K : 1];
  int64_t r = (int64_t)blockIdx.x * R + g;
  int64_t rl = R == 1 || r < rows ? r : rows - 1;  // the row that is loaded
  const auto load = [&](int l) {
    TX::template load<STREAM>(x + rl * ldx, n, TX::avail(rows, rl, ldx, n), l, rx);
    if constexpr (RES) TS::template load<STREAM>(res + rl * ldr, n, TS::avail(rows, rl, ldr, n), l, rr);
  };
  const auto arrived = [&] {
    TX::arrived(rx);
    if constexpr (RES) TS::arrived(rr);
  };
  load(l0);
  if constexpr (HOLD) {
#pragma unroll
    for (int k = 0; k < K; ++k) weight(l0, k, wv[k]);  // in flight beside the first row
    arrived();
  }
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * R; r0 < rows; r0 += step, r += step, turn ^= 1) {
    int l = l0;  // opaque, so that the addresses of all chunks are not kept in registers across rows
    asm volatile("" : "+v"(l));
    float f[E];
    TX::unpack(rx, f);
    TX::load_rest(x + rl * ldx, n, TX::avail(rows, rl, ldx, n), l, f);
    if constexpr (RES) {
      float b[E];
      TS::unpack(rr, b);
      TS::load_rest(res + rl * ldr, n, TS::avail(rows, rl, ldr, n), l, b);
#pragma unroll
      for (int i = 0; i < E; ++i) f[i] = svr::to_f(svr::from_f<S>(f[i] + b[i]));
    }
    rl = r + step < rows ? r + step : rows - 1;
    if constexpr (HOLD) load(l);
    TX::set_rest(n, l, 0.0f, f);
    double c[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      c[k] = svr::pair_sum<0, VE>([&](int i) { return svm::square(f[k * VE + i]); });
      if (!TX::inside(n, l, k)) c[k] = 0.0;
    }
    const double s = svm::group_add<L>(svr::pair_sum<0, K>([&](int k) { return c[k]; }), lds_sum[turn]);
    const float rs = svr::rstd_of(s * inv_n + a.eps);
    const bool own = R == 1 || r < rows;
    if (own && l == 0 && a.rstd) a.rstd[r] = rs;
    if constexpr (HOLD) arrived();
    if constexpr (RES) {
      if (own) {
#pragma unroll
        for (int k = 0; k < K; ++k) TS::template store_chunk<true>(h + r * ldh, n, l, k, f);
      }
    }
    const auto scale_chunk = [&](int k) {
      float wk[VE];
      if constexpr (!HOLD) weight(l, k, wk);
#pragma unroll
      for (int i = 0; i < VE; ++i) f[k * VE + i] = (f[k * VE + i] * rs) * (HOLD ? wv[HOLD ? k : 0][i] : wk[i]);
    };
    if constexpr (!Q) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        scale_chunk(k);
        if (own) TX::store_chunk(y + r * ldy, n, l, k, f);
        if constexpr (!HOLD) __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      constexpr int LANES = BLOCK / VE;  // lanes that hold a block
      static_assert(L >= LANES, "a block lies in one chunk of neighbouring lanes");
      const auto largest = [&](int k) {
        unsigned m = 0;
#pragma unroll
        for (int i = 0; i < VE; ++i) m = svm::umax(m, svm::abs_bits(f[k * VE + i]));
        return TX::inside(n, l, k) ? m : 0u;
      };
      const auto store = [&](int k, float inv) {
        const int e = TX::first(l, k), left = n - e;
        float v[VE];
#pragma unroll
        for (int i = 0; i < VE; ++i) v[i] = f[k * VE + i];
        if (own && left > 0) svm::put_fp8<VE, TAIL>(o.q + r * o.ldq + e, left, v, inv, o.e5m2);
      };
#pragma unroll
      for (int k = 0; k < K; ++k) scale_chunk(k);
      if (o.per_row) {
        unsigned m = 0;
#pragma unroll
        for (int k = 0; k < K; ++k) m = svm::umax(m, largest(k));
        const float scale = svm::fp8_scale(svm::group_max<L>(m, lds_max), o.e5m2);
        const float inv = 1.0f / scale;
        if (own && l == 0) o.scale[r] = scale;
#pragma unroll
        for (int k = 0; k < K; ++k) store(k, inv);
      } else {
        const int blocks = (int)(((unsigned)n + BLOCK - 1) / BLOCK);
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const float scale = svm::fp8_scale(svm::seg_max<LANES>(largest(k)), o.e5m2);
          const int e = TX::first(l, k);
          if (own && l % LANES == 0 && e < n) o.scale[r * blocks + e / BLOCK] = scale;
          store(k, 1.0f / scale);
        }
      }
    }
    if constexpr (!HOLD) load(l);
  }
}

// Calls fn(L, K, FIT) (integral constants) with the smallest tile of VE-value
// chunks and at least MIN threads that holds n values; false when none does.
// The choice follows from n and the types alone.
template <int VE, int MIN, class Fn>
bool with_tile(int64_t n, Fn &&fn) {
  if (n < 1) return false;
  const auto tile = [&](auto tl, auto tk, bool &small) {
    constexpr int L = decltype(tl)::value, K = decltype(tk)::value;
    if constexpr (L >= MIN) {
      if constexpr (L == MIN) {
        if (small && n < VE) {
          fn(tl, tk, std::integral_constant<int, svr::FIT_SMALL>{});
          return true;
        }
        small = false;  // the first tile of MIN threads only
      }
      if (n > (int64_t)L * K * VE || n < VE) return false;
      if (n % VE == 0) fn(tl, tk, std::integral_constant<int, svr::FIT_CHUNKS>{});
      else fn(tl, tk, std::integral_constant<int, svr::FIT_ANY>{});
      return true;
    }
    return false;
  };
  bool small = true;
#define SV_TILE(L, V) \
  if (tile(std::integral_constant<int, L>{}, std::integral_constant<int, (V) / VE>{}, small)) return true;
  // Up to 64 values: 8 per thread, so that a row's lanes read whole cache
  // lines together; then 16 (half the cost per value of the cross-lane sums),
  // or 24 where that leaves fewer threads idle; 32 for the longest rows.
  SV_TILE(1, 8) SV_TILE(4, 8) SV_TILE(8, 8) SV_TILE(8, 16)
  if constexpr (MIN == 16) SV_TILE(16, 8)  // the shortest rows where a block takes 16 or 32 threads
  if constexpr (MIN == 32) SV_TILE(32, 8)
  SV_TILE(16, 16) SV_TILE(32, 16) SV_TILE(64, 16) SV_TILE(64, 24)
  SV_TILE(128, 16) SV_TILE(256, 16) SV_TILE(256, 24) SV_TILE(512, 16) SV_TILE(512, 24)
  SV_TILE(1024, 16) SV_TILE(1024, 32)
#undef SV_TILE
  return false;
}

// The launch of a forward call: with (Q) the output in 8 bits.
template <bool Q>
void forward(const void *x, int64_t ldx, const void *residual, int64_t ldr, int dtype, int sum_dtype, const Rows &a,
             void *y, int64_t ldy, void *sum, int64_t ldsum, const Out8 &o, hipStream_t s) {
  const auto launch = [&](auto t, auto u, auto with_residual) {
    using T = decltype(t);
    using S = decltype(u);
    constexpr bool RES = decltype(with_residual)::value;
    constexpr int VE = svm::chunk_values<T, S>();
    const bool stream = a.rows * a.n * (int64_t)(sizeof(T) + (RES ? sizeof(S) : 0)) >= svm::LAST_LEVEL;
    const bool held = with_tile<VE, Q ? BLOCK / VE : 1>(a.n, [&](auto tl, auto tk, auto tf) {
      constexpr int L = decltype(tl)::value, K = decltype(tk)::value, FIT = decltype(tf)::value, TPB = tpb(L);
      constexpr int R = TPB / L;
      const int64_t blocks = (a.rows + R - 1) / R, most = 256 * (2048 / TPB);
      const unsigned grid = (unsigned)(blocks < most ? blocks : most);
      const auto rows = [&](auto st) {
        k_rms_rows<T, S, RES, Q, decltype(st)::value, L, K, FIT><<<grid, TPB, 0, s>>>(
            (const T *)x, ldx, (const S *)residual, ldr, a, (T *)y, ldy, (S *)sum, ldsum, o);
      };
      // longer rows of whole chunks only, as every kernel is there once more for
      // it.  Shorter ones gain nothing: 2000000 x 128 bf16 (512 MB) by itself 203
      // us with plain loads and 201 so, between a writer and a reader 588 and 599;
      // 270000 x 1000 221 and 230.  Rows that end inside a chunk were not timed.
      if constexpr (FIT == svr::FIT_CHUNKS && L >= 128) {
        if (stream) return rows(std::true_type{});
      }
      rows(std::false_type{});
    });
    if (!held)
      k_rms_any<T, S, RES, Q><<<svm::row_grid(a.rows), ROW_THREADS, 0, s>>>((const T *)x, ldx, (const S *)residual, ldr,
                                                                           a, (T *)y, ldy, (S *)sum, ldsum, o);
  };
  svm::with_types(dtype, sum_dtype, [&](auto t, auto u) {
    if (residual) launch(t, u, std::true_type{});
    else launch(t, t, std::false_type{});
  });
}

}  // namespace
