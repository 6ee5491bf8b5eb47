// Device helpers of the root-mean-square norm and of the gradients' norm:
// sums in double and maxima across threads, chunks of a fixed number of
// values whatever their type, and 8-bit outputs.
#pragma once

#include "sv_rows.hpp"

namespace svm {

using svr::bf16;
using svr::f16;

// ---------------------------------------------------------------- across threads

template <int CTRL>
__device__ __forceinline__ unsigned dpp_bits(unsigned v) {
  return (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}

template <int CTRL>
__device__ __forceinline__ double dpp_double(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)dpp_bits<CTRL>((unsigned)b) |
                                        (uint64_t)dpp_bits<CTRL>((unsigned)(b >> 32)) << 32);
}

// v of this lane and of the lane XOR away, in either order.
template <int XOR>
__device__ __forceinline__ void swap_bits(unsigned v, unsigned &a, unsigned &b) {
  float x, y;
  sv::swap_halves<XOR>(__builtin_bit_cast(float, v), x, y);
  a = __builtin_bit_cast(unsigned, x);
  b = __builtin_bit_cast(unsigned, y);
}

template <int XOR>
__device__ __forceinline__ double swap_add(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  unsigned l0, l1, h0, h1;
  swap_bits<XOR>((unsigned)b, l0, l1);
  swap_bits<XOR>((unsigned)(b >> 32), h0, h1);
  return __builtin_bit_cast(double, (uint64_t)l0 | (uint64_t)h0 << 32) +
         __builtin_bit_cast(double, (uint64_t)l1 | (uint64_t)h1 << 32);
}

// Sum over each aligned group of S lanes (a power of two up to 64), pairwise;
// every lane of the group gets it.
template <int S>
__device__ __forceinline__ double seg_add(double v) {
  if constexpr (S >= 2) v += dpp_double<sv::DPP_QUAD_XOR1>(v);
  if constexpr (S >= 4) v += dpp_double<sv::DPP_QUAD_XOR2>(v);
  if constexpr (S >= 8) v += dpp_double<sv::DPP_ROW_HALF_MIRROR>(v);
  if constexpr (S >= 16) v += dpp_double<sv::DPP_ROW_MIRROR>(v);
  if constexpr (S >= 32) v = swap_add<16>(v);
  if constexpr (S >= 64) v = swap_add<32>(v);
  return v;
}

__device__ __forceinline__ unsigned umax(unsigned a, unsigned b) { return a > b ? a : b; }

template <int S>
__device__ __forceinline__ unsigned seg_max(unsigned v) {
  if constexpr (S >= 2) v = umax(v, dpp_bits<sv::DPP_QUAD_XOR1>(v));
  if constexpr (S >= 4) v = umax(v, dpp_bits<sv::DPP_QUAD_XOR2>(v));
  if constexpr (S >= 8) v = umax(v, dpp_bits<sv::DPP_ROW_HALF_MIRROR>(v));
  if constexpr (S >= 16) v = umax(v, dpp_bits<sv::DPP_ROW_MIRROR>(v));
  if constexpr (S >= 32) {
    unsigned a, b;
    swap_bits<16>(v, a, b);
    v = umax(a, b);
  }
  if constexpr (S >= 64) {
    unsigned a, b;
    swap_bits<32>(v, a, b);
    v = umax(a, b);
  }
  return v;
}

// The same over each group of L consecutive threads (a power of two up to
// 1024).  L > 64 takes a barrier and `lds` (a value per wave of the
// workgroup); the next use of the same `lds` must lie behind another barrier.
template <int L>
__device__ __forceinline__ double group_add(double v, double *lds) {
  v = seg_add<(L < 64 ? L : 64)>(v);
  if constexpr (L > 64) {
    constexpr int W = L / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) lds[wave] = v;
    __syncthreads();
    const double *g = lds + wave / W * W;
    double t[W];
#pragma unroll
    for (int j = 0; j < W; ++j) t[j] = g[j];
    v = svr::pair_sum<0, W>([&](int j) { return t[j]; });
  }
  return v;
}

template <int L>
__device__ __forceinline__ unsigned group_max(unsigned v, unsigned *lds) {
  v = seg_max<(L < 64 ? L : 64)>(v);
  if constexpr (L > 64) {
    constexpr int W = L / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) lds[wave] = v;
    __syncthreads();
    const unsigned *g = lds + wave / W * W;
#pragma unroll
    for (int j = 0; j < W; ++j) v = umax(v, g[j]);
  }
  return v;
}

// ---------------------------------------------------------------- values

// The exact square of a float32 value: 48 bits, and in double neither beyond
// the range nor below it.
__device__ __forceinline__ double square(float v) { return (double)v * (double)v; }

// |v| as bits, whose order as whole numbers is the values' with NaN above
// Inf: a maximum over them keeps a NaN, as float's own maximum does not.
__device__ __forceinline__ unsigned abs_bits(float v) { return __builtin_bit_cast(unsigned, v) & 0x7fffffffu; }

// VE values of type T from p on as float32, of which `count` are there (the
// others are 0 and not read).  Without TAIL all are there or none.
template <class T, int VE, bool TAIL = true>
__device__ __forceinline__ void get(const T *p, int count, float (&f)[VE]) {
  typedef T Vec __attribute__((ext_vector_type(VE)));
  if (count >= VE) {
    Vec v;
    __builtin_memcpy(&v, p, sizeof(Vec));
#pragma unroll
    for (int i = 0; i < VE; ++i) f[i] = svr::to_f<T>(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < VE; ++i) f[i] = TAIL && i < count ? svr::to_f<T>(p[i]) : 0.0f;
  }
}

// `count` of VE float32 values to p, rounded to T.
template <class T, int VE>
__device__ __forceinline__ void put(T *p, int count, const float (&f)[VE]) {
  typedef T Vec __attribute__((ext_vector_type(VE)));
  Vec v;
#pragma unroll
  for (int i = 0; i < VE; ++i) v[i] = svr::from_f<T>(f[i]);
  if (count >= VE) {
    __builtin_memcpy(p, &v, sizeof(Vec));
  } else {
#pragma unroll
    for (int i = 0; i < VE; ++i)
      if (i < count) p[i] = v[i];
  }
}

// VE values of a parameter vector beside rows of T, whose type (T or float32)
// is a launch argument, `count` of them there; 1 for p == nullptr.
template <class T, int VE, bool TAIL = true>
__device__ __forceinline__ void get_weight(const void *p, int dtype, int64_t at, int count, float (&f)[VE]) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < VE; ++i) f[i] = 1.0f;
  } else if (sizeof(T) == 2 && dtype != SV_DTYPE_F32) {
    get<T, VE, TAIL>(reinterpret_cast<const T *>(p) + at, count, f);
  } else {
    get<float, VE, TAIL>(reinterpret_cast<const float *>(p) + at, count, f);
  }
}

// ---------------------------------------------------------------- 8 bits

// The largest finite value of an 8-bit type.
__device__ __forceinline__ float fp8_largest(bool e5m2) { return e5m2 ? 57344.0f : 448.0f; }

// The scale of values whose largest magnitude has the bits `most`: 2^-126 (a
// normal number, whose reciprocal is finite) at least, so that zeros divide
// nothing by nothing; Inf and NaN stay.
__device__ __forceinline__ float fp8_scale(unsigned most, bool e5m2) {
  const float s = __builtin_bit_cast(float, most) / fp8_largest(e5m2);
  return s < 0x1p-126f ? 0x1p-126f : s;
}

// Two values of 8 bits in the low half of a word, from float32 values (round
// to nearest even).  The product with the scale's reciprocal passes the
// largest value by 2^-22 of it at most, which still rounds to it: the next step
// would begin at 464 of 448, or 61440 of 57344.
__device__ __forceinline__ unsigned fp8_pair(float a, float b, bool e5m2) {
  return (unsigned)(e5m2 ? __builtin_amdgcn_cvt_pk_bf8_f32(a, b, 0, false)
                         : __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false)) & 0xffffu;
}

// `count` of VE values f * inv (inv: the scale's reciprocal) to p.
template <int VE, bool TAIL = true>
__device__ __forceinline__ void put_fp8(uint8_t *p, int count, const float (&f)[VE], float inv, bool e5m2) {
  unsigned w[VE / 4];
#pragma unroll
  for (int i = 0; i < VE; i += 4)
    w[i / 4] = fp8_pair(f[i] * inv, f[i + 1] * inv, e5m2) | fp8_pair(f[i + 2] * inv, f[i + 3] * inv, e5m2) << 16;
  if (!TAIL || count >= VE) {
    __builtin_memcpy(p, w, VE);
  } else {
#pragma unroll
    for (int i = 0; i < VE; ++i)
      if (i < count) p[i] = (uint8_t)(w[i / 4] >> i % 4 * 8);
  }
}

// ---------------------------------------------------------------- calls

constexpr int ROW_THREADS = 512;
constexpr int64_t ROW_GRID = 8192;  // workgroups of a row launch, at most
constexpr int BLOCK = 128;          // values that share a scale
constexpr int64_t LAST_LEVEL = (int64_t)256 << 20;  // bytes of the last-level cache

// Values of one chunk of threads that hold T and S side by side: 16 bytes of
// the wider type.
template <class T, class S>
constexpr int chunk_values() { return 16 / (int)(sizeof(T) > sizeof(S) ? sizeof(T) : sizeof(S)); }

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

// Calls fn(T{}, S{}) with the element types of x and of the residual stream
// (T, or float32).
template <class Fn>
inline void with_types(int dtype, int sum_dtype, Fn &&fn) {
  svr::with_type(dtype, [&](auto t) {
    using T = decltype(t);
    if (sizeof(T) == 4 || sum_dtype == dtype) fn(t, t);
    else fn(t, float{});
  });
}

// Checks that the calls share; SV_OK without touching the message.
inline sv_status check_rows(const char *who, int dtype, int sum_dtype, int64_t rows, int64_t n, int param_dtype) {
  if (!svr::dtype_bytes(dtype))
    return svh::fail(SV_ERR_INVALID_ARGUMENT, "%s: dtype %d is not a type code", who, dtype);
  if (sum_dtype != dtype && sum_dtype != SV_DTYPE_F32)
    return svh::fail(SV_ERR_INVALID_ARGUMENT, "%s: sum_dtype %d must be dtype or SV_DTYPE_F32", who, sum_dtype);
  if (param_dtype != dtype && param_dtype != SV_DTYPE_F32)
    return svh::fail(SV_ERR_INVALID_ARGUMENT, "%s: param_dtype %d must be the rows' type or SV_DTYPE_F32", who,
                param_dtype);
  if (rows < 0 || n < 0)
    return svh::fail(SV_ERR_INVALID_ARGUMENT, "%s: rows = %lld, n = %lld must be >= 0", who, (long long)rows,
                (long long)n);
  if (n > svr::MAX_N) return svh::fail(SV_ERR_UNSUPPORTED, "%s: rows of %lld values exceed 2^27", who, (long long)n);
  if (n > 0 && rows > svr::MAX_VALUES / n)
    return svh::fail(SV_ERR_UNSUPPORTED, "%s: %lld x %lld values exceed 2^36", who, (long long)rows, (long long)n);
  if (rows > svr::MAX_VALUES) return svh::fail(SV_ERR_UNSUPPORTED, "%s: %lld rows exceed 2^36", who, (long long)rows);
  return SV_OK;
}

// Checks of the forward calls.
inline sv_status check_forward(const char *who, const void *x, int64_t ldx, const void *residual, int64_t ldr,
                               int dtype, int sum_dtype, int64_t rows, int64_t n, const void *weight, int param_dtype,
                               double eps, const void *sum, int64_t ldsum) {
  sv_status st = check_rows(who, dtype, sum_dtype, rows, n, param_dtype);
  if (st != SV_OK) return st;
  if (!(eps >= 0.0) || eps > 3.0e38) return svh::fail(SV_ERR_INVALID_ARGUMENT, "%s: eps must be >= 0 and finite", who);
  const size_t e = svr::dtype_bytes(dtype), se = svr::dtype_bytes(sum_dtype);
  if ((st = svr::check_matrix(who, "x", x, ldx, rows, n, e)) != SV_OK) return st;
  if (residual || sum) {
    if ((st = svr::check_matrix(who, "residual", residual, ldr, rows, n, se)) != SV_OK) return st;
    if ((st = svr::check_matrix(who, "sum", sum, ldsum, rows, n, se)) != SV_OK) return st;
  } else if (sum_dtype != dtype && rows > 0 && n > 0) {  // an empty residual may be NULL
    return svh::fail(SV_ERR_INVALID_ARGUMENT, "%s: sum_dtype %d without a residual must be dtype", who, sum_dtype);
  }
  if (weight && (st = svr::check_matrix(who, "weight", weight, n, 1, n, svr::dtype_bytes(param_dtype))) != SV_OK)
    return st;
  return SV_OK;
}

inline unsigned row_grid(int64_t rows) { return (unsigned)(rows < ROW_GRID ? rows : ROW_GRID); }

}  // namespace svm
