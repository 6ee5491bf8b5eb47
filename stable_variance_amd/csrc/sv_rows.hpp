// Device and host helpers of the layer norm and the embedding: element types
// of 32 and 16 bits, all computed on in float32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/stable_variance.h"
#include "sv_device.hpp"
#include "sv_host.hpp"

namespace svr {

using sv::Node;
using bf16 = __bf16;
using f16 = _Float16;

// A value as float32 (exact for every type) and back (round to nearest even).
template <class T>
__device__ __forceinline__ float to_f(T v) { return (float)v; }
// The empty asm keeps the compiler from joining a product with its rounding to
// float16 (v_fma_mixlo_f16 rounds once and adds a +0), which it does in some
// of the places that must agree and not in others.
template <class T>
__device__ __forceinline__ T from_f(float v) {
  if constexpr (std::is_same_v<T, f16>) asm("" : "+v"(v));
  return (T)v;
}

// Element i of an array whose type is a launch argument (parameters).
__device__ __forceinline__ float load_as(const void *p, int64_t i, int dtype) {
  if (dtype == SV_DTYPE_BF16) return to_f(reinterpret_cast<const bf16 *>(p)[i]);
  if (dtype == SV_DTYPE_F16) return to_f(reinterpret_cast<const f16 *>(p)[i]);
  return reinterpret_cast<const float *>(p)[i];
}

__device__ __forceinline__ void store_as(void *p, int64_t i, int dtype, float v) {
  if (dtype == SV_DTYPE_BF16) reinterpret_cast<bf16 *>(p)[i] = from_f<bf16>(v);
  else if (dtype == SV_DTYPE_F16) reinterpret_cast<f16 *>(p)[i] = from_f<f16>(v);
  else reinterpret_cast<float *>(p)[i] = v;
}

// ---------------------------------------------------------------- 16-byte chunks

// VE values in one 16-byte load or store.  The address needs the alignment
// of T only: global memory takes 16-byte accesses at any address.
template <class T>
struct Chunk {
  static constexpr int VE = 16 / (int)sizeof(T);
  typedef T Vec __attribute__((ext_vector_type(VE)));
};

template <bool NT, class T, class Vec>
__device__ __forceinline__ void store_chunk_at(T *p, Vec v) {
  if constexpr (NT) {
    typedef Vec Unaligned __attribute__((aligned(sizeof(T))));
    __builtin_nontemporal_store(v, reinterpret_cast<Unaligned *>(p));
  } else {
    __builtin_memcpy(p, &v, sizeof(Vec));
  }
}

// fn(e, f, count) for the chunks of a row of n values that thread `tid` of
// `threads` passes: `count` values (VE but for the row's last chunk) from e
// on, as float32; f may be changed and is passed on to nothing else.
template <class T, class Fn>
__device__ __forceinline__ void for_chunks(const T *__restrict__ p, int n, int tid, int threads, Fn &&fn) {
  constexpr int VE = Chunk<T>::VE;
  for (int e = tid * VE; e < n; e += threads * VE) {
    float f[VE];
    const int count = n - e < VE ? n - e : VE;
    if (count == VE) {
      typename Chunk<T>::Vec v;
      __builtin_memcpy(&v, p + e, 16);
#pragma unroll
      for (int i = 0; i < VE; ++i) f[i] = to_f<T>(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < VE; ++i) f[i] = i < count ? to_f<T>(p[e + i]) : 0.0f;
    }
    fn(e, f, count);
  }
}

// The chunk back: `count` values of f at p + e.
template <class T>
__device__ __forceinline__ void put_chunk(T *__restrict__ p, int e, int count, const float *f) {
  constexpr int VE = Chunk<T>::VE;
  typename Chunk<T>::Vec v;
#pragma unroll
  for (int i = 0; i < VE; ++i) v[i] = from_f<T>(f[i]);
  if (count == VE) {
    __builtin_memcpy(p + e, &v, 16);
  } else {
#pragma unroll
    for (int i = 0; i < VE - 1; ++i)
      if (i < count) p[e + i] = v[i];
  }
}

// 1 / sqrt(v) in double (one Newton step from the hardware's estimate, about
// 2^-46), so that the float32 value is the rounded one; 0, Inf and NaN as
// the estimate gives them.  Above float32's range (a variance or mean square
// of 0 and eps below 8.6e-78) it is the largest finite value: with Inf, zeros
// would give 0 * Inf = NaN in place of 0, and NaN gradients.
__device__ __forceinline__ float rstd_of(double v) {
  const double r = __builtin_amdgcn_rsq(v);
  const double e = 1.0 - v * r * r;
  const double s = r + 0.5 * r * e;
  const float f = (float)(__builtin_isfinite(e) ? s : r);
  return v > 0.0 && f > __FLT_MAX__ ? __FLT_MAX__ : f;
}

// Pairwise sum of N values fn(OFF), fn(OFF + 1), .. (adjacent pairs at each
// level), of fn's type.
template <int OFF, int N, class Fn>
__device__ __forceinline__ auto pair_sum(Fn &&fn) {
  if constexpr (N == 1) return fn(OFF);
  else return pair_sum<OFF, (N + 1) / 2>(fn) + pair_sum<OFF + (N + 1) / 2, N / 2>(fn);
}

// A row of n values held by L threads, K chunks each: thread l's chunk k
// starts at value (k * L + l) * VE.  A chunk is 16 bytes, or has the number of
// values of a wider type that is held beside T.  FIT says what is known of n:
//   FIT_FULL    n == K * L * VE: every chunk is whole
//   FIT_CHUNKS  n is a multiple of VE: a chunk is whole or outside
//   FIT_ANY     the row's last chunk may be part of one
//   FIT_SMALL   n < VE: one thread holds the row and loads value by value
enum Fit { FIT_FULL = 0, FIT_CHUNKS = 1, FIT_ANY = 2, FIT_SMALL = 3 };

template <class T, int L, int K, int FIT, int VALUES = Chunk<T>::VE>
struct RowTile {
  static constexpr int VE = VALUES, E = K * VE;
  typedef T Vec __attribute__((ext_vector_type(VALUES)));

  __device__ static __forceinline__ int first(int l, int k) { return (k * L + l) * VE; }
  // Chunk k holds values of the row.
  __device__ static __forceinline__ bool inside(int n, int l, int k) { return FIT == FIT_FULL || first(l, k) < n; }

  // Values that may be read from the start of row r on: the rest of the
  // matrix, at least n, cut at 2^24.
  __device__ static __forceinline__ int avail(int64_t rows, int64_t r, int64_t ld, int n) {
    if constexpr (FIT == FIT_SMALL) return 0;
    if constexpr (FIT != FIT_ANY) return n;
    const int64_t a = (rows - 1 - r) * ld + n;
    return a < (1 << 24) ? (int)a : (1 << 24);
  }

  // Starts the loads of the row; values past n hold anything.  The row's last
  // chunk may reach into the next row; where there is none, and for chunks
  // outside the row, the row's first chunk is loaded instead (load_rest brings
  // what is missing).  So every thread loads K chunks on every path
  // and the compiler can leave later loads in flight when it waits for these:
  // a load under a condition makes it wait for all.  NT: non-temporal.
  template <bool NT = false>
  __device__ static __forceinline__ void load(const T *__restrict__ p, int n, int avail, int l, Vec (&raw)[K]) {
    if constexpr (FIT == FIT_SMALL) return;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      int e = first(l, k);
      if (FIT != FIT_FULL) {
        const bool ok = FIT == FIT_ANY ? e < n && e + VE <= avail : e < n;
        e = ok ? e : 0;  // avail >= n >= VE
      }
      if constexpr (NT) {
        typedef Vec Unaligned __attribute__((aligned(sizeof(T))));
        raw[k] = __builtin_nontemporal_load(reinterpret_cast<const Unaligned *>(p + e));
      } else {
        __builtin_memcpy(&raw[k], p + e, sizeof(Vec));
      }
    }
  }

  // Waits for the loads here, so that the stores that follow are not waited
  // for as well where the values are first used.
  __device__ static __forceinline__ void arrived(Vec (&raw)[K]) {
    typedef unsigned Bits __attribute__((ext_vector_type(sizeof(Vec) / 4)));
#pragma unroll
    for (int k = 0; k < K; ++k) {
      Bits u = __builtin_bit_cast(Bits, raw[k]);
      asm volatile("" : "+v"(u));
      raw[k] = __builtin_bit_cast(Vec, u);
    }
  }
  template <class S>
  __device__ static __forceinline__ void arrived(Vec (&raw)[K], S &one) {
    arrived(raw);
    using Bits = std::conditional_t<sizeof(S) == 2, unsigned short, unsigned>;
    unsigned b = __builtin_bit_cast(Bits, one);
    asm volatile("" : "+v"(b));
    one = __builtin_bit_cast(S, (Bits)b);
  }

  // The values of the last chunks that load left out.
  __device__ static __forceinline__ void load_rest(const T *__restrict__ p, int n, int avail, int l, float (&f)[E]) {
    if constexpr (FIT == FIT_ANY || FIT == FIT_SMALL) {
      if (((n + VE - 1) & -VE) <= avail) return;  // the same for all lanes of a row
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int e = first(l, k);
        if (e < n && e + VE > avail) {
#pragma unroll
          for (int i = 0; i < VE - 1; ++i)
            if (e + i < n) f[k * VE + i] = to_f<T>(p[e + i]);
        }
      }
    }
  }

  __device__ static __forceinline__ void unpack(const Vec (&raw)[K], float (&f)[E]) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < VE; ++i) f[k * VE + i] = to_f<T>(raw[k][i]);
  }

  // Sets what lies past n in a chunk that the row ends in.  Only the waves
  // that hold such a chunk spend time on it.
  __device__ static __forceinline__ void set_rest(int n, int l, float v, float (&f)[E]) {
    if constexpr (FIT == FIT_ANY || FIT == FIT_SMALL) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int left = n - first(l, k);
        if (left > 0 && left < VE) {
#pragma unroll
          for (int i = 1; i < VE; ++i) f[k * VE + i] = i < left ? f[k * VE + i] : v;
        }
      }
    }
  }

  // Pairwise sum of fn(value index) over the thread's values inside the row.
  template <class Fn>
  __device__ static __forceinline__ float sum(int n, int l, Fn &&fn) {
    float c[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      c[k] = pair_sum<0, VE>([&](int i) { return fn(k * VE + i); });
      if (!inside(n, l, k)) c[k] = 0.0f;
    }
    return pair_sum<0, K>([&](int k) { return c[k]; });
  }

  // Chunk k of the row's values f.  NT: non-temporal.
  template <bool NT = false>
  __device__ static __forceinline__ void store_chunk(T *__restrict__ p, int n, int l, int k, const float (&f)[E]) {
    if (!inside(n, l, k)) return;
    const int e = first(l, k);
    Vec v;
#pragma unroll
    for (int i = 0; i < VE; ++i) v[i] = from_f<T>(f[k * VE + i]);
    if (FIT == FIT_FULL || FIT == FIT_CHUNKS || e + VE <= n) {
      store_chunk_at<NT>(p + e, v);
    } else {
      // 4, 2 and 1 of the values that are left, as their number's bits say
      const int left = n - e;
      typedef T V4 __attribute__((ext_vector_type(4)));
      typedef T V2 __attribute__((ext_vector_type(2)));
      V4 q = {v[0], v[1], v[2], v[3]};
      T *at = p + e;
      if constexpr (VE == 8) {
        if (left & 4) {
          __builtin_memcpy(at, &q, 4 * sizeof(T));
          at += 4;
          q = V4{v[4], v[5], v[6], v[7]};
        }
      }
      V2 d = {q[0], q[1]};
      if (left & 2) {
        __builtin_memcpy(at, &d, 2 * sizeof(T));
        at += 2;
        d = V2{q[2], q[3]};
      }
      if (left & 1) at[0] = d[0];
    }
  }
};

// Chunk k of thread l of a parameter vector whose type is a launch argument:
// VE values from e = (k * L + l) * VE on, `none` past n and for p == nullptr.
template <class T, int L>
__device__ __forceinline__ void load_param(const void *__restrict__ p, int dtype, int n, int l, int k, float none,
                                           float *__restrict__ out) {
  constexpr int VE = Chunk<T>::VE;
  const int e = (k * L + l) * VE;
#pragma unroll
  for (int i = 0; i < VE; ++i) out[i] = none;
  if (!p) return;
  if (e + VE <= n) {
    if (sizeof(T) == 2 && dtype != SV_DTYPE_F32) {
      typename Chunk<T>::Vec v;
      __builtin_memcpy(&v, reinterpret_cast<const T *>(p) + e, 16);
#pragma unroll
      for (int i = 0; i < VE; ++i) out[i] = to_f<T>(v[i]);
    } else {
      float v[VE];
      __builtin_memcpy(v, reinterpret_cast<const float *>(p) + e, 4 * VE);
#pragma unroll
      for (int i = 0; i < VE; ++i) out[i] = v[i];
    }
  } else if (e < n) {
#pragma unroll
    for (int i = 0; i < VE - 1; ++i)
      if (e + i < n) out[i] = load_as(p, e + i, dtype);
  }
}

// The group of L threads that this thread belongs to, in a scalar register
// where a group is whole waves (and the row's addresses with it).
template <int L>
__device__ __forceinline__ int group_of() {
  const int g = threadIdx.x / L;
  return L >= 64 ? __builtin_amdgcn_readfirstlane(g) : g;
}

// Sums of NV values per thread over each group of L consecutive threads, in
// a fixed order (lanes pairwise, then the group's waves pairwise); every
// thread of the group gets them.  L > 64 takes a barrier and `lds`, which
// holds NV floats per wave of the workgroup; the next use of the same `lds`
// must lie behind another barrier.
template <int L, int NV>
__device__ __forceinline__ void group_sum(float (&v)[NV], float *lds) {
#pragma unroll
  for (int i = 0; i < NV; ++i)
    v[i] = sv::seg_tree<sv::NODE_PLAIN, (L < 64 ? L : 64)>(Node{v[i], 0.0f}).s;
  if constexpr (L > 64) {
    constexpr int W = L / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) lds[wave * NV + i] = v[i];
    }
    __syncthreads();
    const float *g = lds + wave / W * W * NV;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float t[W];
#pragma unroll
      for (int j = 0; j < W; ++j) t[j] = g[j * NV + i];
      v[i] = pair_sum<0, W>([&](int j) { return t[j]; });
    }
  }
}

// One more value for a compensated sum: TwoSum, the error added to the carry.
__device__ __forceinline__ void add_to(Node &a, float v) { a = sv::combine(a, {v, 0.0f}); }

// Host: bytes of an element type, 0 for a code that is none.
inline size_t dtype_bytes(int dtype) {
  return dtype == SV_DTYPE_F32 ? 4 : dtype == SV_DTYPE_BF16 || dtype == SV_DTYPE_F16 ? 2 : 0;
}
inline size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }

// Largest row length of the row operators (as a row of the axis-1 variance)
// and largest number of values of a matrix.
constexpr int64_t MAX_N = (int64_t)1 << 27;
constexpr int64_t MAX_VALUES = (int64_t)1 << 36;

// A matrix argument of [rows, n] values: present, aligned to its type, the
// row stride `ld` at least n and the last value within 2^40 of the first.
// SV_OK without touching the message, and for an empty matrix.
inline sv_status check_matrix(const char *who, const char *name, const void *p, int64_t ld, int64_t rows, int64_t n,
                              size_t bytes) {
  if (rows == 0 || n == 0) return SV_OK;
  if (!p) return svh::fail(SV_ERR_INVALID_ARGUMENT, "%s: %s is NULL", who, name);
  if (reinterpret_cast<uintptr_t>(p) % bytes)
    return svh::fail(SV_ERR_INVALID_ARGUMENT, "%s: %s is not aligned to its type", who, name);
  if (ld < n)
    return svh::fail(SV_ERR_INVALID_ARGUMENT, "%s: row stride %lld of %s is below its row length %lld", who,
                     (long long)ld, name, (long long)n);
  if (ld > ((int64_t)1 << 40) / rows)
    return svh::fail(SV_ERR_UNSUPPORTED, "%s: row stride %lld of %s is too large", who, (long long)ld, name);
  return SV_OK;
}

// A row statistic (one float32 for each row, or NULL): aligned to its type, as
// a wave that holds one row reads it through the scalar unit, which ignores an
// address's lowest two bits.
inline sv_status check_stats(const char *who, const char *name, const float *p, int64_t rows) {
  if (rows > 0 && reinterpret_cast<uintptr_t>(p) % sizeof(float))
    return svh::fail(SV_ERR_INVALID_ARGUMENT, "%s: %s is not aligned to its type", who, name);
  return SV_OK;
}

// Calls fn(T{}) with the element type of a valid code.
template <class Fn>
inline void with_type(int dtype, Fn &&fn) {
  if (dtype == SV_DTYPE_F32) fn(float{});
  else if (dtype == SV_DTYPE_BF16) fn(bf16{});
  else fn(f16{});
}

}  // namespace svr
