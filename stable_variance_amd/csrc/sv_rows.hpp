// Device and host helpers of the layer norm and the embedding: element types
// of 32 and 16 bits, all computed on in float32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

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
  if constexpr (sizeof(T) == 2) asm("" : "+v"(v));
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

// Calls fn(T{}) with the element type of a valid code.
template <class Fn>
inline void with_type(int dtype, Fn &&fn) {
  if (dtype == SV_DTYPE_F32) fn(float{});
  else if (dtype == SV_DTYPE_BF16) fn(bf16{});
  else fn(f16{});
}

}  // namespace svr
