// The norm of many tensors as one vector, and their scaling down to a largest
// norm, on gfx950.
//
//   N = sqrt(sum of g^2 over every value of every tensor)
//   k = min(1, max_norm / (N + 1e-6)),   out = g * float32(k)  rounded once
//
// Squares and sums are held in double: the square of a float32 is exact
// there, so no gradient is too large or too small for the sum, and N is good
// to about 2^-45 before it is rounded to float32.  An Inf among the values
// gives N = Inf and k = 0, a NaN gives NaN for both.  Without a limit (max_norm
// = Inf) k is 1 for every N but NaN: Inf / Inf would make it NaN.
//
// The tensors' addresses and sizes travel in the launch's arguments, up to
// TABLE tensors a launch, so that nothing is copied to the device.  Every
// tensor is cut into units of 16 KB or fewer; a workgroup takes a run of
// units, finds its first tensor by bisection and walks on from there.  Its
// sum goes to `part`, and a last workgroup adds those up in order: the same
// bits on every run, no atomics.
#include <algorithm>
#include <stdlib.h>

#include "sv_rms.hpp"

using svh::check_device;
using svh::check_launch;
using svh::fail;
using svh::ok;

namespace {

constexpr int TABLE = 128;         // tensors of one launch (the arguments stay below 4 KB)
constexpr int THREADS = 256;
constexpr int UNIT_BYTES = 16384;  // four chunks of 16 bytes per thread
constexpr int64_t SUM_GRID = 4096;           // workgroups of a sum, at most
constexpr int64_t SCALE_GRID = 1 << 22;      // of a scaling (2^30 work-items)
constexpr int64_t MAX_SIZE = (int64_t)1 << 40;
constexpr int64_t MAX_COUNT = (int64_t)1 << 20;

// The tensors of one launch.  Unit u of the launch belongs to tensor i with
// first[i] <= u < first[i + 1].
template <bool OUT>
struct Table {
  const void *p[TABLE];
  void *out[OUT ? TABLE : 1];
  int64_t n[TABLE];
  uint32_t first[TABLE + 1];
  uint8_t type[TABLE];
  int count;
};

static_assert(sizeof(Table<true>) <= 4000, "a launch's arguments stay below 4 KB");

__host__ __device__ constexpr int64_t unit_values(int dtype) { return UNIT_BYTES / (dtype == SV_DTYPE_F32 ? 4 : 2); }

// Calls fn(i, lo, hi) for the runs of values [lo, hi) of tensor i that make up
// units [u0, u1) of the table.
template <bool OUT, class Fn>
__device__ __forceinline__ void for_runs(const Table<OUT> &t, int64_t u0, int64_t u1, Fn &&fn) {
  int a = 0, b = t.count;  // first[a] <= u0 < first[b]
  while (b - a > 1) {
    const int m = (a + b) >> 1;
    if ((int64_t)t.first[m] <= u0) a = m;
    else b = m;
  }
  for (int64_t u = u0; u < u1; ++a) {
    const int64_t f = t.first[a], end = t.first[a + 1], stop = end < u1 ? end : u1;
    const int64_t unit = unit_values(t.type[a]), lo = (u - f) * unit, hi = (stop - f) * unit;
    fn(a, lo, hi < t.n[a] ? hi : t.n[a]);
    u = stop;
  }
}

// Chunks that a thread has in flight: a unit is one batch of the workgroup.
constexpr int BATCH = UNIT_BYTES / (THREADS * 16);

template <bool NT, class T>
__device__ __forceinline__ typename svr::Chunk<T>::Vec load_chunk(const T *p) {
  typename svr::Chunk<T>::Vec v;
  if constexpr (NT) {
    typedef typename svr::Chunk<T>::Vec Unaligned __attribute__((aligned(sizeof(T))));
    v = __builtin_nontemporal_load(reinterpret_cast<const Unaligned *>(p));
  } else {
    __builtin_memcpy(&v, p, 16);
  }
  return v;
}

template <bool NT, class T>
__device__ __forceinline__ double sum_squares(const T *p, int64_t n) {
  constexpr int VE = svr::Chunk<T>::VE;
  using Vec = typename svr::Chunk<T>::Vec;
  constexpr int64_t STEP = THREADS * VE;
  const T *q = p + threadIdx.x * VE;
  double s[BATCH];
#pragma unroll
  for (int k = 0; k < BATCH; ++k) s[k] = 0.0;
  int64_t e = 0;
  for (; e + BATCH * STEP <= n; e += BATCH * STEP) {
    Vec v[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) v[k] = load_chunk<NT>(q + e + k * STEP);
#pragma unroll
    for (int k = 0; k < BATCH; ++k)
      s[k] += svr::pair_sum<0, VE>([&](int i) { return svm::square(svr::to_f<T>(v[k][i])); });
  }
  for (e += threadIdx.x * VE; e < n; e += STEP) {
    float f[VE];
    svm::get<T, VE>(p + e, (int)(n - e < VE ? n - e : VE), f);
    s[0] += svr::pair_sum<0, VE>([&](int i) { return svm::square(f[i]); });
  }
  return svr::pair_sum<0, BATCH>([&](int k) { return s[k]; });
}

// The sum of squares of each workgroup's units.  AGAIN: the values are read
// again soon (clipping), so the loads leave what the caches hold of them; else
// they are non-temporal.  Eight waves per SIMD (64 registers) with four chunks
// a thread in flight; bound by the read.  1.74 GB of bf16: 257 us, 6.8 TB/s
// (plain loads 293 us, 96 registers 269, one chunk in flight 290); a plain read
// of them takes 247.  Clipping float32 to other buffers, all of it in us, with
// plain loads and with others: 100 MB 53 and 54, 256 MB 123 and 125, 512 MB 243
// and 244, 1.34 GB 632 and 634: the sum alone is slower with plain ones (241
// against 196 at 1.34 GB), and the scaling gets it back.  In place with k = 1,
// where nothing is read again, plain ones lose: 111 and 99 at 512 MB, 273 and 244
// at 1.34 GB.
template <bool AGAIN>
__global__ __launch_bounds__(THREADS, 8) void k_gnorm_sum(Table<false> t, int64_t units, int64_t per, double *part) {
  __shared__ double lds[THREADS / 64];
  const int64_t u0 = blockIdx.x * per, u1 = u0 + per < units ? u0 + per : units;
  double s = 0.0;
  for_runs(t, u0, u1, [&](int i, int64_t lo, int64_t hi) {
    const int type = t.type[i];
    if (type == SV_DTYPE_F32) s += sum_squares<!AGAIN>((const float *)t.p[i] + lo, hi - lo);
    else if (type == SV_DTYPE_BF16) s += sum_squares<!AGAIN>((const svr::bf16 *)t.p[i] + lo, hi - lo);
    else s += sum_squares<!AGAIN>((const svr::f16 *)t.p[i] + lo, hi - lo);
  });
  s = svm::group_add<THREADS>(s, lds);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// The square root of v >= 0 in double by v / sqrt(v), about 2^-45; 0, Inf and
// NaN as they are.
__device__ __forceinline__ double root(double v) {
  if (!(v > 0.0) || !__builtin_isfinite(v)) return v;
  const double r = __builtin_amdgcn_rsq(v);
  const double e = 1.0 - v * r * r;
  return v * (r + 0.5 * r * e);
}

constexpr int JOIN_THREADS = 1024;
// Adds up `count` partial sums; norm, and (max_norm >= 0) the factor k.
__global__ __launch_bounds__(JOIN_THREADS) void k_gnorm_join(const double *part, int64_t count, double max_norm,
                                                             float *norm, float *factor) {
  __shared__ double lds[JOIN_THREADS / 64];
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < count; i += JOIN_THREADS) s += part[i];
  const double v = root(svm::group_add<JOIN_THREADS>(s, lds));
  if (threadIdx.x == 0) {
    *norm = (float)v;
    if (factor) {
      const double k = __builtin_isinf(max_norm) && v == v ? 1.0 : max_norm / (v + 1e-6);
      *factor = k >= 1.0 ? 1.0f : (float)k;  // a NaN stays
    }
  }
}

template <class T>
__device__ __forceinline__ void scale_values(const T *p, T *out, int64_t n, float k) {
  constexpr int VE = svr::Chunk<T>::VE;
  constexpr int64_t STEP = THREADS * VE;
  const T *q = p + threadIdx.x * VE;
  T *o = out + threadIdx.x * VE;
  int64_t e = 0;
  for (; e + BATCH * STEP <= n; e += BATCH * STEP) {
    typename svr::Chunk<T>::Vec v[BATCH];
#pragma unroll
    for (int b = 0; b < BATCH; ++b) v[b] = load_chunk<true>(q + e + b * STEP);
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
#pragma unroll
      for (int j = 0; j < VE; ++j) v[b][j] = svr::from_f<T>(svr::to_f<T>(v[b][j]) * k);
      svr::store_chunk_at<true>(o + e + b * STEP, v[b]);
    }
  }
  for (e += threadIdx.x * VE; e < n; e += STEP) {
    const int count = (int)(n - e < VE ? n - e : VE);
    float f[VE];
    svm::get<T, VE>(p + e, count, f);
#pragma unroll
    for (int j = 0; j < VE; ++j) f[j] = f[j] * k;
    svm::put<T, VE>(out + e, count, f);
  }
}

// One unit per workgroup, in the order of memory: 1.34 GB of float32 scaled in
// 404 us, 6.6 TB/s, where 2048 workgroups of 40 units each take 510.  Loads and
// stores non-temporal (plain stores 475 us, plain loads 465).
__global__ __launch_bounds__(THREADS) void k_gnorm_scale(Table<true> t, int64_t units, int64_t per,
                                                         const float *factor) {
  const float k = *factor;
  const int64_t u0 = blockIdx.x * per, u1 = u0 + per < units ? u0 + per : units;
  for_runs(t, u0, u1, [&](int i, int64_t lo, int64_t hi) {
    if (k == 1.0f && t.p[i] == t.out[i]) return;  // in place: nothing changes
    const int type = t.type[i];
    if (type == SV_DTYPE_F32) scale_values((const float *)t.p[i] + lo, (float *)t.out[i] + lo, hi - lo, k);
    else if (type == SV_DTYPE_BF16)
      scale_values((const svr::bf16 *)t.p[i] + lo, (svr::bf16 *)t.out[i] + lo, hi - lo, k);
    else scale_values((const svr::f16 *)t.p[i] + lo, (svr::f16 *)t.out[i] + lo, hi - lo, k);
  });
}

// ---------------------------------------------------------------- host

// Workgroups of a launch of `units` units, and units of each.
struct Plan {
  int64_t units, per, blocks;
};

Plan plan_of(int64_t units, int64_t grid) {
  const int64_t per = (units + grid - 1) / grid;
  return {units, per, per ? (units + per - 1) / per : 0};
}

// Calls fn(table, plan) for each launch over the tensors; empty tensors take
// no part.  Units of a launch stay below 2^31.
template <bool OUT, class Fn>
void for_tables(const void *const *p, void *const *out, const int64_t *sizes, const int *dtypes, int64_t count,
                Fn &&fn) {
  Table<OUT> t;
  int64_t units = 0;
  t.count = 0;
  const auto flush = [&] {
    t.first[t.count] = (uint32_t)units;
    if (t.count) fn(t, plan_of(units, OUT ? SCALE_GRID : SUM_GRID));
    t.count = 0;
    units = 0;
  };
  for (int64_t i = 0; i < count; ++i) {
    if (!sizes[i]) continue;
    const int64_t unit = unit_values(dtypes[i]), more = (sizes[i] + unit - 1) / unit;
    if (t.count == TABLE || units + more >= (int64_t)1 << 31) flush();
    t.p[t.count] = p ? p[i] : nullptr;
    if constexpr (OUT) t.out[t.count] = out[i];
    t.n[t.count] = sizes[i];
    t.type[t.count] = (uint8_t)dtypes[i];
    t.first[t.count++] = (uint32_t)units;
    units += more;
  }
  flush();
}

bool good_sizes(const int64_t *sizes, const int *dtypes, int64_t count) {
  if (count < 0 || count > MAX_COUNT || (count > 0 && (!sizes || !dtypes))) return false;
  for (int64_t i = 0; i < count; ++i)
    if (!svr::dtype_bytes(dtypes[i]) || sizes[i] < 0 || sizes[i] > MAX_SIZE) return false;
  return true;
}

int64_t partials(const int64_t *sizes, const int *dtypes, int64_t count) {
  int64_t blocks = 0;
  for_tables<false>(nullptr, nullptr, sizes, dtypes, count,
                    [&](const Table<false> &, const Plan &plan) { blocks += plan.blocks; });
  return blocks;
}

// One stretch of memory; `id` 2i for what tensor i reads, 2i + 1 for what is
// written to it (and, in place, read).
struct Span {
  uintptr_t at, end;
  int64_t id;
};

// Finds memory that is written for one tensor and read or written for another
// (or for itself, but in place): -1 none, else the tensor's number; -2: no
// host memory for the search.
int64_t overlap(const void *const *p, void *const *out, const int64_t *sizes, const int *dtypes, int64_t count) {
  Span *spans = (Span *)malloc(sizeof(Span) * 2 * (size_t)(count > 0 ? count : 1));
  if (!spans) return -2;
  int64_t m = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (!sizes[i]) continue;
    const size_t bytes = (size_t)sizes[i] * svr::dtype_bytes(dtypes[i]);
    const uintptr_t a = reinterpret_cast<uintptr_t>(out[i]), b = reinterpret_cast<uintptr_t>(p[i]);
    spans[m++] = {a, a + bytes, 2 * i + 1};
    if (a != b) spans[m++] = {b, b + bytes, 2 * i};
  }
  const auto before = [](const Span &a, const Span &b) { return a.at < b.at; };
  if (!std::is_sorted(spans, spans + m, before)) std::sort(spans, spans + m, before);
  uintptr_t read = 0, written = 0;  // the ends of what has been passed
  int64_t found = -1;
  for (int64_t i = 0; i < m && found < 0; ++i) {
    const bool writes = spans[i].id & 1;
    if (spans[i].at < written || (writes && spans[i].at < read)) found = spans[i].id >> 1;
    uintptr_t &end = writes ? written : read;
    end = end > spans[i].end ? end : spans[i].end;
  }
  free(spans);
  return found;
}

sv_status check_tensors(const char *who, const void *const *p, const int64_t *sizes, const int *dtypes, int64_t count,
                        const void *norm) {
  if (count < 0) return fail(SV_ERR_INVALID_ARGUMENT, "%s: count = %lld must be >= 0", who, (long long)count);
  if (count > MAX_COUNT) return fail(SV_ERR_UNSUPPORTED, "%s: %lld tensors exceed 2^20", who, (long long)count);
  if (count > 0 && (!p || !sizes || !dtypes))
    return fail(SV_ERR_INVALID_ARGUMENT, "%s: an array of the tensors is NULL", who);
  if (!norm || reinterpret_cast<uintptr_t>(norm) % sizeof(float))
    return fail(SV_ERR_INVALID_ARGUMENT, "%s: norm is NULL or not aligned to its type", who);
  for (int64_t i = 0; i < count; ++i) {
    const size_t bytes = svr::dtype_bytes(dtypes[i]);
    if (!bytes)
      return fail(SV_ERR_INVALID_ARGUMENT, "%s: dtype %d of tensor %lld is not a type code", who, dtypes[i],
                  (long long)i);
    if (sizes[i] < 0)
      return fail(SV_ERR_INVALID_ARGUMENT, "%s: size %lld of tensor %lld must be >= 0", who, (long long)sizes[i],
                  (long long)i);
    if (sizes[i] > MAX_SIZE)
      return fail(SV_ERR_UNSUPPORTED, "%s: %lld values of tensor %lld exceed 2^40", who, (long long)sizes[i],
                  (long long)i);
    if (sizes[i] && (!p[i] || reinterpret_cast<uintptr_t>(p[i]) % bytes))
      return fail(SV_ERR_INVALID_ARGUMENT, "%s: tensor %lld is NULL or not aligned to its type", who, (long long)i);
  }
  return SV_OK;
}

sv_status check_workspace(const char *who, const void *workspace, size_t bytes, size_t need) {
  if (!workspace) return fail(SV_ERR_WORKSPACE, "%s: workspace is NULL (%zu bytes needed)", who, need);
  if (bytes < need) return fail(SV_ERR_WORKSPACE, "%s: workspace has %zu bytes, %zu needed", who, bytes, need);
  if (!svh::aligned256(workspace)) return fail(SV_ERR_WORKSPACE, "%s: workspace is not 256-byte aligned", who);
  return SV_OK;
}

// The launches up to the norm (and the factor); the workspace holds the factor
// and, 256 bytes on, the partial sums.
void launch_norm(const void *const *p, const int64_t *sizes, const int *dtypes, int64_t count, double max_norm,
                 float *norm, float *factor, double *part, hipStream_t s) {
  int64_t at = 0;
  for_tables<false>(p, nullptr, sizes, dtypes, count, [&](const Table<false> &t, const Plan &plan) {
    if (factor) k_gnorm_sum<true><<<(unsigned)plan.blocks, THREADS, 0, s>>>(t, plan.units, plan.per, part + at);
    else k_gnorm_sum<false><<<(unsigned)plan.blocks, THREADS, 0, s>>>(t, plan.units, plan.per, part + at);
    at += plan.blocks;
  });
  k_gnorm_join<<<1, JOIN_THREADS, 0, s>>>(part, at, max_norm, norm, factor);
}

}  // namespace

extern "C" {

size_t sv_grad_norm_workspace_size(const int64_t *sizes, const int *dtypes, int64_t count) {
  if (!good_sizes(sizes, dtypes, count)) return (size_t)-1;
  return 256 + svr::round256((size_t)partials(sizes, dtypes, count) * sizeof(double));
}

sv_status sv_grad_norm(const void *const *tensors, const int64_t *sizes, const int *dtypes, int64_t count, float *norm,
                       void *workspace, size_t workspace_bytes, void *stream) {
  static const char who[] = "sv_grad_norm";
  sv_status st = check_tensors(who, tensors, sizes, dtypes, count, norm);
  if (st != SV_OK) return st;
  st = check_workspace(who, workspace, workspace_bytes, sv_grad_norm_workspace_size(sizes, dtypes, count));
  if (st != SV_OK) return st;
  if ((st = check_device()) != SV_OK) return st;
  (void)hipGetLastError();
  launch_norm(tensors, sizes, dtypes, count, 0.0, norm, nullptr, (double *)((char *)workspace + 256),
              reinterpret_cast<hipStream_t>(stream));
  return check_launch(who);
}

sv_status sv_clip_grad_norm(const void *const *tensors, void *const *out, const int64_t *sizes, const int *dtypes,
                            int64_t count, double max_norm, float *norm, void *workspace, size_t workspace_bytes,
                            void *stream) {
  static const char who[] = "sv_clip_grad_norm";
  sv_status st = check_tensors(who, tensors, sizes, dtypes, count, norm);
  if (st != SV_OK) return st;
  if (!(max_norm >= 0.0)) return fail(SV_ERR_INVALID_ARGUMENT, "%s: max_norm must be >= 0", who);
  if (count > 0 && !out) return fail(SV_ERR_INVALID_ARGUMENT, "%s: out is NULL", who);
  for (int64_t i = 0; i < count; ++i)
    if (sizes[i] && (!out[i] || reinterpret_cast<uintptr_t>(out[i]) % svr::dtype_bytes(dtypes[i])))
      return fail(SV_ERR_INVALID_ARGUMENT, "%s: out %lld is NULL or not aligned to its type", who, (long long)i);
  const int64_t bad = overlap(tensors, out, sizes, dtypes, count);
  if (bad == -2) return fail(SV_ERR_HOST_MEMORY, "%s: no host memory for %lld tensors", who, (long long)count);
  if (bad >= 0)
    return fail(SV_ERR_INVALID_ARGUMENT, "%s: tensor %lld overlaps one that is written", who, (long long)bad);
  st = check_workspace(who, workspace, workspace_bytes, sv_grad_norm_workspace_size(sizes, dtypes, count));
  if (st != SV_OK) return st;
  if ((st = check_device()) != SV_OK) return st;
  (void)hipGetLastError();
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  float *factor = (float *)workspace;
  launch_norm(tensors, sizes, dtypes, count, max_norm, norm, factor, (double *)((char *)workspace + 256), s);
  if ((st = check_launch(who)) != SV_OK) return st;  // no factor was written: nothing is scaled
  for_tables<true>(tensors, out, sizes, dtypes, count, [&](const Table<true> &t, const Plan &plan) {
    k_gnorm_scale<<<(unsigned)plan.blocks, THREADS, 0, s>>>(t, plan.units, plan.per, factor);
  });
  return check_launch(who);
}

}  // extern "C"
