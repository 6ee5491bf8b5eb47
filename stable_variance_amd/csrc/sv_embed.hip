// Embedding lookup with scaling, and the gradient of its table by sorted
// tokens, on gfx950.
//
// Lookup:    out[t] = scale * table[id[t]], one rounding.
// Gradient:  grad[v] = scale * sum over the tokens t with id[t] = v of dy[t],
// in token order, as a compensated sum (TwoSum, the errors in a carry), and
// zero for a row that no token names.
//
// The gradient sorts the tokens by id first (stable, so that equal ids stay
// in token order): a least-significant-digit radix sort of (id, token) pairs.
// Every row is then written once, by whoever sums it, and nothing is added
// with atomics: the bits do not depend on scheduling.
//
// An id outside [0, vocab) gives a row of NaN in the lookup and takes no part
// in the gradient; neither do the tokens of the padding id.  Such tokens sort
// behind all others under the key `vocab`.
#include "sv_rows.hpp"

using svh::check_device;
using svh::check_launch;
using svh::fail;
using svh::ok;
using svr::Node;

namespace {

constexpr int64_t MAX_TOKENS = (int64_t)1 << 30;
constexpr int64_t MAX_VOCAB = ((int64_t)1 << 31) - 2;  // the key `vocab` fits 31 bits

// ---------------------------------------------------------------- lookup

// A workgroup per token.
template <class T>
__global__ __launch_bounds__(256) void k_emb_lookup(const void *__restrict__ ids, int id_bytes, int64_t tokens,
                                                    const T *__restrict__ table, int64_t vocab, int64_t dim,
                                                    int64_t ldt, float scale, T *__restrict__ out, int64_t ldo) {
  for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
    const int64_t id = id_bytes == 8 ? reinterpret_cast<const int64_t *>(ids)[t]
                                     : (int64_t) reinterpret_cast<const int32_t *>(ids)[t];
    T *o = out + t * ldo;
    if (id < 0 || id >= vocab) {
      for (int64_t i = threadIdx.x; i < dim; i += 256) o[i] = svr::from_f<T>(__builtin_nanf(""));
    } else {
      const T *r = table + id * ldt;
      for (int64_t i = threadIdx.x; i < dim; i += 256) o[i] = svr::from_f<T>(svr::to_f(r[i]) * scale);
    }
  }
}

// ---------------------------------------------------------------- sort

// Up to 64 workgroups of 1024 threads, each owning one run of `span` tokens
// (a multiple of 1024).  A digit of `bits` <= 9 bits takes two launches: the
// workgroups' histograms, then the scatter, where each workgroup finds its
// digits' places from all histograms.
constexpr int SORT_THREADS = 1024;
constexpr int SORT_WAVES = SORT_THREADS / 64;
constexpr int SORT_MAX_BLOCKS = 64;
constexpr int SORT_MAX_BITS = 9;
constexpr int SORT_RADIX = 1 << SORT_MAX_BITS;

struct SortPlan {
  int passes, bits, blocks;
  int64_t span;
};

SortPlan sort_plan(int64_t tokens, int64_t vocab) {
  SortPlan p;
  int kb = 1;
  while (kb < 31 && ((int64_t)1 << kb) <= vocab) ++kb;  // keys 0 .. vocab
  p.passes = (kb + SORT_MAX_BITS - 1) / SORT_MAX_BITS;
  p.bits = (kb + p.passes - 1) / p.passes;
  const int64_t tiles = (tokens + SORT_THREADS - 1) / SORT_THREADS;
  const int64_t per = (tiles + SORT_MAX_BLOCKS - 1) / SORT_MAX_BLOCKS;
  p.span = per * SORT_THREADS;
  p.blocks = (int)((tokens + p.span - 1) / p.span);
  return p;
}

__device__ __forceinline__ unsigned key_of(const void *ids, int id_bytes, int64_t t, int64_t vocab, int64_t padding) {
  const int64_t id = id_bytes == 8 ? reinterpret_cast<const int64_t *>(ids)[t]
                                   : (int64_t) reinterpret_cast<const int32_t *>(ids)[t];
  return id < 0 || id >= vocab || id == padding ? (unsigned)vocab : (unsigned)id;
}

// hist[block * radix + digit].  The first pass (keys == nullptr) reads ids.
__global__ __launch_bounds__(SORT_THREADS) void k_sort_hist(const void *__restrict__ ids, int id_bytes,
                                                            const unsigned *__restrict__ keys, int64_t tokens,
                                                            int64_t vocab, int64_t padding, int64_t span, int shift,
                                                            int bits, unsigned *__restrict__ hist) {
  __shared__ unsigned h[SORT_RADIX];
  const int radix = 1 << bits;
  if ((int)threadIdx.x < radix) h[threadIdx.x] = 0;
  __syncthreads();
  const int64_t t0 = blockIdx.x * span, t1 = t0 + span < tokens ? t0 + span : tokens;
  for (int64_t t = t0 + threadIdx.x; t < t1; t += SORT_THREADS) {
    const unsigned k = keys ? keys[t] : key_of(ids, id_bytes, t, vocab, padding);
    atomicAdd(&h[(k >> shift) & (radix - 1)], 1u);
  }
  __syncthreads();
  if ((int)threadIdx.x < radix) hist[blockIdx.x * radix + threadIdx.x] = h[threadIdx.x];
}

__global__ __launch_bounds__(SORT_THREADS) void k_sort_scatter(
    const void *__restrict__ ids, int id_bytes, const unsigned *__restrict__ keys, const int *__restrict__ tok,
    int64_t tokens, int64_t vocab, int64_t padding, int64_t span, int shift, int bits,
    const unsigned *__restrict__ hist, unsigned *__restrict__ keys_out, int *__restrict__ tok_out) {
  __shared__ unsigned base[SORT_RADIX];
  __shared__ unsigned count[SORT_WAVES][SORT_RADIX];
  __shared__ unsigned wave_sum[SORT_WAVES];
  const int radix = 1 << bits, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // place of this workgroup's first token of digit tid: the digits below it
  // in all workgroups, then the same digit in the workgroups before
  unsigned total = 0, before = 0;
  if (tid < radix)
    for (int b = 0; b < (int)gridDim.x; ++b) {
      if (b == (int)blockIdx.x) before = total;
      total += hist[b * radix + tid];
    }
  unsigned scan = total;  // inclusive scan over the wave, then over waves
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const unsigned v = __shfl_up(scan, s, 64);
    if (lane >= s) scan += v;
  }
  if (lane == 63) wave_sum[wave] = scan;
  __syncthreads();
  unsigned below = 0;
  for (int i = 0; i < wave; ++i) below += wave_sum[i];
  if (tid < radix) base[tid] = below + scan - total + before;

  const int64_t t0 = blockIdx.x * span, t1 = t0 + span < tokens ? t0 + span : tokens;
  for (int64_t tile = t0; tile < t1; tile += SORT_THREADS) {
    for (int i = tid; i < SORT_WAVES * radix; i += SORT_THREADS) count[i / radix][i % radix] = 0;
    __syncthreads();
    const int64_t t = tile + tid;
    const bool in = t < t1;
    const unsigned k = !in ? 0u : keys ? keys[t] : key_of(ids, id_bytes, t, vocab, padding);
    const unsigned d = (k >> shift) & (radix - 1);
    // lanes of this wave that hold the same digit
    unsigned long long same = __ballot(in);
    for (int b = 0; b < bits; ++b) {
      const bool bit = (d >> b) & 1;
      const unsigned long long m = __ballot(bit);
      same &= bit ? m : ~m;
    }
    const unsigned rank = __popcll(same & ((1ull << lane) - 1));
    if (in && rank == 0) count[wave][d] = __popcll(same);
    __syncthreads();
    if (tid < radix) {  // the waves' places within the tile
      unsigned p = base[tid];
#pragma unroll
      for (int w = 0; w < SORT_WAVES; ++w) {
        const unsigned c = count[w][tid];
        count[w][tid] = p;
        p += c;
      }
      base[tid] = p;
    }
    __syncthreads();
    if (in) {
      const unsigned p = count[wave][d] + rank;
      keys_out[p] = k;
      tok_out[p] = tok ? tok[t] : (int)t;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- gradient

// First place of the sorted keys that is not below `key`.
__device__ __forceinline__ int lower_bound(const unsigned *__restrict__ keys, int n, unsigned key) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = lo + ((hi - lo) >> 1);
    if (keys[mid] < key) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// A workgroup per table row.
template <class T>
__global__ __launch_bounds__(256) void k_emb_grad(const T *__restrict__ dy, int64_t lddy,
                                                  const unsigned *__restrict__ keys, const int *__restrict__ tok,
                                                  int tokens, int64_t vocab, int64_t dim, float scale,
                                                  T *__restrict__ grad, int64_t ldg) {
  __shared__ int ends[2];
  for (int64_t v = blockIdx.x; v < vocab; v += gridDim.x) {
    __syncthreads();
    if (threadIdx.x < 2) ends[threadIdx.x] = lower_bound(keys, tokens, (unsigned)v + threadIdx.x);
    __syncthreads();
    const int lo = ends[0], hi = ends[1];
    for (int64_t i = threadIdx.x; i < dim; i += 256) {
      Node s = sv::zero_node();
      for (int j = lo; j < hi; ++j) svr::add_to(s, svr::to_f(dy[(int64_t)tok[j] * lddy + i]));
      grad[v * ldg + i] = svr::from_f<T>(sv::root_value(s) * scale);
    }
  }
}

// ---------------------------------------------------------------- checks

sv_status check_shape(const char *who, int id_bytes, int64_t tokens, int dtype, int64_t vocab, int64_t dim) {
  if (!svr::dtype_bytes(dtype)) return fail(SV_ERR_INVALID_ARGUMENT, "%s: dtype %d is not a type code", who, dtype);
  if (id_bytes != 4 && id_bytes != 8)
    return fail(SV_ERR_INVALID_ARGUMENT, "%s: ids of %d bytes (4 or 8)", who, id_bytes);
  if (tokens < 0 || vocab < 0 || dim < 0)
    return fail(SV_ERR_INVALID_ARGUMENT, "%s: tokens = %lld, vocab = %lld, dim = %lld must be >= 0", who,
                (long long)tokens, (long long)vocab, (long long)dim);
  if (tokens > MAX_TOKENS) return fail(SV_ERR_UNSUPPORTED, "%s: %lld tokens exceed 2^30", who, (long long)tokens);
  if (vocab > MAX_VOCAB) return fail(SV_ERR_UNSUPPORTED, "%s: %lld rows exceed 2^31 - 2", who, (long long)vocab);
  if (dim > svr::MAX_N) return fail(SV_ERR_UNSUPPORTED, "%s: rows of %lld values exceed 2^27", who, (long long)dim);
  if (dim > 0 && (tokens > svr::MAX_VALUES / dim || vocab > svr::MAX_VALUES / dim))
    return fail(SV_ERR_UNSUPPORTED, "%s: %lld values per row exceed 2^36 in all", who, (long long)dim);
  return SV_OK;
}

}  // namespace

extern "C" {

sv_status sv_embedding(const void *ids, int id_bytes, int64_t tokens, const void *table, int dtype, int64_t vocab,
                       int64_t dim, int64_t ldt, float scale, void *out, int64_t ldo, void *stream) {
  static const char who[] = "sv_embedding";
  sv_status st = check_shape(who, id_bytes, tokens, dtype, vocab, dim);
  if (st != SV_OK) return st;
  const size_t e = svr::dtype_bytes(dtype);
  if ((st = svr::check_matrix(who, "ids", ids, 1, tokens, 1, (size_t)id_bytes)) != SV_OK) return st;
  if (tokens > 0 && (st = svr::check_matrix(who, "table", table, ldt, vocab, dim, e)) != SV_OK) return st;
  if ((st = svr::check_matrix(who, "out", out, ldo, tokens, dim, e)) != SV_OK) return st;
  if (tokens == 0 || dim == 0) return ok();
  if ((st = check_device()) != SV_OK) return st;
  (void)hipGetLastError();
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  svr::with_type(dtype, [&](auto t) {
    using T = decltype(t);
    k_emb_lookup<T><<<(unsigned)(tokens < 65536 ? tokens : 65536), 256, 0, s>>>(
        ids, id_bytes, tokens, (const T *)table, vocab, dim, ldt, scale, (T *)out, ldo);
  });
  return check_launch(who);
}

size_t sv_embedding_backward_workspace_size(int64_t tokens, int64_t vocab, int64_t dim, int dtype) {
  if (!svr::dtype_bytes(dtype) || tokens < 0 || vocab < 0 || dim < 0 || tokens > MAX_TOKENS || vocab > MAX_VOCAB ||
      dim > svr::MAX_N || (dim > 0 && (tokens > svr::MAX_VALUES / dim || vocab > svr::MAX_VALUES / dim)))
    return (size_t)-1;
  if (vocab == 0 || dim == 0) return 0;
  return 4 * svr::round256((size_t)tokens * 4) + (size_t)SORT_MAX_BLOCKS * SORT_RADIX * 4;
}

sv_status sv_embedding_backward(const void *dy, int64_t lddy, const void *ids, int id_bytes, int64_t tokens,
                                int dtype, int64_t vocab, int64_t dim, float scale, int64_t padding, void *grad,
                                int64_t ldg, void *workspace, size_t workspace_bytes, void *stream) {
  static const char who[] = "sv_embedding_backward";
  sv_status st = check_shape(who, id_bytes, tokens, dtype, vocab, dim);
  if (st != SV_OK) return st;
  if (padding < -1 || padding >= vocab)
    if (padding != -1)
      return fail(SV_ERR_INVALID_ARGUMENT, "%s: padding id %lld outside [0, %lld) (-1: none)", who,
                  (long long)padding, (long long)vocab);
  const size_t e = svr::dtype_bytes(dtype);
  if ((st = svr::check_matrix(who, "ids", ids, 1, tokens, 1, (size_t)id_bytes)) != SV_OK) return st;
  if ((st = svr::check_matrix(who, "dy", dy, lddy, tokens, dim, e)) != SV_OK) return st;
  if ((st = svr::check_matrix(who, "grad", grad, ldg, vocab, dim, e)) != SV_OK) return st;
  if (vocab == 0 || dim == 0) return ok();
  const size_t need = sv_embedding_backward_workspace_size(tokens, vocab, dim, dtype);
  if (!workspace) return fail(SV_ERR_WORKSPACE, "%s: workspace is NULL (%zu bytes needed)", who, need);
  if (workspace_bytes < need)
    return fail(SV_ERR_WORKSPACE, "%s: workspace has %zu bytes, %zu needed", who, workspace_bytes, need);
  if (!svh::aligned256(workspace)) return fail(SV_ERR_WORKSPACE, "%s: workspace is not 256-byte aligned", who);
  if ((st = check_device()) != SV_OK) return st;
  (void)hipGetLastError();
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const size_t part = svr::round256((size_t)tokens * 4);
  char *w = reinterpret_cast<char *>(workspace);
  unsigned *keys[2] = {(unsigned *)w, (unsigned *)(w + part)};
  int *tok[2] = {(int *)(w + 2 * part), (int *)(w + 3 * part)};
  unsigned *hist = (unsigned *)(w + 4 * part);
  int cur = 0;
  if (tokens > 0) {
    const SortPlan p = sort_plan(tokens, vocab);
    for (int i = 0; i < p.passes; ++i) {
      const unsigned *kin = i ? keys[cur] : nullptr;
      const int *tin = i ? tok[cur] : nullptr;
      k_sort_hist<<<p.blocks, SORT_THREADS, 0, s>>>(ids, id_bytes, kin, tokens, vocab, padding, p.span, i * p.bits,
                                                    p.bits, hist);
      k_sort_scatter<<<p.blocks, SORT_THREADS, 0, s>>>(ids, id_bytes, kin, tin, tokens, vocab, padding, p.span,
                                                       i * p.bits, p.bits, hist, keys[cur ^ 1], tok[cur ^ 1]);
      cur ^= 1;
    }
  }
  svr::with_type(dtype, [&](auto t) {
    using T = decltype(t);
    k_emb_grad<T><<<(unsigned)(vocab < 65536 ? vocab : 65536), 256, 0, s>>>(
        (const T *)dy, lddy, keys[cur], tok[cur], (int)tokens, vocab, dim, scale, (T *)grad, ldg);
  });
  return check_launch(who);
}

}  // extern "C"
