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

// A table row, an output row or a gradient row of `dim` values in chunks of
// VE values (16 bytes; single values for dim < 16 bytes).  The last chunk is
// moved back to end with the row: it then repeats some of the chunk before,
// with the same bits, and no chunk needs a mask.  Chunks need the alignment
// of T only.
template <class T, int VE>
struct Cols {
  typedef T Vec __attribute__((ext_vector_type(VE)));

  __device__ static __forceinline__ int64_t first(int64_t chunk, int64_t dim) {
    const int64_t e = chunk * VE;
    return e + VE <= dim ? e : dim - VE;
  }
  __device__ static __forceinline__ Vec load(const T *p) {
    Vec v;
    __builtin_memcpy(&v, p, sizeof(T) * VE);
    return v;
  }
  // Non-temporal: results that nothing here reads again should not displace
  // the rows that are read more than once.
  __device__ static __forceinline__ void store(T *p, Vec v) {
    typedef Vec Unaligned __attribute__((aligned(sizeof(T))));
    __builtin_nontemporal_store(v, reinterpret_cast<Unaligned *>(p));
  }
};

__device__ __forceinline__ int64_t load_id(const void *__restrict__ ids, int id_bytes, int64_t t) {
  return id_bytes == 8 ? reinterpret_cast<const int64_t *>(ids)[t]
                       : (int64_t) reinterpret_cast<const int32_t *>(ids)[t];
}

constexpr int THREADS = 256;
constexpr int64_t MAX_BLOCKS = (int64_t)1 << 23;  // 2^31 work-items, within HIP's grid limit

// L threads per token and tile of L * U chunks; tile u belongs to token
// u / tiles.  All U loads are in flight together.  Bound by memory: a call for
// 32768 rows of 4096 bf16 out of 64000 takes 72-75 us among others, 4.8-5.0
// TB/s of distinct rows and results (358 MB).  Under the profiler the kernel
// takes 77-79 us and moves 441 MB, 5.6 TB/s: a frequent row is fetched by every
// die's cache.
template <class T, int VE, int L, int U>
__global__ __launch_bounds__(THREADS) void k_emb_lookup(const void *__restrict__ ids, int id_bytes, int64_t units,
                                                        int tiles, const T *__restrict__ table, int64_t vocab,
                                                        int64_t dim, int64_t ldt, float scale, T *__restrict__ out,
                                                        int64_t ldo) {
  using C = Cols<T, VE>;
  const int l = threadIdx.x % L;
  const int64_t chunks = (dim + VE - 1) / VE;
  for (int64_t u = (int64_t)blockIdx.x * (THREADS / L) + threadIdx.x / L; u < units;
       u += (int64_t)gridDim.x * (THREADS / L)) {
    const int64_t t = (unsigned)u / (unsigned)tiles, c0 = (u - t * tiles) * (L * U) + l;
    const int64_t id = load_id(ids, id_bytes, t);
    const bool good = id >= 0 && id < vocab;
    typename C::Vec v[U];
    if (good) {
      const T *r = table + id * ldt;
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (c0 + i * L < chunks) v[i] = C::load(r + C::first(c0 + i * L, dim));
    }
    T *o = out + t * ldo;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      typename C::Vec w;
#pragma unroll
      for (int j = 0; j < VE; ++j)
        w[j] = svr::from_f<T>(good ? svr::to_f<T>(v[i][j]) * scale : __builtin_nanf(""));
      if (c0 + i * L < chunks) C::store(o + C::first(c0 + i * L, dim), w);
    }
  }
}

// Calls fn(VE, L, U) for rows of dim values: the fewest threads that hold a
// row with one chunk each, else tiles of 64 threads with up to MAXE values
// each.
template <class T, int MAXE, class Fn>
void with_cols(int64_t dim, Fn &&fn) {
  constexpr int V = 16 / (int)sizeof(T);
  using std::integral_constant;
  constexpr integral_constant<int, V> v{};
  constexpr integral_constant<int, 1> one{};
  constexpr integral_constant<int, 64> wave{};
  if (dim < V) return fn(one, integral_constant<int, 8>{}, one);
  if (dim <= 8 * V) return fn(v, integral_constant<int, 8>{}, one);
  if (dim <= 16 * V) return fn(v, integral_constant<int, 16>{}, one);
  if (dim <= 32 * V) return fn(v, integral_constant<int, 32>{}, one);
  if constexpr (MAXE >= 4 * V)
    if (dim > 128 * V) return fn(v, wave, integral_constant<int, 4>{});
  if constexpr (MAXE >= 2 * V)
    if (dim > 64 * V) return fn(v, wave, integral_constant<int, 2>{});
  fn(v, wave, one);
}

// ---------------------------------------------------------------- sort

// Bound by latency, not by bytes: 16384 tokens with two digits take 20 us in
// four launches, 65536 with one digit 12 us, up to 1024 tokens 6 us in one.
// Up to 64 workgroups of 1024 threads, each owning one run of `span` tokens
// (a multiple of 1024).  A digit of `bits` <= 10 bits takes two launches: the
// workgroups' histograms, then the scatter, where each workgroup finds its
// digits' places from all histograms.
constexpr int SORT_THREADS = 1024;
constexpr int SORT_WAVES = SORT_THREADS / 64;
constexpr int SORT_MAX_BLOCKS = 64;
constexpr int SORT_MAX_BITS = 10;
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
  const int64_t id = load_id(ids, id_bytes, t);
  return id < 0 || id >= vocab || id == padding ? (unsigned)vocab : (unsigned)id;
}

// Lanes of this wave with the same digit among those with `in` set.
__device__ __forceinline__ unsigned long long same_digit(unsigned d, int bits, bool in) {
  unsigned long long same = __ballot(in);
  for (int b = 0; b < bits; ++b) {
    const bool bit = (d >> b) & 1;
    const unsigned long long m = __ballot(bit);
    same &= bit ? m : ~m;
  }
  return same;
}

// hist[block * radix + digit].  The first pass (keys == nullptr) reads ids.
// One lane adds for all that hold its digit: frequent tokens would otherwise
// queue at one counter.
__global__ __launch_bounds__(SORT_THREADS) void k_sort_hist(const void *__restrict__ ids, int id_bytes,
                                                            const unsigned *__restrict__ keys, int64_t tokens,
                                                            int64_t vocab, int64_t padding, int64_t span, int shift,
                                                            int bits, unsigned *__restrict__ hist) {
  __shared__ unsigned h[SORT_RADIX];
  const int radix = 1 << bits;
  if ((int)threadIdx.x < radix) h[threadIdx.x] = 0;
  __syncthreads();
  const int64_t t0 = blockIdx.x * span, t1 = t0 + span < tokens ? t0 + span : tokens;
  for (int64_t tile = t0; tile < t1; tile += SORT_THREADS) {
    const int64_t t = tile + threadIdx.x;
    const bool in = t < t1;
    const unsigned k = !in ? 0u : keys ? keys[t] : key_of(ids, id_bytes, t, vocab, padding);
    const unsigned d = (k >> shift) & (radix - 1);
    const unsigned long long same = same_digit(d, bits, in);
    if (in && (same & ((1ull << (threadIdx.x & 63)) - 1)) == 0) atomicAdd(&h[d], (unsigned)__popcll(same));
  }
  __syncthreads();
  if ((int)threadIdx.x < radix) hist[blockIdx.x * radix + threadIdx.x] = h[threadIdx.x];
}

__global__ __launch_bounds__(SORT_THREADS) void k_sort_scatter(
    const void *__restrict__ ids, int id_bytes, const unsigned *__restrict__ keys, const int *__restrict__ tok,
    int64_t tokens, int64_t vocab, int64_t padding, int64_t span, int shift, int bits,
    const unsigned *__restrict__ hist, unsigned *__restrict__ keys_out, int *__restrict__ tok_out,
    unsigned *__restrict__ sample, int sample_shift) {
  __shared__ unsigned base[SORT_RADIX];
  __shared__ unsigned count[SORT_WAVES][SORT_RADIX];
  __shared__ unsigned wave_sum[SORT_WAVES];
  const int radix = 1 << bits, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t t0 = blockIdx.x * span, t1 = t0 + span < tokens ? t0 + span : tokens;
  unsigned k_next = 0;
  int tok_next = 0;
  const auto load = [&](int64_t t) {
    if (t < t1) {
      k_next = keys ? keys[t] : key_of(ids, id_bytes, t, vocab, padding);
      tok_next = tok ? tok[t] : (int)t;
    }
  };
  load(t0 + tid);  // in flight while the places are added up
  // place of this workgroup's first token of digit tid: the digits below it
  // in all workgroups, then the same digit in the workgroups before
  unsigned total = 0, before = 0;
  if (tid < radix) {
#pragma unroll 16
    for (int b = 0; b < (int)gridDim.x; ++b) {
      const unsigned h = hist[b * radix + tid];
      before += b < (int)blockIdx.x ? h : 0;
      total += h;
    }
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

  for (int64_t tile = t0; tile < t1; tile += SORT_THREADS) {
    for (int i = tid; i < SORT_WAVES * radix; i += SORT_THREADS) count[i / radix][i % radix] = 0;
    __syncthreads();
    const bool in = tile + tid < t1;
    const unsigned k = in ? k_next : 0u;
    const int this_tok = tok_next;
    load(tile + SORT_THREADS + tid);
    const unsigned d = (k >> shift) & (radix - 1);
    const unsigned long long same = same_digit(d, bits, in);
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
      tok_out[p] = this_tok;
      if (sample && (p & ((1u << sample_shift) - 1)) == 0) sample[p >> sample_shift] = k;
    }
    __syncthreads();
  }
}

// Up to 1024 RUNS tokens in one workgroup and one launch: all passes in LDS.
// Each wave owns RUNS runs of 64 tokens in order.
constexpr int SMALL_TOKENS = 4 * SORT_THREADS;

template <int SMALL_RUNS>
__global__ __launch_bounds__(SORT_THREADS) void k_sort_small(const void *__restrict__ ids, int id_bytes, int tokens,
                                                             int64_t vocab, int64_t padding, int passes, int bits,
                                                             unsigned *__restrict__ keys_out,
                                                             int *__restrict__ tok_out) {
  __shared__ unsigned skey[SORT_THREADS * SMALL_RUNS];
  __shared__ unsigned short stok[SORT_THREADS * SMALL_RUNS];
  __shared__ unsigned base[SORT_RADIX];
  __shared__ unsigned count[SORT_WAVES][SORT_RADIX];
  __shared__ unsigned wave_sum[SORT_WAVES];
  const int radix = 1 << bits, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  unsigned k[SMALL_RUNS], rank[SMALL_RUNS];
  int tok[SMALL_RUNS];
#pragma unroll
  for (int i = 0; i < SMALL_RUNS; ++i) {
    const int t = wave * (64 * SMALL_RUNS) + i * 64 + lane;
    tok[i] = t;
    k[i] = t < tokens ? key_of(ids, id_bytes, t, vocab, padding) : 0u;
  }
  for (int pass = 0; pass < passes; ++pass) {
    const int shift = pass * bits;
    for (int i = tid; i < SORT_WAVES * radix; i += SORT_THREADS) count[i / radix][i % radix] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < SMALL_RUNS; ++i) {
      const bool in = wave * (64 * SMALL_RUNS) + i * 64 + lane < tokens;
      const unsigned d = (k[i] >> shift) & (radix - 1);
      const unsigned long long same = same_digit(d, bits, in);
      const unsigned r = __popcll(same & ((1ull << lane) - 1));
      const unsigned before = count[wave][d];
      sv::wave_lds_sync();
      if (in && r == 0) count[wave][d] = before + __popcll(same);
      sv::wave_lds_sync();
      rank[i] = before + r;
    }
    __syncthreads();
    // digit tid: its waves' places, then the digits' places
    unsigned total = 0;
    if (tid < radix) {
#pragma unroll
      for (int w = 0; w < SORT_WAVES; ++w) {
        const unsigned c = count[w][tid];
        count[w][tid] = total;
        total += c;
      }
    }
    unsigned scan = total;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const unsigned v = __shfl_up(scan, s, 64);
      if (lane >= s) scan += v;
    }
    if (lane == 63) wave_sum[wave] = scan;
    __syncthreads();
    unsigned below = 0;
    for (int i = 0; i < wave; ++i) below += wave_sum[i];
    if (tid < radix) base[tid] = below + scan - total;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < SMALL_RUNS; ++i) {
      if (wave * (64 * SMALL_RUNS) + i * 64 + lane < tokens) {
        const unsigned d = (k[i] >> shift) & (radix - 1);
        const unsigned p = base[d] + count[wave][d] + rank[i];
        skey[p] = k[i];
        stok[p] = (unsigned short)tok[i];
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < SMALL_RUNS; ++i) {
      const int t = wave * (64 * SMALL_RUNS) + i * 64 + lane;
      if (t < tokens) {
        k[i] = skey[t];
        tok[i] = stok[t];
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < SMALL_RUNS; ++i) {
    const int t = wave * (64 * SMALL_RUNS) + i * 64 + lane;
    if (t < tokens) {
      keys_out[t] = k[i];
      tok_out[t] = tok[i];
    }
  }
}

// ---------------------------------------------------------------- gradient

// A row's tokens are the run of its key in the sorted list.  A run of up to
// PIECE tokens is summed by one group of threads.  A longer one is cut into
// pieces of PIECE tokens from its own start on (so the cut depends on that
// row's tokens only); every piece leaves a node (sum and carried errors) per
// column and a second launch joins a row's nodes in order.
//
// Pieces are found by block of PIECE places of the sorted list: a run longer
// than PIECE has at most one piece starting in a block, and a block meets at
// most two such runs, the one that holds its first place and the one that
// holds its last.  Their nodes go to slots 2 b and 2 b + 1 of block b.
constexpr int PIECE = 32;
constexpr int64_t WIDE_ROWS = 16384;  // rows and pieces from which tiles are wide

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

// Lanes of a wave that belong to this thread's group of L.
template <int L>
__device__ __forceinline__ unsigned long long group_lanes() {
  return L == 64 ? ~0ull : ((1ull << (L % 64)) - 1) << ((threadIdx.x & 63) / L * L);
}

// lower_bound by a group of L neighbouring threads together: each step looks
// at L places at once.
template <int L>
__device__ __forceinline__ int lower_bound_group(const unsigned *__restrict__ keys, int n, unsigned key) {
  const int l = threadIdx.x % L;
  int lo = 0, len = n;
  while (len > 0) {
    const int chunk = (len + L - 1) / L, first = l * chunk;  // thread l looks at the last place of its chunk
    const int end = first + chunk < len ? first + chunk : len;
    const int c = __popcll(__ballot(first < len && keys[first < len ? lo + end - 1 : lo] < key) & group_lanes<L>());
    const int skip = c * chunk < len ? c * chunk : len;
    lo += skip;
    len = (chunk < len - skip ? chunk : len - skip) - 1;  // the chunk's last place is not below the key
  }
  return lo;
}

// The piece of `key`'s run that starts in the block of places [b0, b0 +
// PIECE), [lo, end), found by a group; end == lo if there is none (no run of
// more than PIECE, or none of its pieces starts here).
template <int L>
__device__ __forceinline__ void find_piece(const unsigned *__restrict__ keys, int tokens, unsigned key, int b0,
                                           int &lo, int &end) {
  const int l = threadIdx.x % L;
  const int s = lower_bound_group<L>(keys, tokens, key);
  lo = b0 <= s ? s : s + (b0 - s + PIECE - 1) / PIECE * PIECE;
  const unsigned beyond = keys[s + PIECE < tokens ? s + PIECE : 0];
  int held = 0;
#pragma unroll
  for (int i = 0; i < PIECE; i += L) {
    const int at = lo + i + l;
    const unsigned k = keys[at < tokens ? at : 0];
    held += __popcll(__ballot(i + l < PIECE && at < tokens && k == key) & group_lanes<L>());
  }
  end = s + PIECE < tokens && beyond == key && lo < b0 + PIECE ? lo + held : lo;
}

// The same node as sv::combine with a value without carry.
__device__ __forceinline__ void add_value(Node &a, float v) {
  const float s = a.s + v;
  const float bv = s - a.s;
  const float av = s - bv;
  a.c = a.c + ((a.s - av) + (v - bv));
  a.s = s;
}

// Keys that the search for a row's tokens finds in LDS: the whole list, or
// every 2^sample_shift-th key, which leaves a few steps in memory.
constexpr int LDS_KEYS = 4096;

// Adds the dy rows of the tokens at places [lo, hi), hi > lo, to the chunks
// of one thread, Q tokens' loads at a time.  Narrow tiles read the next
// tokens' numbers meanwhile (wide ones lose more by the registers).
template <class T, int VE, int L, int U>
__device__ __forceinline__ void sum_run(const T *__restrict__ dy, int64_t lddy, const int *__restrict__ tok, int lo,
                                        int hi, const int64_t (&e)[U], Node (&a)[U][VE]) {
  using C = Cols<T, VE>;
  constexpr int Q = L < 64 ? 16 : 8;  // short rows have little else in flight
#pragma unroll
  for (int i = 0; i < U; ++i)
#pragma unroll
    for (int j = 0; j < VE; ++j) a[i][j] = sv::zero_node();
  constexpr bool AHEAD = U == 1;
  int t[Q];
  const auto tokens_at = [&](int p) {
#pragma unroll
    for (int q = 0; q < Q; ++q) t[q] = tok[p + q < hi ? p + q : hi - 1];
  };
  if constexpr (AHEAD) tokens_at(lo);
  for (int p = lo; p < hi; p += Q) {
    typename C::Vec v[Q][U];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int64_t row = AHEAD ? t[q] : tok[p + q < hi ? p + q : hi - 1];
#pragma unroll
      for (int i = 0; i < U; ++i) v[q][i] = C::load(dy + row * lddy + e[i]);
    }
    if (AHEAD && p + Q < hi) tokens_at(p + Q);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      if (p + q < hi) {
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
          for (int j = 0; j < VE; ++j) add_value(a[i][j], svr::to_f<T>(v[q][i][j]));
      }
    }
  }
}

template <class T, int VE, int L, int U>
__device__ __forceinline__ void store_roots(T *__restrict__ row, const int64_t (&e)[U], const bool (&in)[U],
                                            float scale, const Node (&a)[U][VE]) {
  using C = Cols<T, VE>;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    typename C::Vec w;
#pragma unroll
    for (int j = 0; j < VE; ++j) w[j] = svr::from_f<T>(sv::root_value(a[i][j]) * scale);
    if (in[i]) C::store(row + e[i], w);
  }
}

// Bound by memory where the table is large: 16384 tokens into 64000 x 4096 bf16
// 139 us, 4.8 TB/s, of which writing the zeros of the other rows alone takes
// about 90 (a fill runs at 6.9 TB/s, this at 5.8).  Bound by the chain of
// loads (list, place, token, row) where it is small, about 10 us.
// Blocks [0, pieces): a wave (or group of L threads) per block of PIECE
// places and tile of L * U chunks.  Blocks behind: `per` <= L (row, tile)
// units per group, rows of up to PIECE tokens.
template <class T, int VE, int L, int U>
__global__ __launch_bounds__(THREADS) void k_emb_grad(const T *__restrict__ dy, int64_t lddy,
                                                      const unsigned *__restrict__ keys, const int *__restrict__ tok,
                                                      const unsigned *__restrict__ sample, int sample_shift,
                                                      int tokens, int64_t vocab, int64_t dim, int tiles, float scale,
                                                      int64_t piece_blocks, int per, T *__restrict__ grad, int64_t ldg,
                                                      Node *__restrict__ part) {
  using C = Cols<T, VE>;
  constexpr int G = THREADS / L;
  __shared__ unsigned list[LDS_KEYS];
  const int g = threadIdx.x / L, l = threadIdx.x % L;
  const int chunks = (int)((dim + VE - 1) / VE);
  const int samples = (tokens + (1 << sample_shift) - 1) >> sample_shift;  // <= LDS_KEYS
#pragma unroll 4
  for (int i = threadIdx.x; i < samples; i += THREADS) list[i] = sample[i];
  __syncthreads();
  if (blockIdx.x < piece_blocks) {
    const int64_t u = (int64_t)blockIdx.x * G + g;
    const int64_t b = (unsigned)u / (unsigned)tiles;
    const int64_t places = (tokens + PIECE - 1) / PIECE;
    if (b >= places) return;
    const int b0 = (int)(b * PIECE), b1 = b0 + PIECE < tokens ? b0 + PIECE : tokens;
    int64_t e[U];
    bool in[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int c = (int)(u - b * tiles) * (L * U) + i * L + l;
      in[i] = c < chunks;
      e[i] = C::first(in[i] ? c : 0, dim);
    }
    int plo[2] = {0, 0}, pend[2] = {0, 0};
    const auto plan = [&](const unsigned *list) {
      const unsigned kf = list[b0], kl = list[b1 - 1], kb = list[b0 > 0 ? b0 - 1 : 0],
                     ka = list[b1 < tokens ? b1 : b1 - 1];
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        const unsigned key = which ? kl : kf;
        // a run longer than PIECE reaches out of the block
        const bool before = !which && b0 > 0 && kb == key;
        const bool after = kl == key && b1 < tokens && ka == key;
        if (key < (unsigned)vocab && (before || after) && !(which && kl == kf))
          find_piece<L>(list, tokens, key, b0, plo[which], pend[which]);
      }
    };
    if (sample_shift == 0) plan(list);
    else plan(keys);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const int lo = plo[which], end = pend[which];
      if (lo == end) continue;
      Node a[U][VE];
      sum_run<T, VE, L, U>(dy, lddy, tok, lo, end, e, a);
      Node *o = part + (b * 2 + which) * dim;
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (in[i])
#pragma unroll
          for (int j = 0; j < VE; ++j) o[e[i] + j] = a[i][j];
    }
    return;
  }
  // Group w of W takes units w, w + W, ..: rows that many tokens name often lie
  // next to each other (small ids), so they go to different groups.  Thread i
  // of the group looks up the tokens of the group's unit i.
  const int64_t units = vocab * tiles;
  const int64_t groups = ((int64_t)gridDim.x - piece_blocks) * G;
  const int64_t w = ((int64_t)blockIdx.x - piece_blocks) * G + g;
  const bool mine = w + l * groups < units && l < per;
  const unsigned mv = (unsigned)(mine ? w + l * groups : 0) / (unsigned)tiles;
  int lo_of = 0, hi_of = 0;
  // one past PIECE stands for any longer run
  const auto look = [&](const unsigned *keys, int from, int n) {
    lo_of = hi_of = from + lower_bound(keys + from, n, mv);
    if (lo_of < tokens && keys[lo_of] == mv) {
      const int left = tokens - lo_of;
      hi_of += lower_bound(keys + lo_of, left <= PIECE ? left : PIECE + 1, mv + 1);
    }
  };
  if (mine) {
    if (sample_shift == 0) {
      look(list, 0, tokens);
    } else {  // behind the last sample below the row's key, up to the next sample
      const int i = lower_bound(list, samples, mv);
      const int from = i > 0 ? ((i - 1) << sample_shift) + 1 : 0;
      const int to = (i << sample_shift) < tokens ? i << sample_shift : tokens;
      look(keys, from, to - from);
    }
  }
  for (int k = 0; k < per; ++k) {
    const int64_t u = w + k * groups;
    const int lo = L == 64 ? __builtin_amdgcn_readlane(lo_of, k) : __shfl(lo_of, k, L);
    const int hi = L == 64 ? __builtin_amdgcn_readlane(hi_of, k) : __shfl(hi_of, k, L);
    if (u >= units) break;
    if (hi - lo > PIECE) continue;
    const int64_t v = (unsigned)u / (unsigned)tiles;
    int64_t e[U];
    bool in[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int c = (int)(u - v * tiles) * (L * U) + i * L + l;
      in[i] = c < chunks;
      e[i] = C::first(in[i] ? c : 0, dim);
    }
    T *row = grad + v * ldg;
    if (lo == hi) {
      typename C::Vec zero{};
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (in[i]) C::store(row + e[i], zero);
      continue;
    }
    Node a[U][VE];
    sum_run<T, VE, L, U>(dy, lddy, tok, lo, hi, e, a);
    store_roots<T, VE, L, U>(row, e, in, scale, a);
  }
}

// Rows of more than PIECE tokens: a workgroup per block of PIECE places and
// tile; it works if such a run starts in its block (the run of the block's
// last place, the only one that can).  The workgroup's groups of L threads
// join equal shares of the row's nodes in order, then the shares are joined
// pairwise.
constexpr int JOIN_THREADS = 512;
template <class T, int VE, int L, int U>
__global__ __launch_bounds__(JOIN_THREADS) void k_emb_join(const unsigned *__restrict__ keys, int tokens,
                                                           int64_t vocab, int64_t dim, int tiles, unsigned blocks,
                                                           float scale, T *__restrict__ grad, int64_t ldg,
                                                           const Node *__restrict__ part) {
  using C = Cols<T, VE>;
  constexpr int G = JOIN_THREADS / L;
  __shared__ Node lds[G / 2][L * VE];
  const int g = threadIdx.x / L, l = threadIdx.x % L, lane = threadIdx.x & 63;
  const int chunks = (int)((dim + VE - 1) / VE);
  for (unsigned bt = blockIdx.x; bt < blocks; bt += gridDim.x) {
    const int64_t b = bt / (unsigned)tiles;
    const int tile = (int)(bt - b * tiles);
    const int b0 = (int)(b * PIECE), b1 = b0 + PIECE < tokens ? b0 + PIECE : tokens;
    if (b1 == tokens) continue;  // no run that starts here is longer than PIECE
    const unsigned key = keys[b1 - 1], next = keys[b1], mine = keys[b0 + lane % PIECE];
    const unsigned last = b0 > 0 ? keys[b0 - 1] : ~key;
    if (next != key || last == key || key >= (unsigned)vocab) continue;
    const int s = b0 + __builtin_ctzll(__ballot(mine == key));
    // pieces start at s, s + PIECE, ..: those whose place still holds the key.
    // The first 64 at once, then by steps of 64 pieces, then the rest.
    const auto holds = [&](int64_t piece) {
      const int64_t at = s + piece * PIECE;
      return __ballot(at < tokens && keys[at < tokens ? at : 0] == key);
    };
    int count = 1 + __popcll(holds(1 + lane));
    if (count == 1) continue;
    if (count == 65) {
      unsigned long long hit;
      do {
        hit = holds((int64_t)count + 64 * lane + 63);
        count += 64 * __popcll(hit);
      } while (!~hit);
      count += __popcll(holds((int64_t)count + lane));
    }
    const int share = (count + G - 1) / G;
    const int q0 = g * share, q1 = q0 + share < count ? q0 + share : count;
    for (int i = 0; i < U; ++i) {
      const int c = tile * (L * U) + i * L + l;
      const bool in = c < chunks;
      const int64_t e = C::first(in ? c : 0, dim);
      Node a[VE];
#pragma unroll
      for (int j = 0; j < VE; ++j) a[j] = sv::zero_node();
#pragma unroll 2
      for (int q = q0; q < q1; ++q) {
        const int first = s + q * PIECE;
        // the run's first piece lies behind another run unless it opens its block
        const Node *p = part + ((int64_t)(first / PIECE) * 2 + (q == 0 && s != b0)) * dim + e;
#pragma unroll
        for (int j = 0; j < VE; ++j) a[j] = sv::combine(a[j], p[j]);
      }
      for (int h = G / 2; h >= 1; h /= 2) {
        __syncthreads();
        if (g >= h && g < 2 * h) {
#pragma unroll
          for (int j = 0; j < VE; ++j) lds[g - h][l * VE + j] = a[j];
        }
        __syncthreads();
        if (g < h) {
#pragma unroll
          for (int j = 0; j < VE; ++j) a[j] = sv::combine(a[j], lds[g][l * VE + j]);
        }
      }
      if (g == 0 && in) {
        typename C::Vec w;
#pragma unroll
        for (int j = 0; j < VE; ++j) w[j] = svr::from_f<T>(sv::root_value(a[j]) * scale);
        C::store(grad + (int64_t)key * ldg + e, w);
      }
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
    with_cols<T, 4 * (16 / (int)sizeof(T))>(dim, [&](auto ve, auto l, auto u) {
      constexpr int VE = decltype(ve)::value, L = decltype(l)::value, U = decltype(u)::value, G = THREADS / L;
      const int64_t tiles = (dim + VE * L * U - 1) / (VE * L * U), units = tokens * tiles;
      const int64_t blocks = (units + G - 1) / G;
      k_emb_lookup<T, VE, L, U><<<(unsigned)(blocks < MAX_BLOCKS ? blocks : MAX_BLOCKS), THREADS, 0, s>>>(
          ids, id_bytes, units, (int)tiles, (const T *)table, vocab, dim, ldt, scale, (T *)out, ldo);
    });
  });
  return check_launch(who);
}

size_t sv_embedding_backward_workspace_size(int64_t tokens, int64_t vocab, int64_t dim, int dtype) {
  if (!svr::dtype_bytes(dtype) || tokens < 0 || vocab < 0 || dim < 0 || tokens > MAX_TOKENS || vocab > MAX_VOCAB ||
      dim > svr::MAX_N || (dim > 0 && (tokens > svr::MAX_VALUES / dim || vocab > svr::MAX_VALUES / dim)))
    return (size_t)-1;
  if (vocab == 0 || dim == 0) return 0;
  const size_t places = (size_t)(tokens + PIECE - 1) / PIECE;
  return 4 * svr::round256((size_t)tokens * 4) + (size_t)(SORT_MAX_BLOCKS * SORT_RADIX + LDS_KEYS) * 4 +
         (tokens > PIECE ? places * 2 * (size_t)dim * sizeof(Node) : 0);
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
  unsigned *sample = hist + SORT_MAX_BLOCKS * SORT_RADIX;
  Node *nodes = (Node *)(sample + LDS_KEYS);
  // few enough keys for LDS, and at least 16 apart: the rest is in one cache line
  int sample_shift = tokens <= LDS_KEYS ? 0 : 4;
  while (((tokens + ((int64_t)1 << sample_shift) - 1) >> sample_shift) > LDS_KEYS) ++sample_shift;
  int cur = 0;
  if (tokens > 0) {
    const SortPlan p = sort_plan(tokens, vocab);
    if (tokens <= SMALL_TOKENS) {
      auto *k = tokens <= SORT_THREADS       ? k_sort_small<1>
                : tokens <= 2 * SORT_THREADS ? k_sort_small<2>
                                             : k_sort_small<SMALL_TOKENS / SORT_THREADS>;
      k<<<1, SORT_THREADS, 0, s>>>(ids, id_bytes, (int)tokens, vocab, padding, p.passes, p.bits, keys[0], tok[0]);
    } else {
      for (int i = 0; i < p.passes; ++i) {
        const unsigned *kin = i ? keys[cur] : nullptr;
        const int *tin = i ? tok[cur] : nullptr;
        k_sort_hist<<<p.blocks, SORT_THREADS, 0, s>>>(ids, id_bytes, kin, tokens, vocab, padding, p.span, i * p.bits,
                                                      p.bits, hist);
        k_sort_scatter<<<p.blocks, SORT_THREADS, 0, s>>>(ids, id_bytes, kin, tin, tokens, vocab, padding, p.span,
                                                         i * p.bits, p.bits, hist, keys[cur ^ 1], tok[cur ^ 1],
                                                         i + 1 == p.passes ? sample : nullptr, sample_shift);
        cur ^= 1;
      }
    }
  }
  svr::with_type(dtype, [&](auto t) {
    using T = decltype(t);
    const auto go = [&](auto ve, auto l, auto u) {
      constexpr int VE = decltype(ve)::value, L = decltype(l)::value, U = decltype(u)::value, G = THREADS / L;
      const int64_t tiles = (dim + VE * L * U - 1) / (VE * L * U), units = vocab * tiles;
      const int64_t places = (tokens + PIECE - 1) / PIECE;
      const int64_t pieces = tokens > PIECE ? (places * tiles + G - 1) / G : 0;
      // units per group: about 4096 workgroups, so that a few rows share the
      // latency of the search for their tokens
      constexpr int MAX_PER = L < 16 ? L : 16;
      int64_t per = units / (4096 * G);
      per = per < 1 ? 1 : per > MAX_PER ? MAX_PER : per;
      const int64_t row_blocks = (units + per * G - 1) / (per * G);
      k_emb_grad<T, VE, L, U><<<(unsigned)(pieces + row_blocks), THREADS, 0, s>>>(
          (const T *)dy, lddy, keys[cur], tok[cur], sample_shift ? sample : keys[cur], sample_shift, (int)tokens, vocab,
          dim, (int)tiles, scale, pieces, (int)per,
          (T *)grad, ldg, nodes);
      if (pieces) {
        const int64_t blocks = places * tiles;
        k_emb_join<T, VE, L, U><<<(unsigned)(blocks < MAX_BLOCKS / 2 ? blocks : MAX_BLOCKS / 2), JOIN_THREADS, 0, s>>>(
            keys[cur], (int)tokens, vocab, dim, (int)tiles, (unsigned)blocks, scale, (T *)grad, ldg, nodes);
      }
    };
    // Wide tiles write longer runs of a row; narrow ones give more groups work.
    // Wide and narrow, us a call (dim > 64 chunks; shorter rows have one form):
    //   16384 tokens into 64000 rows x 4096 bf16   164  193
    //   65536                64000 x 4096          287  318    float32  490  535
    //   65536                20000 x 4096          224  228             345  367
    //   65536                 2000 x 4096          187  187             278  299
    //    5000                20000 x 4096           64   62              93   91
    //   65536                64000 x 1024          117  106             162  161
    //   65536                  300 x 1024           82   62              92   89
    //   65536                64000 x  600          100   86             136  123
    // So the rule, which looks at the rows and pieces alone, fits rows of 4096
    // values; for shorter rows of large tables narrow tiles would be up to a
    // fifth faster, and for float32 rows of 4096 wide ones by 6% in small tables.
    if (vocab + tokens / PIECE >= WIDE_ROWS) with_cols<T, 2 * (16 / (int)sizeof(T))>(dim, go);
    else with_cols<T, 16 / (int)sizeof(T)>(dim, go);
  });
  return check_launch(who);
}

}  // extern "C"
