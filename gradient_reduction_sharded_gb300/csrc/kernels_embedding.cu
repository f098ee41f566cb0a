// Vectors of a table by token id, and the table's gradient.
//
// Forward is a gather.  Backward sorts the tokens by their row of the table (a
// stable counting sort, digit by digit, so that equal rows keep the order of
// their tokens) and then writes every row of the gradient once: the sum of its
// tokens' vectors in order, or zeros.  Nothing is added by atomics, so two runs
// give the same bits.
//
// Token frequencies are steep (a few ids, or a padding id that counts, can be a
// large part of a batch), so the sorted tokens are cut into windows, and a row
// whose tokens cross from one window into the next is added up by windows
// first.  A window has parts of at most two such rows: the one that comes in
// from the left (slot 0) and the one that goes on to the right (slot 1).
//
// Forward of 32768 vectors of 2048 bf16 takes 42 us; where ids fall as 1 / rank
// some 12200 of the vectors are distinct, and their 50 MB and the result's 134
// need 27: it is bound by latency, a thread waits for its id and then for its
// one load (DRAM 3 TB/s, L2 32 %).
//
// Backward is bound by memory.  16384 tokens into 151936 rows of 2048 take 135:
// the sums and zeros 114 (631 MB of DRAM traffic, 5.5 TB/s; issue 72 %), the sort
// about 17 in three launches bound by latency, the joining of split rows 5.  One
// block sorting all 16384 took 41, rows cleared beside the sort made it 143.
// Vectors that are not whole 16-byte chunks go by elements.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "api_util.h"
#include "device.cuh"
#include "internal.h"
#include "launch.cuh"
#include "operators.cuh"

namespace grs {
namespace {

constexpr int EMB_THREADS = 256;
constexpr int EMB_WARPS = EMB_THREADS / 32;
constexpr int EMB_DIGIT = 9;               // bits of a sorting pass at most
constexpr int EMB_EACH = (1 << EMB_DIGIT) / EMB_THREADS;  // bins of a thread
constexpr int EMB_MAX_CHUNKS = 128;        // chunks whose counts every sorting block may add up by itself
constexpr int EMB_MAX_ROWS = 32;           // rows of the table that a block takes
constexpr int EMB_TOKENS = 512;            // of a block's tokens in shared memory
constexpr int EMB_JOIN = 32;               // units of a row that a joining block takes
enum : int { SITE_EMB_TOKEN = 1, SITE_EMB_ROW = 2 };

__device__ int emb_flags[FLAG_COUNT];

// Row of the table of an id, `rows` for one that the table does not hold.
__device__ __forceinline__ int32_t emb_row(int32_t id, int32_t begin, int32_t rows) {
  const int64_t r = int64_t(id) - begin;
  return r >= 0 && r < rows ? static_cast<int32_t>(r) : rows;
}

// ------------------------------------------------------------------- sort
// One pass orders (row, token) pairs by a digit of the row, the order of
// equal digits kept.  The first pass takes the ids themselves (keys NULL).
// A block has a chunk of 256 J pairs; counts[chunk][bin] says how many of each
// digit.  The first pass's counts come from a kernel of their own, which
// clears the later ones'; these are counted where a pass puts its pairs (by
// integer atomics, whose order changes nothing).
struct SortArgs {
  const int32_t *ids, *keys, *tokens;
  int32_t *keys_out, *tokens_out;
  int32_t *counts, *next;    // of this pass and the next one (NULL: the last)
  int32_t *totals;           // [bin] when a scan has run, else NULL
  int32_t n, begin, rows, shift, bins, chunks, clear;  // clear: tables behind `counts` to clear
};

__device__ __forceinline__ int32_t sort_key(const SortArgs& a, int64_t i) {
  return a.keys != nullptr ? __ldg(a.keys + i) : emb_row(__ldg(a.ids + i), a.begin, a.rows);
}

template <int J>
__global__ void __launch_bounds__(EMB_THREADS) emb_count_kernel(const __grid_constant__ SortArgs a) {
  __shared__ int32_t hist[1 << EMB_DIGIT];
  pdl_wait();
  pdl_trigger();
  for (int b = threadIdx.x; b < a.bins; b += EMB_THREADS) hist[b] = 0;
  __syncthreads();
  const int64_t s0 = int64_t(blockIdx.x) * (EMB_THREADS * J);
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int64_t i = s0 + j * EMB_THREADS + threadIdx.x;
    if (i < a.n) atomicAdd(&hist[(sort_key(a, i) >> a.shift) & (a.bins - 1)], 1);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < a.bins; b += EMB_THREADS) {
    int32_t* c = a.counts + int64_t(blockIdx.x) * a.bins + b;
    *c = hist[b];
    for (int t = 1; t <= a.clear; ++t) c[int64_t(t) * a.chunks * a.bins] = 0;
  }
}

// Exclusive prefix over a block's threads; *total = the sum.
__device__ __forceinline__ int32_t emb_prefix(int32_t x, int32_t* warp_total, int32_t* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int32_t s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  if (lane == 31) warp_total[w] = s;
  __syncthreads();
  const int32_t v = lane < EMB_WARPS ? warp_total[lane] : 0;
  const int32_t t = __reduce_add_sync(0xffffffffu, lane < w ? v : 0);
  *total = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  return t + s - x;
}

// For very many chunks: each bin's counts to what lies before each chunk.
__global__ void __launch_bounds__(EMB_THREADS) emb_scan_kernel(const __grid_constant__ SortArgs a) {
  __shared__ int32_t warp_total[EMB_WARPS];
  pdl_wait();
  pdl_trigger();
  int32_t carry = 0;
  for (int64_t c0 = 0; c0 < a.chunks; c0 += EMB_THREADS) {
    const int64_t c = c0 + threadIdx.x;
    const int32_t x = c < a.chunks ? a.counts[c * a.bins + blockIdx.x] : 0;
    int32_t all;
    const int32_t before = emb_prefix(x, warp_total, &all);
    if (c < a.chunks) a.counts[c * a.bins + blockIdx.x] = carry + before;
    carry += all;
  }
  if (threadIdx.x == 0) a.totals[blockIdx.x] = carry;
}

// A warp ranks its 32 J pairs, 32 at a time, by a match of equal digits, and
// counts them by digit in shared memory; a prefix over the warps turns the
// counts into the warp's starts in the chunk.
template <int J>
__global__ void __launch_bounds__(EMB_THREADS) emb_scatter_kernel(const __grid_constant__ SortArgs a) {
  __shared__ int32_t at[EMB_WARPS][1 << EMB_DIGIT], start[1 << EMB_DIGIT];
  __shared__ int32_t warp_total[EMB_WARPS];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, bins = a.bins;
  const int64_t s0 = int64_t(blockIdx.x) * (EMB_THREADS * J) + w * (32 * J);
  int32_t key[J], token[J], rank[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int64_t i = s0 + j * 32 + lane;
    key[j] = i < a.n ? sort_key(a, i) : -1;
    token[j] = i < a.n && a.tokens != nullptr ? __ldg(a.tokens + i) : static_cast<int32_t>(i);
  }
  // The thread's bins: how many there are in all, and before this chunk.
  const int b0 = threadIdx.x * EMB_EACH;
  int32_t total[EMB_EACH] = {}, before[EMB_EACH] = {};
  if (a.totals != nullptr) {
#pragma unroll
    for (int q = 0; q < EMB_EACH; ++q)
      if (b0 + q < bins) {
        total[q] = __ldg(a.totals + b0 + q);
        before[q] = __ldg(a.counts + int64_t(blockIdx.x) * bins + b0 + q);
      }
  } else {
#pragma unroll 8
    for (int c = 0; c < a.chunks; ++c)
#pragma unroll
      for (int q = 0; q < EMB_EACH; ++q)
        if (b0 + q < bins) {
          const int32_t v = __ldg(a.counts + int64_t(c) * bins + b0 + q);
          total[q] += v;
          if (c < static_cast<int>(blockIdx.x)) before[q] += v;
        }
  }
  for (int b = lane; b < bins; b += 32) at[w][b] = 0;
  __syncwarp();
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int d = key[j] < 0 ? -1 : (key[j] >> a.shift) & (bins - 1);
    const unsigned same = __match_any_sync(0xffffffffu, d);
    rank[j] = d >= 0 ? at[w][d] + __popc(same & ((1u << lane) - 1u)) : 0;
    __syncwarp();
    if (d >= 0 && lane == __ffs(same) - 1) at[w][d] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  int32_t all = 0;
#pragma unroll
  for (int q = 0; q < EMB_EACH; ++q)
    if (b0 + q < bins) {
      int32_t sum = 0;
#pragma unroll
      for (int k = 0; k < EMB_WARPS; ++k) {
        const int32_t c = at[k][b0 + q];
        at[k][b0 + q] = sum;
        sum += c;
      }
      all += total[q];
    }
  int32_t whole, s = emb_prefix(all, warp_total, &whole);
#pragma unroll
  for (int q = 0; q < EMB_EACH; ++q)
    if (b0 + q < bins) {
      start[b0 + q] = s + before[q];
      s += total[q];
    }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < J; ++j) {
    if (key[j] < 0) continue;
    const int d = (key[j] >> a.shift) & (bins - 1);
    const int32_t to = start[d] + at[w][d] + rank[j];
    if (!GRS_CHECK(to >= 0 && to < a.n, emb_flags, SITE_EMB_TOKEN)) continue;
    a.keys_out[to] = key[j];
    a.tokens_out[to] = token[j];
    if (a.next != nullptr)
      atomicAdd(a.next + int64_t(to / (EMB_THREADS * J)) * bins + ((static_cast<uint32_t>(key[j]) >> a.shift) / bins & (bins - 1)), 1);
  }
}

// All passes by one block, for few tokens: pairs go from pass to pass through
// shared memory.
constexpr int EMB_SMALL = 16;  // pairs of a thread: up to 4096
struct SmallSortArgs {
  const int32_t* ids;
  int32_t *keys_out, *tokens_out;
  int32_t n, begin, rows, digit, passes;
};

__global__ void __launch_bounds__(EMB_THREADS) emb_small_sort_kernel(const __grid_constant__ SmallSortArgs a) {
  __shared__ int32_t at[EMB_WARPS][1 << EMB_DIGIT], warp_total[EMB_WARPS];
  __shared__ int2 pairs[EMB_SMALL * EMB_THREADS];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, bins = 1 << a.digit;
  const int each = (a.n + EMB_THREADS - 1) / EMB_THREADS;  // of a thread; a warp has 32 each neighbours
  int32_t key[EMB_SMALL], token[EMB_SMALL], rank[EMB_SMALL];
#pragma unroll
  for (int j = 0; j < EMB_SMALL; ++j) {
    const int i = w * 32 * each + j * 32 + lane;
    key[j] = j < each && i < a.n ? emb_row(__ldg(a.ids + i), a.begin, a.rows) : -1;
    token[j] = i;
  }
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.digit;
    for (int b = lane; b < bins; b += 32) at[w][b] = 0;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < EMB_SMALL; ++j) {
      if (j >= each) break;
      const int d = key[j] < 0 ? -1 : (key[j] >> shift) & (bins - 1);
      const unsigned same = __match_any_sync(0xffffffffu, d);
      rank[j] = d >= 0 ? at[w][d] + __popc(same & ((1u << lane) - 1u)) : 0;
      __syncwarp();
      if (d >= 0 && lane == __ffs(same) - 1) at[w][d] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
    const int b0 = threadIdx.x * EMB_EACH;
    int32_t total[EMB_EACH] = {}, all = 0, whole;
#pragma unroll
    for (int q = 0; q < EMB_EACH; ++q) {
      if (b0 + q < bins)
#pragma unroll
        for (int k = 0; k < EMB_WARPS; ++k) {
          const int32_t c = at[k][b0 + q];
          at[k][b0 + q] = total[q];
          total[q] += c;
        }
      all += total[q];
    }
    int32_t s = emb_prefix(all, warp_total, &whole);
#pragma unroll
    for (int q = 0; q < EMB_EACH; ++q) {
      if (b0 + q < bins)
#pragma unroll
        for (int k = 0; k < EMB_WARPS; ++k) at[k][b0 + q] += s;
      s += total[q];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < EMB_SMALL; ++j)
      if (key[j] >= 0) {
        const int to = at[w][(key[j] >> shift) & (bins - 1)] + rank[j];
        if (GRS_CHECK(to >= 0 && to < a.n, emb_flags, SITE_EMB_TOKEN)) pairs[to] = make_int2(key[j], token[j]);
      }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < EMB_SMALL; ++j) {
      const int i = w * 32 * each + j * 32 + lane;
      if (j < each && i < a.n) {
        key[j] = pairs[i].x;
        token[j] = pairs[i].y;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < EMB_SMALL; ++j) {
    const int i = w * 32 * each + j * 32 + lane;
    if (j < each && i < a.n) {
      a.keys_out[i] = key[j];
      a.tokens_out[i] = token[j];
    }
  }
}

// How many of keys[lo, hi) are below `key`, plus lo: a warp, 32 places a step.
__device__ __forceinline__ int32_t warp_lower_bound(const int32_t* keys, int64_t lo, int64_t hi, int64_t key) {
  const int lane = threadIdx.x & 31;
  while (lo < hi) {
    const int64_t step = (hi - lo + 31) / 32, i = lo + lane * step;
    const int below = __popc(__ballot_sync(0xffffffffu, i < hi && __ldg(keys + i) < key));
    if (below == 0) break;
    hi = lo + below * step < hi ? lo + below * step : hi;
    lo += (below - 1) * step + 1;
  }
  return static_cast<int32_t>(lo);
}

// ------------------------------------------------------------------- sums
template <typename T, typename G>
struct EmbArgs {
  const T* dy;
  G* dtable;
  const int32_t *keys, *tokens;
  float* parts;       // [windows][2][d]
  int32_t n, rows, d, units, window, windows;
  int32_t group;      // threads of a row, a power of 2
  int32_t each;       // rows of a block
  float scale;
};

// E elements of a vector on their way, as they are in memory.
template <typename T, int E>
struct Bits {
  static constexpr int N = E == 1 ? 1 : static_cast<int>(sizeof(T)) / 2;
  uint4 w[N];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (E == 1) {
      if constexpr (sizeof(T) == 2) w[0].x = uint32_t(__ldg(p)) << 16;
      else w[0].x = __float_as_uint(__ldg(p));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    }
  }
  __device__ __forceinline__ void add_to(float (&s)[E]) const {
    if constexpr (E == 1) {
      s[0] += __uint_as_float(w[0].x);
    } else if constexpr (sizeof(T) == 2) {
      add_bf16x8(s, w[0]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        s[4 * i] += __uint_as_float(w[i].x);
        s[4 * i + 1] += __uint_as_float(w[i].y);
        s[4 * i + 2] += __uint_as_float(w[i].z);
        s[4 * i + 3] += __uint_as_float(w[i].w);
      }
    }
  }
};

// Adds the vectors of tokens[from, to), elements [c, c + E), in order.  The
// loads of a batch are all on their way before the first is used.
template <int E, typename T, typename G>
__device__ __forceinline__ void emb_add(const EmbArgs<T, G>& a, const int32_t* tokens, int32_t from, int32_t to, int64_t c, float (&s)[E]) {
  constexpr int B = E == 8 && sizeof(T) == 4 ? 4 : 8;
#pragma unroll 1
  for (int32_t p0 = from; p0 < to; p0 += B) {
    Bits<T, E> v[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      v[b].clear();
      if (p0 + b < to) {
        const int32_t t = tokens[p0 + b];
        if (GRS_CHECK(t >= 0 && t < a.n, emb_flags, SITE_EMB_TOKEN)) v[b].load(a.dy + int64_t(t) * a.d + c);
      }
    }
#pragma unroll
    for (int b = 0; b < B; ++b)
      if (p0 + b < to) v[b].add_to(s);
  }
}

template <int E, typename T, typename G>
__device__ __forceinline__ void emb_store(const EmbArgs<T, G>& a, int64_t row, int64_t c, float (&s)[E]) {
#pragma unroll
  for (int q = 0; q < E; ++q) s[q] *= a.scale;
  if (GRS_CHECK(row < a.rows && c + E <= a.d, emb_flags, SITE_EMB_ROW)) store_floats<E>(a.dtable + row * a.d + c, s);
}

// Window w of the sorted tokens: whether its first row comes in from the left
// and its last one goes on to the right.
struct Window {
  int64_t p0, p1;
  int32_t first, last;
  bool in, on;
  template <typename T, typename G>
  __device__ __forceinline__ Window(const EmbArgs<T, G>& a, int64_t w) {
    p0 = w * a.window;
    p1 = p0 + a.window < a.n ? p0 + a.window : a.n;
    first = __ldg(a.keys + p0);
    last = __ldg(a.keys + p1 - 1);
    in = first < a.rows && p0 > 0 && __ldg(a.keys + p0 - 1) == first;
    on = last < a.rows && p1 < a.n && __ldg(a.keys + p1) == last;
  }
};

// Rows without tokens are most of a large vocabulary: zeros to store.  The
// first blocks add up the windows' parts, so that these are long done when the
// last rows are stored.
template <typename T, typename G, int E>
__global__ void __launch_bounds__(EMB_THREADS) emb_sum_kernel(const __grid_constant__ EmbArgs<T, G> a) {
  __shared__ int32_t starts[EMB_MAX_ROWS + 1], tokens[EMB_TOKENS];
  pdl_wait();
  pdl_trigger();
  const int w = threadIdx.x >> 5;
  if (static_cast<int64_t>(blockIdx.x) < a.windows) {
    const Window x(a, blockIdx.x);
    for (int slot = 0; slot < 2; ++slot) {
      if (slot == 0 ? !x.in : !x.on || (x.in && x.last == x.first)) continue;
      const int32_t from = slot == 0 ? static_cast<int32_t>(x.p0) : warp_lower_bound(a.keys, x.p0, x.p1, x.last);
      const int32_t to = slot == 0 ? warp_lower_bound(a.keys, x.p0, x.p1, int64_t(x.first) + 1) : static_cast<int32_t>(x.p1);
      for (int64_t u = threadIdx.x; u < a.units; u += EMB_THREADS) {
        float sum[E] = {};
        emb_add<E>(a, a.tokens, from, to, u * E, sum);
        float* o = a.parts + (int64_t(blockIdx.x) * 2 + slot) * a.d + u * E;
#pragma unroll
        for (int q = 0; q < E; ++q) o[q] = sum[q];
      }
    }
    return;
  }
  const int64_t row0 = (int64_t(blockIdx.x) - a.windows) * a.each;
  const int rows = a.rows - row0 < a.each ? static_cast<int>(a.rows - row0) : a.each;
  if (w < 2) {
    const int32_t at = warp_lower_bound(a.keys, 0, a.n, row0 + (w == 0 ? 0 : rows));
    starts[w == 0 ? 0 : rows] = at;
  }
  __syncthreads();
  const int32_t lo = starts[0], hi = starts[rows];
  for (int r = threadIdx.x; r > 0 && r < rows; r += EMB_THREADS) {
    int32_t b = lo, e = hi;
    while (b < e) {
      const int32_t mid = b + (e - b) / 2;
      if (__ldg(a.keys + mid) < row0 + r) b = mid + 1;
      else e = mid;
    }
    starts[r] = b;
  }
  const bool near = hi - lo <= EMB_TOKENS;
  if (near)
    for (int i = threadIdx.x; i < hi - lo; i += EMB_THREADS) tokens[i] = __ldg(a.tokens + lo + i);
  __syncthreads();
  const int g = threadIdx.x / a.group, u0 = threadIdx.x - g * a.group, groups = EMB_THREADS / a.group;
#pragma unroll 1
  for (int r = g; r < rows; r += groups) {
    const int32_t s = starts[r], e = starts[r + 1];
    if (s < e && s / a.window != (e - 1) / a.window) continue;  // joined from its parts
    for (int u = u0; u < a.units; u += a.group) {
      float sum[E] = {};
      if (s < e) {
        if (near) emb_add<E>(a, tokens, s - lo, e - lo, int64_t(u) * E, sum);
        else emb_add<E>(a, a.tokens, s, e, int64_t(u) * E, sum);
      }
      emb_store<E>(a, row0 + r, int64_t(u) * E, sum);
    }
  }
}

// The row that begins in window w and goes on from it: its parts in order.
// A block takes some units of the row, its groups of threads a run of the
// windows each.
template <typename T, typename G, int E>
__global__ void __launch_bounds__(EMB_THREADS) emb_join_kernel(const __grid_constant__ EmbArgs<T, G> a) {
  __shared__ float red[EMB_THREADS / EMB_JOIN][EMB_JOIN][E + 1];
  pdl_wait();
  pdl_trigger();
  const Window x(a, blockIdx.x);
  if (!x.on || (x.in && x.first == x.last)) return;
  const int32_t end = warp_lower_bound(a.keys, x.p1, a.n, int64_t(x.last) + 1);
  const int64_t n = (end - 1) / a.window - int64_t(blockIdx.x) + 1;  // windows
  constexpr int GROUPS = EMB_THREADS / EMB_JOIN;
  const int g = threadIdx.x / EMB_JOIN, i = threadIdx.x % EMB_JOIN;
  const int64_t per = (n + GROUPS - 1) / GROUPS;
  for (int64_t u0 = int64_t(blockIdx.y) * EMB_JOIN; u0 < a.units; u0 += int64_t(gridDim.y) * EMB_JOIN) {
    const int64_t u = u0 + i;
    float sum[E] = {};
    if (u < a.units) {
#pragma unroll 4
      for (int64_t k = g * per; k < n && k < (g + 1) * per; ++k) {
        const float* p = a.parts + ((blockIdx.x + k) * 2 + (k == 0 ? 1 : 0)) * a.d + u * E;
#pragma unroll
        for (int q = 0; q < E; ++q) sum[q] += p[q];
      }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < E; ++q) red[g][i][q] = sum[q];
    __syncthreads();
    if (g != 0 || u >= a.units) continue;
    for (int k = 1; k < GROUPS; ++k)
#pragma unroll
      for (int q = 0; q < E; ++q) sum[q] += red[k][i][q];
    emb_store<E>(a, x.last, u * E, sum);
  }
}

// y[t] = scale * table[row], a thread E elements of a token.
template <typename T, int E>
__global__ void __launch_bounds__(EMB_THREADS) emb_forward_kernel(const int32_t* __restrict__ ids, const T* __restrict__ table,
                                                                  T* __restrict__ y, int64_t tokens, int32_t begin, int32_t rows,
                                                                  int32_t d, int32_t units, float scale) {
  pdl_wait();
  pdl_trigger();
  const int64_t i = int64_t(blockIdx.x) * EMB_THREADS + threadIdx.x, t = i / units;
  if (t >= tokens) return;
  const int64_t c = (i - t * units) * E;
  const int32_t row = emb_row(__ldg(ids + t), begin, rows);
  float v[E] = {};
  if (row < rows) load_floats<E>(table + int64_t(row) * d + c, v);
#pragma unroll
  for (int q = 0; q < E; ++q) v[q] *= scale;
  if (GRS_CHECK(c + E <= d, emb_flags, SITE_EMB_ROW)) store_floats<E>(y + t * d + c, v);
}

// ------------------------------------------------------------------- host
struct EmbPlan {
  int32_t rows, bits, passes, digit, window;
  int64_t chunk, chunks, windows;
  int64_t at_keys, at_tokens, at_counts, at_totals, at_parts, bytes;  // of the workspace
};

EmbPlan emb_plan(const grs_embedding* s) {
  EmbPlan p;
  p.rows = s->row_end - s->row_begin;
  p.bits = 0;
  while (p.bits < 31 && (int64_t(p.rows) >> p.bits) != 0) ++p.bits;  // keys 0..rows
  p.passes = (p.bits + EMB_DIGIT - 1) / EMB_DIGIT;
  p.digit = (p.bits + p.passes - 1) / p.passes;
  // Windows of about sqrt(n) / 4 tokens: a row with all of them is added up in two steps of like length.
  p.window = 32;
  while (int64_t(p.window) * p.window * 16 < s->tokens) p.window *= 2;
  p.chunk = EMB_THREADS * (s->tokens <= 64 * 512 ? 2 : 8);  // small chunks as long as there are few
  p.chunks = (s->tokens + p.chunk - 1) / p.chunk;
  p.windows = (s->tokens + p.window - 1) / p.window;
  int64_t at = 0;
  auto take = [&at](int64_t bytes) {
    const int64_t here = at;
    at += (bytes + 15) & ~int64_t(15);
    return here;
  };
  p.at_keys = take(2 * s->tokens * 4);
  p.at_tokens = take(2 * s->tokens * 4);
  p.at_counts = take(p.passes * p.chunks * (int64_t(1) << p.digit) * 4);
  p.at_totals = take((int64_t(1) << p.digit) * 4);
  p.at_parts = take(p.windows > 1 ? p.windows * 2 * s->hidden * 4 : 0);
  p.bytes = at;
  return p;
}

grs_status check_embedding(const grs_embedding* s, const char* who) {
  if (s == nullptr) return api_fail(GRS_ERR_INVALID_ARG, who, "shape is NULL");
  if (s->tokens < 0 || s->tokens > GRS_MAX_ROWS || s->hidden < 1 || s->hidden > GRS_MAX_WIDTH)
    return api_fail(GRS_ERR_SHAPE, who, "tokens must be in [0, GRS_MAX_ROWS] and hidden in [1, GRS_MAX_WIDTH]");
  if (s->row_begin < 0 || s->row_end <= s->row_begin)
    return api_fail(GRS_ERR_INVALID_ARG, who, "the row range must be 0 <= begin < end");
  if (!std::isfinite(s->scale)) return api_fail(GRS_ERR_INVALID_ARG, who, "scale must be finite");
  if (!dtype_ok(s->dtype) || !dtype_ok(s->grad_dtype)) return api_fail(GRS_ERR_INVALID_ARG, who, "unknown element type");
  return GRS_OK;
}

template <int J>
cudaError_t emb_sort(const grs_embedding* s, const EmbPlan& p, const int32_t* ids, uint8_t* ws, const int32_t** keys,
                     const int32_t** tokens, void* stream) {
  const int64_t n = s->tokens;
  int32_t* k[2] = {reinterpret_cast<int32_t*>(ws + p.at_keys), reinterpret_cast<int32_t*>(ws + p.at_keys) + n};
  int32_t* t[2] = {reinterpret_cast<int32_t*>(ws + p.at_tokens), reinterpret_cast<int32_t*>(ws + p.at_tokens) + n};
  const int bins = 1 << p.digit;
  const int64_t table = p.chunks * bins;
  const dim3 grid(static_cast<unsigned>(p.chunks)), block(EMB_THREADS);
  cudaError_t e = cudaSuccess;
  if (n <= EMB_SMALL * EMB_THREADS) {
    *keys = k[0];
    *tokens = t[0];
    const SmallSortArgs a{ids, k[0], t[0], static_cast<int32_t>(n), s->row_begin, p.rows, p.digit, p.passes};
    return launch_pdl(emb_small_sort_kernel, dim3(1), block, 0, stream, a);
  }
  for (int i = 0; i < p.passes && e == cudaSuccess; ++i) {  // more tokens than that are several chunks
    SortArgs a{};
    a.ids = ids;
    a.keys = i == 0 ? nullptr : k[(i - 1) & 1];
    a.tokens = i == 0 ? nullptr : t[(i - 1) & 1];
    a.keys_out = k[i & 1];
    a.tokens_out = t[i & 1];
    a.counts = reinterpret_cast<int32_t*>(ws + p.at_counts) + i * table;
    a.next = i + 1 < p.passes ? a.counts + table : nullptr;
    a.n = static_cast<int32_t>(n);
    a.begin = s->row_begin;
    a.rows = p.rows;
    a.shift = i * p.digit;
    a.bins = bins;
    a.chunks = static_cast<int32_t>(p.chunks);
    a.clear = p.passes - 1;
    if (i == 0) e = launch_pdl(emb_count_kernel<J>, grid, block, 0, stream, a);
    if (e == cudaSuccess && p.chunks > EMB_MAX_CHUNKS) {
      a.totals = reinterpret_cast<int32_t*>(ws + p.at_totals);
      e = launch_pdl(emb_scan_kernel, dim3(bins), block, 0, stream, a);
    }
    if (e == cudaSuccess) e = launch_pdl(emb_scatter_kernel<J>, grid, block, 0, stream, a);
    *keys = a.keys_out;
    *tokens = a.tokens_out;
  }
  return e;
}

bool emb_whole(const grs_embedding* s, const void* a, const void* b) {
  return s->hidden % 8 == 0 && api_aligned(a, 16) && api_aligned(b, 16);
}

template <typename T, typename G, int E>
cudaError_t emb_backward(const grs_embedding* s, const int32_t* ids, const void* dy, void* dtable, uint8_t* ws, void* stream) {
  const EmbPlan p = emb_plan(s);
  EmbArgs<T, G> a{};
  cudaError_t e = p.chunk == 2 * EMB_THREADS ? emb_sort<2>(s, p, ids, ws, &a.keys, &a.tokens, stream)
                                             : emb_sort<8>(s, p, ids, ws, &a.keys, &a.tokens, stream);
  a.dy = static_cast<const T*>(dy);
  a.dtable = static_cast<G*>(dtable);
  a.parts = reinterpret_cast<float*>(ws + p.at_parts);
  a.n = static_cast<int32_t>(s->tokens);
  a.rows = p.rows;
  a.d = s->hidden;
  a.units = s->hidden / E;
  a.window = p.window;
  a.windows = p.windows > 1 ? static_cast<int32_t>(p.windows) : 0;
  a.scale = s->scale;
  a.group = 1;
  while (a.group < a.units && a.group < EMB_THREADS) a.group *= 2;
  // Rows of a block: as many as leave eight blocks an SM.
  const int64_t groups = EMB_THREADS / a.group;
  int64_t each = p.rows / (152 * 8) / groups * groups;
  if (each < groups) each = groups;
  if (each > EMB_MAX_ROWS) each = EMB_MAX_ROWS;
  a.each = static_cast<int32_t>(each);
  const int64_t blocks = a.windows + (p.rows + each - 1) / each, slices = (int64_t(a.units) + EMB_JOIN - 1) / EMB_JOIN;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  const dim3 block(EMB_THREADS);
  if (e == cudaSuccess)
    e = launch_pdl(emb_sum_kernel<T, G, E>, dim3(static_cast<unsigned>(blocks)), block, 0, stream, a);
  if (e == cudaSuccess && a.windows > 0)
    e = launch_pdl(emb_join_kernel<T, G, E>, dim3(static_cast<unsigned>(a.windows), static_cast<unsigned>(slices < 65535 ? slices : 65535)), block,
                   0, stream, a);
  return e;
}

template <typename T, typename G>
cudaError_t emb_backward(const grs_embedding* s, const int32_t* ids, const void* dy, void* dtable, uint8_t* ws, void* stream) {
  return emb_whole(s, dy, dtable) ? emb_backward<T, G, 8>(s, ids, dy, dtable, ws, stream)
                                  : emb_backward<T, G, 1>(s, ids, dy, dtable, ws, stream);
}

template <typename T, int E>
cudaError_t emb_forward(const grs_embedding* s, const int32_t* ids, const void* table, void* y, void* stream) {
  const int32_t units = s->hidden / E;
  const int64_t blocks = (s->tokens * units + EMB_THREADS - 1) / EMB_THREADS;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  return launch_pdl(emb_forward_kernel<T, E>, dim3(static_cast<unsigned>(blocks)), dim3(EMB_THREADS), 0, stream, ids,
                    static_cast<const T*>(table), static_cast<T*>(y), s->tokens, s->row_begin, s->row_end - s->row_begin, s->hidden, units,
                    s->scale);
}

}  // namespace

cudaError_t embedding_flags(int** at) { return cudaGetSymbolAddress(reinterpret_cast<void**>(at), emb_flags); }

}  // namespace grs

using namespace grs;

extern "C" {

int64_t grs_embedding_workspace_bytes(const grs_embedding* s) {
  if (check_embedding(s, "grs_embedding_workspace_bytes") != GRS_OK) return -1;
  return emb_plan(s).bytes;
}

grs_status grs_embedding_forward(const grs_embedding* s, const int32_t* ids, const void* table, void* y, void* stream) {
  static const char who[] = "grs_embedding_forward";
  const grs_status st = check_embedding(s, who);
  if (st != GRS_OK) return st;
  if (s->tokens == 0) return GRS_OK;
  if (ids == nullptr || table == nullptr || y == nullptr) return api_fail(GRS_ERR_INVALID_ARG, who, "NULL argument");
  const uintptr_t ea = dtype_size(s->dtype);
  if (!api_aligned(ids, 4) || !api_aligned(table, ea) || !api_aligned(y, ea))
    return api_fail(GRS_ERR_ALIGNMENT, who, "a pointer is not aligned to its element");
  const bool f = s->dtype == GRS_DTYPE_FP32, whole = emb_whole(s, table, y);
  const cudaError_t e = f ? (whole ? emb_forward<float, 8>(s, ids, table, y, stream) : emb_forward<float, 1>(s, ids, table, y, stream))
                          : (whole ? emb_forward<uint16_t, 8>(s, ids, table, y, stream) : emb_forward<uint16_t, 1>(s, ids, table, y, stream));
  return e == cudaSuccess ? GRS_OK : api_cuda_fail(e, who);
}

grs_status grs_embedding_backward(const grs_embedding* s, const int32_t* ids, const void* dy, void* dtable, void* workspace,
                                  void* stream) {
  static const char who[] = "grs_embedding_backward";
  const grs_status st = check_embedding(s, who);
  if (st != GRS_OK) return st;
  if (dtable == nullptr || (s->tokens > 0 && (ids == nullptr || dy == nullptr || workspace == nullptr)))
    return api_fail(GRS_ERR_INVALID_ARG, who, "NULL argument");
  if (!api_aligned(ids, 4) || !api_aligned(dy, dtype_size(s->dtype)) || !api_aligned(dtable, dtype_size(s->grad_dtype)) ||
      !api_aligned(workspace, 16))
    return api_fail(GRS_ERR_ALIGNMENT, who, "a misaligned pointer");
  cudaError_t e;
  if (s->tokens == 0) {
    e = cudaMemsetAsync(dtable, 0, size_t(s->row_end - s->row_begin) * s->hidden * dtype_size(s->grad_dtype), static_cast<cudaStream_t>(stream));
  } else {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const bool f = s->dtype == GRS_DTYPE_FP32, g = s->grad_dtype == GRS_DTYPE_FP32;
    e = f ? (g ? emb_backward<float, float>(s, ids, dy, dtable, ws, stream) : emb_backward<float, uint16_t>(s, ids, dy, dtable, ws, stream))
          : (g ? emb_backward<uint16_t, float>(s, ids, dy, dtable, ws, stream)
               : emb_backward<uint16_t, uint16_t>(s, ids, dy, dtable, ws, stream));
  }
  return e == cudaSuccess ? GRS_OK : api_cuda_fail(e, who);
}

}  // extern "C"
