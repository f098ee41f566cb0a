// Vectors of a table by token id, and the table's gradient.
//
// Forward is a gather.  Backward sorts the tokens by their row of the table
// (a stable counting sort, digit by digit, so that equal rows keep the order
// of their tokens), finds where each row's tokens begin, and writes every row
// of the gradient once: the sum of its tokens' vectors in order, or zeros.
// Nothing is added by atomics, so two runs give the same bits.
//
// Token frequencies are steep (a few ids, or a padding id that counts, can be
// a large part of a batch), so a row with more than a window of tokens is
// added up in parts first: the sorted tokens are cut into windows, and as such
// a row is longer than a window, a window holds parts of at most two of them,
// the one that its first token belongs to and the one of its last.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "api_util.h"
#include "device.cuh"
#include "internal.h"
#include "launch.cuh"
#include "operators.cuh"

namespace grs {
namespace {

constexpr int EMB_THREADS = 256;
constexpr int EMB_SORT_THREADS = 1024;
constexpr int EMB_ROWS = 8;                           // rows of the table that a group of threads takes
constexpr int EMB_WARPS = EMB_SORT_THREADS / 32;
constexpr int EMB_DIGIT = 9;                          // bits of a sorting pass at most
constexpr int64_t EMB_TABLE = 256 * 1024;             // counts that every sorting block may add up by itself
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
struct SortArgs {
  const int32_t *ids, *keys, *tokens;
  int32_t *keys_out, *tokens_out;
  int32_t *counts, *totals;  // counts[chunk][bin]; totals[bin] when a scan has run, else NULL
  int32_t n, begin, rows, shift, bins, chunks;
};

__device__ __forceinline__ int32_t sort_key(const SortArgs& a, int32_t i) {
  return a.keys != nullptr ? a.keys[i] : emb_row(a.ids[i], a.begin, a.rows);
}

template <int J>
__global__ void __launch_bounds__(EMB_SORT_THREADS) emb_count_kernel(const __grid_constant__ SortArgs a) {
  extern __shared__ int32_t hist[];
  pdl_wait();
  pdl_trigger();
  for (int b = threadIdx.x; b < a.bins; b += EMB_SORT_THREADS) hist[b] = 0;
  __syncthreads();
  const int64_t s0 = int64_t(blockIdx.x) * (EMB_SORT_THREADS * J);
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int64_t i = s0 + j * EMB_SORT_THREADS + threadIdx.x;
    if (i < a.n) atomicAdd(&hist[(sort_key(a, i) >> a.shift) & (a.bins - 1)], 1);  // whole numbers: any order gives the same
  }
  __syncthreads();
  for (int b = threadIdx.x; b < a.bins; b += EMB_SORT_THREADS) a.counts[int64_t(blockIdx.x) * a.bins + b] = hist[b];
}

// Exclusive prefix of a block's values, one a thread; *total = their sum.
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
  int32_t t = lane < w ? warp_total[lane] : 0, all = warp_total[lane];
  t = __reduce_add_sync(0xffffffffu, t);
  *total = __reduce_add_sync(0xffffffffu, all);
  __syncthreads();
  return t + s - x;
}

// For very many chunks: each bin's counts to what lies before each chunk.
__global__ void __launch_bounds__(EMB_SORT_THREADS) emb_scan_kernel(const __grid_constant__ SortArgs a) {
  __shared__ int32_t warp_total[EMB_WARPS];
  pdl_wait();
  pdl_trigger();
  int32_t carry = 0;
  for (int64_t c0 = 0; c0 < a.chunks; c0 += EMB_SORT_THREADS) {
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
__global__ void __launch_bounds__(EMB_SORT_THREADS) emb_scatter_kernel(const __grid_constant__ SortArgs a) {
  extern __shared__ int32_t at[];  // [EMB_WARPS][bins], the bins' totals, what lies before the chunk
  __shared__ int32_t warp_total[EMB_WARPS];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, bins = a.bins;
  const int64_t s0 = int64_t(blockIdx.x) * (EMB_SORT_THREADS * J) + w * (32 * J);
  int32_t *mine = at + w * bins, *total = at + EMB_WARPS * bins, *before = total + bins;
  int32_t key[J], token[J], rank[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int64_t i = s0 + j * 32 + lane;
    key[j] = i < a.n ? sort_key(a, i) : -1;
    token[j] = i < a.n && a.tokens != nullptr ? a.tokens[i] : static_cast<int32_t>(i);
  }
  for (int i = threadIdx.x; i < (EMB_WARPS + 2) * bins; i += EMB_SORT_THREADS) at[i] = 0;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int d = key[j] < 0 ? -1 : (key[j] >> a.shift) & (bins - 1);
    const unsigned same = __match_any_sync(0xffffffffu, d);
    rank[j] = d >= 0 ? mine[d] + __popc(same & ((1u << lane) - 1u)) : 0;
    __syncwarp();
    if (d >= 0 && lane == __ffs(same) - 1) mine[d] += __popc(same);
    __syncwarp();
  }
  if (a.chunks > 1 && a.totals == nullptr) {
    for (int c = w; c < a.chunks; c += EMB_WARPS)
      for (int x = lane; x < bins; x += 32) {
        const int32_t v = a.counts[int64_t(c) * bins + x];
        if (v != 0) {
          atomicAdd(&total[x], v);
          if (c < static_cast<int>(blockIdx.x)) atomicAdd(&before[x], v);
        }
      }
  }
  __syncthreads();
  const int x = threadIdx.x;
  int32_t sum = 0;
  if (x < bins) {
    for (int k = 0; k < EMB_WARPS; ++k) {
      const int32_t c = at[k * bins + x];
      at[k * bins + x] = sum;
      sum += c;
    }
    if (a.chunks > 1) sum = a.totals != nullptr ? a.totals[x] : total[x];
  }
  int32_t all;
  const int32_t start = emb_prefix(x < bins ? sum : 0, warp_total, &all);
  if (x < bins) before[x] = start + (a.totals != nullptr ? a.counts[int64_t(blockIdx.x) * bins + x] : before[x]);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < J; ++j) {
    if (key[j] < 0) continue;
    const int d = (key[j] >> a.shift) & (bins - 1);
    const int32_t to = before[d] + mine[d] + rank[j];
    if (!GRS_CHECK(to >= 0 && to < a.n, emb_flags, SITE_EMB_TOKEN)) continue;
    a.keys_out[to] = key[j];
    a.tokens_out[to] = token[j];
  }
}

// starts[r] = how many of the sorted rows are below r, r in [0, rows].
__global__ void __launch_bounds__(EMB_THREADS) emb_starts_kernel(const int32_t* __restrict__ keys, int32_t n, int32_t rows,
                                                                 int32_t* __restrict__ starts) {
  pdl_wait();
  pdl_trigger();
  const int64_t r = int64_t(blockIdx.x) * EMB_THREADS + threadIdx.x;
  if (r > rows) return;
  int32_t lo = 0, hi = n;
  while (lo < hi) {
    const int32_t mid = lo + (hi - lo) / 2;
    if (__ldg(keys + mid) < r) lo = mid + 1;
    else hi = mid;
  }
  starts[r] = lo;
}

// ------------------------------------------------------------------- sums
template <typename T, typename G>
struct EmbArgs {
  const T* dy;
  G* dtable;
  const int32_t *keys, *tokens, *starts;
  float* parts;  // [windows][2][d]
  int32_t n, rows, d, units, window;
  int32_t group;  // threads of a row, a power of 2
  float scale;
};

// Adds the vectors of the sorted tokens [from, to), elements [c, c + E), in order.
template <int E, typename T, typename G>
__device__ __forceinline__ void emb_add(const EmbArgs<T, G>& a, int32_t from, int32_t to, int64_t c, float (&s)[E]) {
  constexpr int B = 8;  // loads in flight
  for (int32_t p0 = from; p0 < to; p0 += B) {
    float v[B][E];
#pragma unroll
    for (int b = 0; b < B; ++b) {
#pragma unroll
      for (int q = 0; q < E; ++q) v[b][q] = 0.0f;
      if (p0 + b < to) {
        const int32_t t = __ldg(a.tokens + p0 + b);
        if (GRS_CHECK(t >= 0 && t < a.n, emb_flags, SITE_EMB_TOKEN)) load_floats<E>(a.dy + int64_t(t) * a.d + c, v[b]);
      }
    }
#pragma unroll
    for (int b = 0; b < B; ++b)
      if (p0 + b < to)
#pragma unroll
        for (int q = 0; q < E; ++q) s[q] += v[b][q];
  }
}

// Parts of the rows of more than a window of tokens: a block a window.
template <typename T, typename G, int E>
__global__ void __launch_bounds__(EMB_THREADS) emb_parts_kernel(const __grid_constant__ EmbArgs<T, G> a) {
  pdl_wait();
  pdl_trigger();
  const int64_t p0 = int64_t(blockIdx.x) * a.window, p1 = p0 + a.window < a.n ? p0 + a.window : a.n;
  int32_t done = -1;
  for (int slot = 0; slot < 2; ++slot) {
    const int32_t row = __ldg(a.keys + (slot == 0 ? p0 : p1 - 1));
    if (row == done || row >= a.rows) break;  // (one row all the window long; from here on tokens without a row)
    done = row;
    const int32_t s = __ldg(a.starts + row), e = __ldg(a.starts + row + 1);
    if (e - s <= a.window) continue;
    for (int64_t u = threadIdx.x; u < a.units; u += EMB_THREADS) {
      float sum[E] = {};
      emb_add<E>(a, s > p0 ? s : static_cast<int32_t>(p0), e < p1 ? e : static_cast<int32_t>(p1), u * E, sum);
      float* o = a.parts + (int64_t(blockIdx.x) * 2 + slot) * a.d + u * E;
#pragma unroll
      for (int q = 0; q < E; ++q) o[q] = sum[q];
    }
  }
}

// dtable[row] = scale * the sum of its tokens' vectors.  A group of threads
// takes a row, a thread E elements at a time; most rows of a large vocabulary
// have no token and are zeros to store.
template <typename T, typename G, int E>
__global__ void __launch_bounds__(EMB_THREADS) emb_sum_kernel(const __grid_constant__ EmbArgs<T, G> a) {
  pdl_wait();
  pdl_trigger();
  const int group = a.group, g = threadIdx.x / group, u0 = threadIdx.x - g * group, groups = EMB_THREADS / group;
  const int64_t first = int64_t(blockIdx.x) * (EMB_ROWS * groups) + g;
#pragma unroll 1
  for (int k = 0; k < EMB_ROWS; ++k) {
    const int64_t row = first + k * groups;
    if (row >= a.rows) return;
    const int32_t s = __ldg(a.starts + row), e = __ldg(a.starts + row + 1);
    for (int u = u0; u < a.units; u += group) {
      const int64_t c = int64_t(u) * E;
      float sum[E] = {};
      if (e - s <= a.window) {
        emb_add<E>(a, s, e, c, sum);
      } else {
        for (int32_t w = s / a.window; w <= (e - 1) / a.window; ++w) {
          const int slot = w * int64_t(a.window) >= s ? 0 : 1;
          const float* p = a.parts + (int64_t(w) * 2 + slot) * a.d + c;
#pragma unroll
          for (int q = 0; q < E; ++q) sum[q] += p[q];
        }
      }
#pragma unroll
      for (int q = 0; q < E; ++q) sum[q] *= a.scale;
      if (GRS_CHECK(c + E <= a.d, emb_flags, SITE_EMB_ROW)) store_floats<E>(a.dtable + row * a.d + c, sum);
    }
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
  int64_t at_keys, at_tokens, at_counts, at_starts, at_parts, bytes;  // of the workspace
};

int64_t round16(int64_t b) { return (b + 15) & ~int64_t(15); }

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
  p.chunk = s->tokens <= 152 * 1024 ? 1024 : 4096;
  p.chunks = (s->tokens + p.chunk - 1) / p.chunk;
  p.windows = (s->tokens + p.window - 1) / p.window;
  int64_t at = 0;
  auto take = [&at](int64_t bytes) {
    const int64_t here = at;
    at += round16(bytes);
    return here;
  };
  p.at_keys = take(2 * s->tokens * 4);
  p.at_tokens = take(2 * s->tokens * 4);
  p.at_counts = take((p.chunks + 1) * (int64_t(1) << p.digit) * 4);
  p.at_starts = take((int64_t(p.rows) + 1) * 4);
  p.at_parts = take(p.windows * 2 * s->hidden * 4);
  p.bytes = at;
  return p;
}

grs_status check_embedding(const grs_embedding* s, const char* who) {
  if (s == nullptr) return api_fail(GRS_ERR_INVALID_ARG, who, "shape is NULL");
  if (s->tokens < 0 || s->tokens > INT32_MAX || s->hidden < 1 || s->hidden > GRS_MAX_WIDTH)
    return api_fail(GRS_ERR_SHAPE, who, "tokens must be in [0, 2^31) and hidden in [1, GRS_MAX_WIDTH]");
  if (s->row_begin < 0 || s->row_end <= s->row_begin)
    return api_fail(GRS_ERR_INVALID_ARG, who, "the row range must be 0 <= begin < end");
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
  const dim3 grid(static_cast<unsigned>(p.chunks)), block(EMB_SORT_THREADS);
  cudaError_t e = allow_smem<emb_scatter_kernel<J>>((EMB_WARPS + 2) * (1 << EMB_DIGIT) * 4);
  for (int i = 0; i < p.passes && e == cudaSuccess; ++i) {
    SortArgs a{};
    a.ids = ids;
    a.keys = i == 0 ? nullptr : k[(i - 1) & 1];
    a.tokens = i == 0 ? nullptr : t[(i - 1) & 1];
    a.keys_out = k[i & 1];
    a.tokens_out = t[i & 1];
    a.counts = reinterpret_cast<int32_t*>(ws + p.at_counts);
    a.n = static_cast<int32_t>(n);
    a.begin = s->row_begin;
    a.rows = p.rows;
    a.shift = i * p.digit;
    a.bins = bins;
    a.chunks = static_cast<int32_t>(p.chunks);
    if (p.chunks > 1) e = launch_pdl(emb_count_kernel<J>, grid, block, size_t(bins) * 4, stream, a);
    if (e == cudaSuccess && p.chunks * bins > EMB_TABLE) {
      a.totals = a.counts + p.chunks * bins;
      e = launch_pdl(emb_scan_kernel, dim3(bins), block, 0, stream, a);
    }
    if (e == cudaSuccess) e = launch_pdl(emb_scatter_kernel<J>, grid, block, size_t(EMB_WARPS + 2) * bins * 4, stream, a);
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
  cudaError_t e = p.chunk == 1024 ? emb_sort<1>(s, p, ids, ws, &a.keys, &a.tokens, stream)
                                  : emb_sort<4>(s, p, ids, ws, &a.keys, &a.tokens, stream);
  int32_t* starts = reinterpret_cast<int32_t*>(ws + p.at_starts);
  a.dy = static_cast<const T*>(dy);
  a.dtable = static_cast<G*>(dtable);
  a.starts = starts;
  a.parts = reinterpret_cast<float*>(ws + p.at_parts);
  a.n = static_cast<int32_t>(s->tokens);
  a.rows = p.rows;
  a.d = s->hidden;
  a.units = s->hidden / E;
  a.window = p.window;
  a.scale = s->scale;
  a.group = 1;
  while (a.group < a.units && a.group < EMB_THREADS) a.group *= 2;
  const int64_t each = EMB_ROWS * (EMB_THREADS / a.group), blocks = (p.rows + each - 1) / each;
  const dim3 block(EMB_THREADS);
  if (e == cudaSuccess)
    e = launch_pdl(emb_starts_kernel, dim3(static_cast<unsigned>(p.rows / EMB_THREADS + 1)), block, 0, stream, a.keys, a.n, p.rows, starts);
  if (e == cudaSuccess && s->tokens > p.window)
    e = launch_pdl(emb_parts_kernel<T, G, E>, dim3(static_cast<unsigned>(p.windows)), block, 0, stream, a);
  if (e == cudaSuccess) e = launch_pdl(emb_sum_kernel<T, G, E>, dim3(static_cast<unsigned>(blocks)), block, 0, stream, a);
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

cudaError_t take_embedding_flags(int (&total)[FLAG_COUNT], cudaStream_t st) { return take_flags(emb_flags, total, st); }

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
