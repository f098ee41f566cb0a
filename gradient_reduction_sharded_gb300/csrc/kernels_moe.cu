// Tokens sorted by expert and back.
//
// A slot is one (token, choice) pair, index token * top_k + choice; a row is
// a place in the expert-sorted order.  The sort is a stable counting sort of
// the slots by expert id; everything after it follows slot_row, the row of
// each slot, token by token: a token's vector is read (or written) once and
// its rows are written (or read) once, with no atomics and no order left
// open.
//
// The vectors' kernels are bound by memory.  A thread has 16 bytes (8 bf16 or
// 8 fp32 elements) of a token and of all its rows, up to eight rows' loads in
// flight before the first is used; with the conversion between the loads the
// compiler waits for each (combine of 16384 tokens x 8 rows of 2048 bf16: 277 us
// against 88).  At that size dispatch takes 91 us, combine and dispatch_backward
// 88 and combine_backward 171, 6.6 to 6.9 TB/s of a copy rate of 6.78; 6001 x 6
// rows 27, 29 and 50 us.  The sort of those 131072 slots among 32 experts takes 8 us,
// of 20 slots 2.6 (one launch), bound by latency.  Vectors of any other size
// go as shifted chunks at 2 to 5 TB/s.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "api_util.h"
#include "device.cuh"
#include "internal.h"
#include "launch.cuh"
#include "packed.cuh"
#include "shifted.cuh"

namespace grs {
namespace {

constexpr int MOE_THREADS = 256;
constexpr int MOE_SORT_THREADS = 1024;
constexpr int MOE_WARPS = MOE_SORT_THREADS / 32;

// Local expert of a slot, -1 when it goes elsewhere (or is no expert).
__device__ __forceinline__ int local_expert(const int32_t* ids, int64_t slot, int64_t n, int32_t begin, int32_t count) {
  if (slot >= n) return -1;
  const int64_t e = int64_t(ids[slot]) - begin;
  return e >= 0 && e < count ? static_cast<int>(e) : -1;
}

// A sorting block takes a chunk of 1024 J consecutive slots, a warp of it 32 J.
// Counts of one chunk's slots per expert: counts[chunk * count + expert].
template <int J>
__global__ void __launch_bounds__(MOE_SORT_THREADS) moe_count_kernel(const int32_t* __restrict__ ids, int64_t n, int32_t begin,
                                                                     int32_t count, int32_t* __restrict__ counts) {
  extern __shared__ int32_t hist[];
  pdl_wait();
  pdl_trigger();
  for (int e = threadIdx.x; e < count; e += MOE_SORT_THREADS) hist[e] = 0;
  __syncthreads();
  const int64_t s0 = int64_t(blockIdx.x) * (MOE_SORT_THREADS * J);
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int e = local_expert(ids, s0 + j * MOE_SORT_THREADS + threadIdx.x, n, begin, count);
    if (e >= 0) atomicAdd(&hist[e], 1);  // counts of whole numbers: any order gives the same
  }
  __syncthreads();
  for (int e = threadIdx.x; e < count; e += MOE_SORT_THREADS) counts[int64_t(blockIdx.x) * count + e] = hist[e];
}

// Exclusive prefix of a block's 1024 values; *total = their sum.
__device__ __forceinline__ int32_t block_prefix(int32_t x, int32_t* warp_total, int32_t* total) {
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

// For very many chunks: counts to each (chunk, expert)'s first row, a block an
// expert; then moe_rows_kernel finds its starts with one load (`ready`).
__global__ void __launch_bounds__(MOE_SORT_THREADS) moe_scan_kernel(int32_t* __restrict__ counts, int32_t n_chunks, int32_t count,
                                                                    int32_t* __restrict__ totals) {
  __shared__ int32_t warp_total[MOE_WARPS];
  pdl_wait();
  pdl_trigger();
  int32_t carry = 0;
  for (int64_t c0 = 0; c0 < n_chunks; c0 += MOE_SORT_THREADS) {
    const int64_t c = c0 + threadIdx.x;
    const int32_t x = c < n_chunks ? counts[c * count + blockIdx.x] : 0;
    int32_t all;
    const int32_t before = block_prefix(x, warp_total, &all);
    if (c < n_chunks) counts[c * count + blockIdx.x] = carry + before;
    carry += all;
  }
  if (threadIdx.x == 0) totals[blockIdx.x] = carry;
}

// Rows of one chunk's slots.  A warp ranks its slots, 32 at a time, by a match
// of equal experts, and counts them per expert in shared memory; a prefix over
// the warps turns the counts into the warp's starts behind the chunk's.  So
// the order of slots is kept.  The chunk's starts come from its own counts
// alone (one chunk), from all chunks' counts (few of them: each block adds up
// the whole table), or from the scan above (`totals`).
template <int J>
__global__ void __launch_bounds__(MOE_SORT_THREADS) moe_rows_kernel(const int32_t* __restrict__ ids, int64_t n, int32_t begin,
                                                                    int32_t count, int32_t n_chunks,
                                                                    const int32_t* __restrict__ counts,
                                                                    const int32_t* __restrict__ totals,
                                                                    int32_t* __restrict__ offsets,
                                                                    int32_t* __restrict__ row_slot,
                                                                    int32_t* __restrict__ slot_row) {
  extern __shared__ int32_t at[];  // [MOE_WARPS][count], then the experts' totals and what lies before the chunk
  __shared__ int32_t warp_total[MOE_WARPS];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t s0 = int64_t(blockIdx.x) * (MOE_SORT_THREADS * J) + w * (32 * J);
  int32_t *mine = at + w * count, *total = at + MOE_WARPS * count, *before = total + count;
  int e[J], rank[J];
#pragma unroll
  for (int j = 0; j < J; ++j) e[j] = local_expert(ids, s0 + j * 32 + lane, n, begin, count);
  for (int i = threadIdx.x; i < (MOE_WARPS + 2) * count; i += MOE_SORT_THREADS) at[i] = 0;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const unsigned same = __match_any_sync(0xffffffffu, e[j]);
    rank[j] = e[j] >= 0 ? mine[e[j]] + __popc(same & ((1u << lane) - 1u)) : 0;
    __syncwarp();
    if (e[j] >= 0 && lane == __ffs(same) - 1) mine[e[j]] += __popc(same);
    __syncwarp();
  }
  if (n_chunks > 1 && totals == nullptr) {
    for (int c = w; c < n_chunks; c += MOE_WARPS)
      for (int x = lane; x < count; x += 32) {
        const int32_t v = counts[int64_t(c) * count + x];
        if (v != 0) {
          atomicAdd(&total[x], v);
          if (c < static_cast<int>(blockIdx.x)) atomicAdd(&before[x], v);
        }
      }
  }
  __syncthreads();
  // The warps' counts to their offsets in the chunk (at most 1024 experts: a thread each).
  const int x = threadIdx.x;
  int32_t sum = 0;
  if (x < count) {
    for (int k = 0; k < MOE_WARPS; ++k) {
      const int32_t c = at[k * count + x];
      at[k * count + x] = sum;
      sum += c;
    }
    if (n_chunks > 1) sum = totals != nullptr ? totals[x] : total[x];
  }
  int32_t rows;
  int32_t start = block_prefix(x < count ? sum : 0, warp_total, &rows);
  if (x < count) {
    if (blockIdx.x == 0) offsets[x] = start;
    start += totals != nullptr ? counts[int64_t(blockIdx.x) * count + x] : before[x];
    before[x] = start;
  }
  if (blockIdx.x == 0 && x == 0) offsets[count] = rows;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int64_t slot = s0 + j * 32 + lane;
    if (slot >= n) continue;
    const int32_t row = e[j] >= 0 ? before[e[j]] + mine[e[j]] + rank[j] : -1;
    slot_row[slot] = row;
    if (row >= 0) row_slot[row] = static_cast<int32_t>(slot);
    if (slot >= rows) row_slot[slot] = -1;  // rows that no slot has
  }
}

// ------------------------------------------------------------- vectors
// Every thread handles 8 consecutive elements of a token and of its rows.
// With whole vectors (hidden a multiple of 8 elements, 16-byte aligned) a
// thread stands by itself; otherwise a warp takes a run of 256 elements whose
// rows all start anywhere (shifted.cuh).
template <typename T>
struct MoeArgs {
  const T *a, *b;              // inputs: tokens' or rows' vectors
  T *o;                        // output
  const int32_t* slot_row;
  const float* weights;        // may be null
  float* dweights;
  int64_t tokens, slots;
  int32_t k, d, units;         // units: 8-element groups of a vector, 256-element runs of a loose one
  int32_t group;               // threads of a token (combine_backward)
};

// A row index of the caller's map, -1 unless it is a row.
template <typename T>
__device__ __forceinline__ int64_t moe_row(const MoeArgs<T>& a, int64_t slot) {
  const int64_t r = __ldg(a.slot_row + slot);
  return r >= 0 && r < a.slots ? r : -1;
}

// The thread's elements [c, c + 8) of vector v, on their way and as pairs;
// zeros if v < 0 and beyond the vector.  Nothing behind vector v is read: the
// caller's matrix may end with it (the vectors before it are there).
template <bool kWhole, typename T>
struct Vec {
  Moving<T> m;
  int mis;  // loose vectors: bytes that the run starts after a 16-byte boundary

  // D: the type of a vector's width.
  template <typename D>
  __device__ __forceinline__ void start(const T* base, int64_t v, int c, D d) {
#pragma unroll
    for (int i = 0; i < Moving<T>::N; ++i) m.own[i] = 0u;
    mis = 0;
    if (v < 0) return;
    const int64_t before = v * d + c;
    const T* p = base + before;
    if constexpr (kWhole) {
      m.start(p);
    } else {
      mis = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
      m.start_within(p, mis, before < 8 ? static_cast<int>(before) : 8, static_cast<int>(d - c));
    }
  }
  __device__ __forceinline__ void finish() {
    if constexpr (!kWhole) m.finish(mis);
  }
  __device__ __forceinline__ float2 pair(int q) const { return m.pair(q); }
};

// Where a vector's elements from c on are stored.
template <bool kWhole, typename T>
__device__ __forceinline__ Run store_run(const T* p, int c, int d) {
  if constexpr (kWhole) return Run{0, true};
  return Run{static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15), d - (c & ~255) >= 256};
}

template <bool kWhole, typename T>
__device__ __forceinline__ void vec_store(T* m, int64_t v, int c, int d, const float2 (&o)[4]) {
  T* p = m + v * d + c;
  store8(p, store_run<kWhole>(p, c, d), kWhole ? 8 : d - c, o);
}

// The token and the first element of this thread as one of block `block`;
// false beyond the last.
template <bool kWhole, typename T>
__device__ __forceinline__ bool moe_place(const MoeArgs<T>& a, int64_t block, int64_t* t, int* c) {
  const int64_t i = kWhole ? block * MOE_THREADS + threadIdx.x : block * (MOE_THREADS / 32) + (threadIdx.x >> 5);
  *t = i <= UINT32_MAX ? static_cast<uint32_t>(i) / static_cast<uint32_t>(a.units) : i / a.units;
  const int u = static_cast<int>(i - *t * a.units);
  *c = kWhole ? u * 8 : u * 256 + (threadIdx.x & 31) * 8;
  return *t < a.tokens;
}

// xs[row] = x[t] for each of the token's rows: x is read once.  Whole vectors
// are bits to copy: fp32 ones go as 16-bit halves, twice as many elements, so
// their width (up to 2^31) comes from the units in 64 bits.  A block does
// the work of U blocks, so that a thread has U loads in flight where few
// stores follow each (10986 x 1 rows of 4096 bf16: 6.4 TB/s with two, 4.5 with
// one; x 2: 6.4 and 5.9).
template <typename T, bool kWhole, int U>
__global__ void __launch_bounds__(MOE_THREADS) moe_dispatch_kernel(const __grid_constant__ MoeArgs<T> a) {
  pdl_wait();
  pdl_trigger();
  const auto d = [&] {
    if constexpr (kWhole) return int64_t(a.units) * 8;
    else return a.d;
  }();
  int64_t t[U];
  int c[U];
  bool on[U];
  Vec<kWhole, T> x[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    on[u] = moe_place<kWhole>(a, int64_t(blockIdx.x) * U + u, &t[u], &c[u]);
    if (on[u]) x[u].start(a.a, t[u], c[u], d);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!on[u]) return;
    x[u].finish();
    constexpr int B = U > 1 ? 2 : 8;
    for (int j0 = 0; j0 < a.k; j0 += B) {
      int64_t r[B];
#pragma unroll
      for (int j = 0; j < B; ++j) r[j] = j0 + j < a.k ? moe_row(a, t[u] * a.k + j0 + j) : -1;
#pragma unroll
      for (int j = 0; j < B; ++j)
        if (r[j] >= 0) {
          T* p = a.o + r[j] * d + c[u];
          store_words(p, store_run<kWhole>(p, c[u], a.d), kWhole ? 8 : a.d - c[u], x[u].m.own);  // the bits as they are
        }
    }
  }
}

// The next two kernels have B rows of a token in flight at once: as many as
// tokens have, of 2, 4, 6 and 8: places without a row cost registers, so loads
// in flight (combine of 4096 x 2 rows of 4096 bf16: 15.0 us, and 29.0 with
// eight; both kernels of the backward pass of 6001 x 6
// of 2048: 79.3 us, and 85.2).
// Loose ones two: more rows' shifting is more code than the instruction caches
// like (combine of 6001 x 6 rows of 2051: bf16 53 us with 2, 68 with 4, 85
// with 8; fp32 74, 124, 235).

// y[t] = sum over the token's rows of weight * row; without weights, of the row.
template <typename T, bool kWhole, int B>
__global__ void __launch_bounds__(MOE_THREADS) moe_combine_kernel(const __grid_constant__ MoeArgs<T> a) {
  pdl_wait();
  pdl_trigger();
  int64_t t;
  int c;
  if (!moe_place<kWhole>(a, blockIdx.x, &t, &c)) return;
  float2 s[4] = {both(0.0f), both(0.0f), both(0.0f), both(0.0f)};
  for (int j0 = 0; j0 < a.k; j0 += B) {
    Vec<kWhole, T> v[B];
    float w[B];
#pragma unroll
    for (int j = 0; j < B; ++j) {
      const int64_t slot = t * a.k + j0 + j, r = j0 + j < a.k ? moe_row(a, slot) : -1;
      w[j] = r < 0 ? 0.0f : a.weights != nullptr ? __ldg(a.weights + slot) : 1.0f;
      v[j].start(a.a, r, c, a.d);
    }
#pragma unroll
    for (int j = 0; j < B; ++j) {
      v[j].finish();
#pragma unroll
      for (int q = 0; q < 4; ++q) s[q] = fma2(v[j].pair(q), both(w[j]), s[q]);
    }
  }
  vec_store<kWhole>(a.o, t, c, a.d, s);
}

// dys[row] = weight * dy[t] and dweights[slot] = <ys[row], dy[t]>.  A group of
// threads a token; its threads' parts of a batch of products meet once.
template <typename T, bool kWhole, int B>
__global__ void __launch_bounds__(MOE_THREADS) moe_combine_bwd_kernel(const __grid_constant__ MoeArgs<T> a) {
  __shared__ float red[MOE_THREADS / 32][B];
  pdl_wait();
  pdl_trigger();
  const int groups = blockDim.x / a.group, g = threadIdx.x / a.group, i = threadIdx.x - g * a.group;
  const int64_t t = int64_t(blockIdx.x) * groups + g;
  const bool on = t < a.tokens;
  const int per = kWhole ? a.group * 8 : a.group / 32 * 256;
  const int c0 = kWhole ? i * 8 : (i >> 5) * 256 + (i & 31) * 8;
  for (int j0 = 0; j0 < a.k; j0 += B) {
    int64_t r[B];
    float w[B], dot[B];
#pragma unroll
    for (int j = 0; j < B; ++j) {
      const int64_t slot = t * a.k + j0 + j;
      r[j] = on && j0 + j < a.k ? moe_row(a, slot) : -1;
      w[j] = r[j] >= 0 ? __ldg(a.weights + slot) : 0.0f;
      dot[j] = 0.0f;
    }
    if (on)
#pragma unroll 1
      for (int c = c0; (kWhole ? c : c & ~255) < a.d; c += per) {
        Vec<kWhole, T> gv, v[B];
        gv.start(a.a, t, c, a.d);
#pragma unroll
        for (int j = 0; j < B; ++j) v[j].start(a.b, r[j], c, a.d);
        gv.finish();
        float2 gy[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) gy[q] = gv.pair(q);
#pragma unroll
        for (int j = 0; j < B; ++j) {
          if (r[j] < 0) continue;
          v[j].finish();
          float2 s = both(0.0f), o[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            s = fma2(v[j].pair(q), gy[q], s);
            o[q] = mul2(gy[q], both(w[j]));
          }
          dot[j] += s.x + s.y;
          vec_store<kWhole>(a.o, r[j], c, a.d, o);
        }
      }
#pragma unroll
    for (int j = 0; j < B; ++j)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float x = __shfl_xor_sync(0xffffffffu, dot[j], o);
        if (o < a.group) dot[j] = __fadd_rn(dot[j], x);
      }
    if (a.group > 32) {  // one token a block
      __syncthreads();   // red may still be read
      if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int j = 0; j < B; ++j) red[threadIdx.x >> 5][j] = dot[j];
      __syncthreads();
      if (threadIdx.x < B && j0 + threadIdx.x < a.k) {
        float s = red[0][threadIdx.x];
        for (int k = 1; k < static_cast<int>(blockDim.x >> 5); ++k) s = __fadd_rn(s, red[k][threadIdx.x]);
        if (on) a.dweights[t * a.k + j0 + threadIdx.x] = s;
      }
    } else if (on && i == 0) {
#pragma unroll
      for (int j = 0; j < B; ++j)
        if (j0 + j < a.k) a.dweights[t * a.k + j0 + j] = dot[j];
    }
  }
}

grs_status check_moe(const grs_moe* s, const char* who) {
  if (s == nullptr) return api_fail(GRS_ERR_INVALID_ARG, who, "shape is NULL");
  if (s->tokens < 0 || s->top_k < 1 || s->hidden < 1 || s->hidden > GRS_MAX_WIDTH)
    return api_fail(GRS_ERR_SHAPE, who, "tokens must be >= 0, top_k >= 1 and hidden in [1, GRS_MAX_WIDTH]");
  if (s->tokens > INT32_MAX / s->top_k) return api_fail(GRS_ERR_SHAPE, who, "tokens * top_k must be below 2^31");
  if (s->expert_begin < 0 || s->expert_end <= s->expert_begin)
    return api_fail(GRS_ERR_INVALID_ARG, who, "the expert range must be 0 <= begin < end");
  if (s->expert_end - s->expert_begin > GRS_MOE_MAX_EXPERTS)
    return api_fail(GRS_ERR_SHAPE, who, "more than GRS_MOE_MAX_EXPERTS local experts");
  if (!dtype_ok(s->dtype)) return api_fail(GRS_ERR_INVALID_ARG, who, "unknown element type");
  return GRS_OK;
}

// Slots of a sorting block: 1024 while that makes one block an SM, else 4096.
int moe_chunk_slots(const grs_moe* s) { return s->tokens * s->top_k <= 152 * 1024 ? 1024 : 4096; }
int64_t moe_chunks(const grs_moe* s) {
  const int64_t c = moe_chunk_slots(s);
  return (s->tokens * s->top_k + c - 1) / c;
}

template <int J>
cudaError_t moe_sort(const grs_moe* s, const int32_t* ids, int32_t* offsets, int32_t* row_slot, int32_t* slot_row, int32_t* ws,
                     void* stream) {
  const int64_t n = s->tokens * s->top_k;
  const int32_t count = s->expert_end - s->expert_begin, chunks = static_cast<int32_t>(moe_chunks(s));
  const dim3 grid(static_cast<unsigned>(chunks)), block(MOE_SORT_THREADS);
  cudaError_t e = cudaSuccess;
  if (chunks > 1) e = launch_pdl(moe_count_kernel<J>, grid, block, size_t(count) * 4, stream, ids, n, s->expert_begin, count, ws);
  // Each block of the last kernel reads the whole table up to 256 Ki counts (1 MB); beyond, the scan is cheaper.
  const bool scan = int64_t(chunks) * count > 256 * 1024;
  int32_t* totals = scan ? ws + int64_t(chunks) * count : nullptr;
  if (e == cudaSuccess && scan)
    e = launch_pdl(moe_scan_kernel, dim3(static_cast<unsigned>(count)), block, 0, stream, ws, chunks, count, totals);
  if (e == cudaSuccess) e = allow_smem<moe_rows_kernel<J>>((MOE_WARPS + 2) * GRS_MOE_MAX_EXPERTS * 4);
  if (e == cudaSuccess)
    e = launch_pdl(moe_rows_kernel<J>, grid, block, size_t(MOE_WARPS + 2) * count * 4, stream, ids, n, s->expert_begin, count, chunks,
                   static_cast<const int32_t*>(ws), static_cast<const int32_t*>(totals), offsets, row_slot, slot_row);
  return e;
}

template <typename T>
MoeArgs<T> moe_args(const grs_moe* s, const void* a, const void* b, void* o, const int32_t* slot_row, const float* weights,
                    float* dweights, bool whole) {
  const int32_t units = whole ? s->hidden / 8 : (s->hidden - 1) / 256 + 1;
  return {static_cast<const T*>(a), static_cast<const T*>(b), static_cast<T*>(o), slot_row, weights, dweights, s->tokens,
          s->tokens * s->top_k, s->top_k, s->hidden, units, 0};
}

// A dispatch of whole fp32 vectors: 16-bit halves, 16 bytes a thread and row.
MoeArgs<uint16_t> moe_copy_args(const grs_moe* s, const void* x, void* xs, const int32_t* slot_row) {
  MoeArgs<uint16_t> a = moe_args<uint16_t>(s, x, nullptr, xs, slot_row, nullptr, nullptr, true);
  a.units *= 2;
  return a;
}

// 16-byte aligned vectors of whole 8-element groups.
bool moe_whole(const grs_moe* s, const void* a, const void* b, const void* o) {
  return s->hidden % 8 == 0 && api_aligned(a, 16) && api_aligned(b, 16) && api_aligned(o, 16);
}

enum class MoeOp { kDispatch, kCombine, kCombineBackward };

template <typename T, bool kWhole, int B>
cudaError_t moe_launch(MoeOp op, MoeArgs<T> a, void* stream) {
  if (op == MoeOp::kCombineBackward) {
    // Threads of a token: its units in whole groups as far as a block goes.
    int threads = MOE_THREADS;
    if (kWhole && a.units <= 32) {
      a.group = 1;
      while (a.group < a.units) a.group *= 2;
    } else {
      int warps = kWhole ? (a.units + 31) / 32 : a.units;
      if (a.tokens >= 16 * 152) {
        // Many tokens: 32 bytes of each row a thread.  With 180 MB of bf16 rows of 2048: 6.4 TB/s, 5.6 with 16
        // bytes and 256 threads, 5.6 with a warp a token; of 4096: 6.2, 6.1 and 4.9, so up to 128 threads.
        if (kWhole && sizeof(T) == 2) warps = warps >= 8 ? 4 : (warps + 1) / 2;
        // A warp for a loose one of up to 8 KB, whose products meet without a barrier.
        if (!kWhole && a.d * static_cast<int64_t>(sizeof(T)) <= 8192) warps = 1;
      }
      a.group = 32 * (warps < MOE_THREADS / 32 ? warps : MOE_THREADS / 32);
      threads = a.group > 32 ? a.group : 64;  // (two tokens a block: a finer tail than eight, 54.3 and 55.7 us for 6001 x 6)
    }
    const int64_t per = threads / a.group, blocks = (a.tokens + per - 1) / per;
    return launch_pdl(moe_combine_bwd_kernel<T, kWhole, B>, dim3(static_cast<unsigned>(blocks)), dim3(threads), 0, stream, a);
  }
  constexpr int U = kWhole && B == 2 ? 2 : 1;
  const bool dispatch = op == MoeOp::kDispatch;
  const int64_t per = (kWhole ? MOE_THREADS : MOE_THREADS / 32) * (dispatch ? U : 1), blocks = (a.tokens * a.units + per - 1) / per;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(blocks)), block(MOE_THREADS);
  if constexpr (!kWhole || sizeof(T) == 2)  // (whole fp32 vectors are copied as 16-bit halves)
    if (dispatch) return launch_pdl(moe_dispatch_kernel<T, kWhole, U>, grid, block, 0, stream, a);
  return launch_pdl(moe_combine_kernel<T, kWhole, B>, grid, block, 0, stream, a);
}

template <typename T>
cudaError_t moe_launch(MoeOp op, const MoeArgs<T>& a, bool whole, void* stream) {
  if (!whole) return moe_launch<T, false, 2>(op, a, stream);
  return a.k <= 2 ? moe_launch<T, true, 2>(op, a, stream)
         : a.k <= 4 ? moe_launch<T, true, 4>(op, a, stream)
         : a.k <= 6 ? moe_launch<T, true, 6>(op, a, stream)
                    : moe_launch<T, true, 8>(op, a, stream);
}

cudaError_t moe_run(MoeOp op, const grs_moe* s, const void* a, const void* b, void* o, const int32_t* slot_row,
                    const float* weights, float* dweights, void* stream) {
  const bool whole = moe_whole(s, a, b, o);
  if (op == MoeOp::kDispatch && whole && s->dtype == GRS_DTYPE_FP32) return moe_launch(op, moe_copy_args(s, a, o, slot_row), true, stream);
  if (s->dtype == GRS_DTYPE_FP32) {
    const MoeArgs<float> x = moe_args<float>(s, a, b, o, slot_row, weights, dweights, whole);
    return moe_launch(op, x, whole, stream);
  }
  const MoeArgs<uint16_t> x = moe_args<uint16_t>(s, a, b, o, slot_row, weights, dweights, whole);
  return moe_launch(op, x, whole, stream);
}

}  // namespace
}  // namespace grs

using namespace grs;

extern "C" {

int64_t grs_moe_workspace_bytes(const grs_moe* s) {
  if (check_moe(s, "grs_moe_workspace_bytes") != GRS_OK) return -1;
  return (moe_chunks(s) + 1) * (s->expert_end - s->expert_begin) * 4;  // counts of each chunk, totals
}

grs_status grs_moe_sort(const grs_moe* s, const int32_t* expert_ids, int32_t* expert_offsets, int32_t* row_slot,
                        int32_t* slot_row, void* workspace, void* stream) {
  static const char who[] = "grs_moe_sort";
  const grs_status st = check_moe(s, who);
  if (st != GRS_OK) return st;
  const int64_t n = s->tokens * s->top_k;
  if (expert_offsets == nullptr || (n > 0 && (expert_ids == nullptr || row_slot == nullptr || slot_row == nullptr || workspace == nullptr)))
    return api_fail(GRS_ERR_INVALID_ARG, who, "NULL argument");
  if (!api_aligned(expert_ids, 4) || !api_aligned(expert_offsets, 4) || !api_aligned(row_slot, 4) || !api_aligned(slot_row, 4) ||
      !api_aligned(workspace, 16))
    return api_fail(GRS_ERR_ALIGNMENT, who, "misaligned pointer");
  int32_t* ws = static_cast<int32_t*>(workspace);
  cudaError_t e;
  if (n == 0)
    e = cudaMemsetAsync(expert_offsets, 0, (size_t(s->expert_end - s->expert_begin) + 1) * 4, static_cast<cudaStream_t>(stream));
  else
    e = moe_chunk_slots(s) == 1024 ? moe_sort<1>(s, expert_ids, expert_offsets, row_slot, slot_row, ws, stream)
                                   : moe_sort<4>(s, expert_ids, expert_offsets, row_slot, slot_row, ws, stream);
  return e == cudaSuccess ? GRS_OK : api_cuda_fail(e, who);
}

grs_status grs_moe_dispatch(const grs_moe* s, const void* x, const int32_t* slot_row, void* xs, void* stream) {
  static const char who[] = "grs_moe_dispatch";
  const grs_status st = check_moe(s, who);
  if (st != GRS_OK) return st;
  if (s->tokens == 0) return GRS_OK;
  if (x == nullptr || slot_row == nullptr || xs == nullptr) return api_fail(GRS_ERR_INVALID_ARG, who, "NULL argument");
  const uintptr_t ea = dtype_size(s->dtype);
  if (!api_aligned(x, ea) || !api_aligned(xs, ea) || !api_aligned(slot_row, 4))
    return api_fail(GRS_ERR_ALIGNMENT, who, "a pointer is not aligned to its element");
  const cudaError_t e = moe_run(MoeOp::kDispatch, s, x, nullptr, xs, slot_row, nullptr, nullptr, stream);
  return e == cudaSuccess ? GRS_OK : api_cuda_fail(e, who);
}

static grs_status combine(const grs_moe* s, const void* ys, const int32_t* slot_row, const float* weights, bool weighted, void* y,
                          void* stream, const char* who) {
  const grs_status st = check_moe(s, who);
  if (st != GRS_OK) return st;
  if (s->tokens == 0) return GRS_OK;
  if (ys == nullptr || slot_row == nullptr || y == nullptr || (weighted && weights == nullptr))
    return api_fail(GRS_ERR_INVALID_ARG, who, "NULL argument");
  const uintptr_t ea = dtype_size(s->dtype);
  if (!api_aligned(ys, ea) || !api_aligned(y, ea) || !api_aligned(slot_row, 4) || !api_aligned(weights, 4))
    return api_fail(GRS_ERR_ALIGNMENT, who, "a pointer is not aligned to its element");
  const cudaError_t e = moe_run(MoeOp::kCombine, s, ys, nullptr, y, slot_row, weights, nullptr, stream);
  return e == cudaSuccess ? GRS_OK : api_cuda_fail(e, who);
}

grs_status grs_moe_dispatch_backward(const grs_moe* s, const void* dxs, const int32_t* slot_row, void* dx, void* stream) {
  return combine(s, dxs, slot_row, nullptr, false, dx, stream, "grs_moe_dispatch_backward");
}

grs_status grs_moe_combine(const grs_moe* s, const void* ys, const int32_t* slot_row, const float* weights, void* y, void* stream) {
  return combine(s, ys, slot_row, weights, true, y, stream, "grs_moe_combine");
}

grs_status grs_moe_combine_backward(const grs_moe* s, const void* dy, const void* ys, const int32_t* slot_row, const float* weights,
                                    void* dys, float* dweights, void* stream) {
  static const char who[] = "grs_moe_combine_backward";
  const grs_status st = check_moe(s, who);
  if (st != GRS_OK) return st;
  if (s->tokens == 0) return GRS_OK;
  if (dy == nullptr || ys == nullptr || slot_row == nullptr || weights == nullptr || dys == nullptr || dweights == nullptr)
    return api_fail(GRS_ERR_INVALID_ARG, who, "NULL argument");
  const uintptr_t ea = dtype_size(s->dtype);
  if (!api_aligned(dy, ea) || !api_aligned(ys, ea) || !api_aligned(dys, ea) || !api_aligned(slot_row, 4) ||
      !api_aligned(weights, 4) || !api_aligned(dweights, 4))
    return api_fail(GRS_ERR_ALIGNMENT, who, "a pointer is not aligned to its element");
  const cudaError_t e = moe_run(MoeOp::kCombineBackward, s, dy, ys, dys, slot_row, weights, dweights, stream);
  return e == cudaSuccess ? GRS_OK : api_cuda_fail(e, who);
}

}  // extern "C"
