// Tokens sorted by expert and back.
//
// A slot is one (token, choice) pair, index token * top_k + choice; a row is
// a place in the expert-sorted order.  The sort is a stable counting sort of
// the slots by expert id; everything after it follows slot_row, the row of
// each slot, token by token: a token's vector is read (or written) once and
// its rows are written (or read) once, with no atomics and no order left
// open.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "api_util.h"
#include "device.cuh"
#include "internal.h"
#include "launch.cuh"

namespace grs {
namespace {

constexpr int MOE_THREADS = 256;
constexpr int MOE_CHUNK = 4096;        // slots of one sorting block
constexpr int MOE_SORT_THREADS = 1024; // 32 warps of 128 slots each
constexpr int MOE_WARPS = MOE_SORT_THREADS / 32;
static_assert(MOE_CHUNK == MOE_WARPS * 128, "four groups of 32 slots a warp");

__device__ __forceinline__ float moe_load(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }
__device__ __forceinline__ float moe_load(const float* p) { return *p; }
__device__ __forceinline__ void moe_store(uint16_t* p, float x) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
__device__ __forceinline__ void moe_store(float* p, float x) { *p = x; }

// Local expert of a slot, -1 when it goes elsewhere (or is no expert).
__device__ __forceinline__ int local_expert(const int32_t* ids, int64_t slot, int64_t n, int32_t begin, int32_t count) {
  if (slot >= n) return -1;
  const int64_t e = int64_t(ids[slot]) - begin;
  return e >= 0 && e < count ? static_cast<int>(e) : -1;
}

// Counts of one chunk's slots per expert: counts[expert * n_chunks + chunk].
__global__ void __launch_bounds__(MOE_SORT_THREADS) moe_count_kernel(const int32_t* __restrict__ ids, int64_t n, int32_t begin,
                                                                     int32_t count, int32_t* __restrict__ counts) {
  extern __shared__ int32_t hist[];
  pdl_wait();
  pdl_trigger();
  for (int e = threadIdx.x; e < count; e += MOE_SORT_THREADS) hist[e] = 0;
  __syncthreads();
  const int64_t s0 = int64_t(blockIdx.x) * MOE_CHUNK;
  for (int i = threadIdx.x; i < MOE_CHUNK; i += MOE_SORT_THREADS) {
    const int e = local_expert(ids, s0 + i, n, begin, count);
    if (e >= 0) atomicAdd(&hist[e], 1);  // counts of whole numbers: any order gives the same
  }
  __syncthreads();
  for (int e = threadIdx.x; e < count; e += MOE_SORT_THREADS) counts[int64_t(e) * gridDim.x + blockIdx.x] = hist[e];
}

// Exclusive prefix over counts[0 .. len) in place, by one block; the
// experts' offsets are the prefixes at chunk 0.
__global__ void __launch_bounds__(MOE_SORT_THREADS) moe_scan_kernel(int32_t* __restrict__ counts, int32_t n_chunks, int32_t count,
                                                                    int32_t* __restrict__ offsets) {
  __shared__ int32_t warp_total[MOE_WARPS];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t len = int64_t(n_chunks) * count;
  int32_t carry = 0;
  for (int64_t base = 0; base < len; base += MOE_SORT_THREADS) {
    const int64_t i = base + threadIdx.x;
    const int32_t x = i < len ? counts[i] : 0;
    int32_t s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    if (lane == 31) warp_total[w] = s;
    __syncthreads();
    int32_t before = carry, all = 0;
    for (int k = 0; k < MOE_WARPS; ++k) {
      if (k < w) before += warp_total[k];
      all += warp_total[k];
    }
    if (i < len) {
      counts[i] = before + s - x;
      if (i % n_chunks == 0) offsets[i / n_chunks] = before + s - x;
    }
    carry += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) offsets[count] = carry;
}

// Rows of one chunk's slots.  A warp owns 128 consecutive slots; its count
// per expert so far is in shared memory, turned into a start per warp by a
// prefix over the warps, and slots of one group of 32 are ranked by a match
// of equal experts: the order of slots is kept.
__global__ void __launch_bounds__(MOE_SORT_THREADS) moe_rows_kernel(const int32_t* __restrict__ ids, int64_t n, int32_t begin,
                                                                    int32_t count, const int32_t* __restrict__ starts,
                                                                    const int32_t* __restrict__ offsets,
                                                                    int32_t* __restrict__ row_slot,
                                                                    int32_t* __restrict__ slot_row) {
  extern __shared__ int32_t at[];  // [MOE_WARPS][count]
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t s0 = int64_t(blockIdx.x) * MOE_CHUNK + w * 128;
  int32_t* mine = at + w * count;
  for (int i = threadIdx.x; i < MOE_WARPS * count; i += MOE_SORT_THREADS) at[i] = 0;
  __syncthreads();
  int e[4];
  int rank[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    e[j] = local_expert(ids, s0 + j * 32 + lane, n, begin, count);
    const unsigned same = __match_any_sync(0xffffffffu, e[j]);
    rank[j] = 0;
    if (e[j] >= 0) {
      rank[j] = mine[e[j]] + __popc(same & ((1u << lane) - 1u));
    }
    __syncwarp();
    if (e[j] >= 0 && lane == __ffs(same) - 1) mine[e[j]] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  for (int x = threadIdx.x; x < count; x += MOE_SORT_THREADS) {
    int32_t s = starts[int64_t(x) * gridDim.x + blockIdx.x];
    for (int k = 0; k < MOE_WARPS; ++k) {
      const int32_t c = at[k * count + x];
      at[k * count + x] = s;
      s += c;
    }
  }
  __syncthreads();
  const int32_t total = offsets[count];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t slot = s0 + j * 32 + lane;
    if (slot >= n) continue;
    const int32_t row = e[j] >= 0 ? mine[e[j]] + rank[j] : -1;
    slot_row[slot] = row;
    if (row >= 0) row_slot[row] = static_cast<int32_t>(slot);
    if (slot >= total) row_slot[slot] = -1;  // rows that no slot has
  }
}

// A row index of the caller's map, -1 unless it is a row.
__device__ __forceinline__ int64_t checked_row(const int32_t* slot_row, int64_t slot, int64_t n_slots) {
  const int64_t r = slot_row[slot];
  return r >= 0 && r < n_slots ? r : -1;
}

template <typename T>
__global__ void __launch_bounds__(MOE_THREADS) moe_dispatch_kernel(const T* __restrict__ x, const int32_t* __restrict__ slot_row,
                                                                   T* __restrict__ xs, int64_t tokens, int32_t k, int32_t d) {
  pdl_wait();
  pdl_trigger();
  for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x)
    for (int c = threadIdx.x; c < d; c += MOE_THREADS) {
      const T v = x[t * d + c];
      for (int j = 0; j < k; ++j) {
        const int64_t r = checked_row(slot_row, t * k + j, tokens * k);
        if (r >= 0) xs[r * d + c] = v;
      }
    }
}

// y[t] = sum over the token's rows of weight * row; without weights, of the row.
template <typename T>
__global__ void __launch_bounds__(MOE_THREADS) moe_combine_kernel(const T* __restrict__ ys, const int32_t* __restrict__ slot_row,
                                                                  const float* __restrict__ weights, T* __restrict__ y,
                                                                  int64_t tokens, int32_t k, int32_t d) {
  pdl_wait();
  pdl_trigger();
  for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x)
    for (int c = threadIdx.x; c < d; c += MOE_THREADS) {
      float s = 0.0f;
      for (int j = 0; j < k; ++j) {
        const int64_t r = checked_row(slot_row, t * k + j, tokens * k);
        if (r >= 0) s = fmaf(weights != nullptr ? weights[t * k + j] : 1.0f, moe_load(ys + r * d + c), s);
      }
      moe_store(y + t * d + c, s);
    }
}

template <typename T>
__global__ void __launch_bounds__(MOE_THREADS) moe_combine_bwd_kernel(const T* __restrict__ dy, const T* __restrict__ ys,
                                                                      const int32_t* __restrict__ slot_row,
                                                                      const float* __restrict__ weights, T* __restrict__ dys,
                                                                      float* __restrict__ dweights, int64_t tokens, int32_t k,
                                                                      int32_t d) {
  __shared__ float red[MOE_THREADS / 32];
  pdl_wait();
  pdl_trigger();
  for (int64_t slot = blockIdx.x; slot < tokens * k; slot += gridDim.x) {
    const int64_t r = checked_row(slot_row, slot, tokens * k), t = slot / k;
    const float w = weights[slot];
    float s = 0.0f;
    if (r >= 0)
      for (int c = threadIdx.x; c < d; c += MOE_THREADS) {
        const float g = moe_load(dy + t * d + c);
        moe_store(dys + r * d + c, w * g);
        s = fmaf(g, moe_load(ys + r * d + c), s);
      }
    s = warp_sum(s);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
      s = red[0];
      for (int j = 1; j < MOE_THREADS / 32; ++j) s += red[j];
      dweights[slot] = s;
    }
    __syncthreads();
  }
}

grs_status check_moe(const grs_moe* s, const char* who) {
  if (s == nullptr) return api_fail(GRS_ERR_INVALID_ARG, who, "shape is NULL");
  if (s->tokens < 0 || s->top_k < 1 || s->hidden < 1) return api_fail(GRS_ERR_SHAPE, who, "tokens >= 0, top_k >= 1, hidden >= 1");
  if (s->tokens > INT32_MAX / s->top_k) return api_fail(GRS_ERR_SHAPE, who, "tokens * top_k must be below 2^31");
  if (s->expert_begin < 0 || s->expert_end <= s->expert_begin)
    return api_fail(GRS_ERR_INVALID_ARG, who, "the expert range must be 0 <= begin < end");
  if (s->expert_end - s->expert_begin > GRS_MOE_MAX_EXPERTS)
    return api_fail(GRS_ERR_SHAPE, who, "more than GRS_MOE_MAX_EXPERTS local experts");
  if (!dtype_ok(s->dtype)) return api_fail(GRS_ERR_INVALID_ARG, who, "unknown element type");
  return GRS_OK;
}

int64_t moe_chunks(const grs_moe* s) { return (s->tokens * s->top_k + MOE_CHUNK - 1) / MOE_CHUNK; }

unsigned moe_grid(int64_t n) { return static_cast<unsigned>(n < 1 << 20 ? n : 1 << 20); }

}  // namespace
}  // namespace grs

using namespace grs;

extern "C" {

int64_t grs_moe_workspace_bytes(const grs_moe* s) {
  if (check_moe(s, "grs_moe_workspace_bytes") != GRS_OK) return -1;
  return moe_chunks(s) * (s->expert_end - s->expert_begin) * 4;
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
  const int32_t count = s->expert_end - s->expert_begin;
  const int32_t chunks = static_cast<int32_t>(moe_chunks(s));
  int32_t* counts = static_cast<int32_t*>(workspace);
  cudaError_t e = cudaSuccess;
  if (chunks == 0) {
    e = cudaMemsetAsync(expert_offsets, 0, (size_t(count) + 1) * 4, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GRS_OK : api_cuda_fail(e, who);
  }
  e = launch_pdl(moe_count_kernel, dim3(chunks), dim3(MOE_SORT_THREADS), count * 4, stream, expert_ids, n, s->expert_begin, count,
               counts);
  if (e == cudaSuccess)
    e = launch_pdl(moe_scan_kernel, dim3(1), dim3(MOE_SORT_THREADS), 0, stream, counts, chunks, count, expert_offsets);
  if (e == cudaSuccess) {
    const size_t smem = size_t(MOE_WARPS) * count * 4;
    if (smem > 48 * 1024)
      e = cudaFuncSetAttribute(moe_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    const int32_t *starts = counts, *offsets = expert_offsets;
    if (e == cudaSuccess)
      e = launch_pdl(moe_rows_kernel, dim3(chunks), dim3(MOE_SORT_THREADS), smem, stream, expert_ids, n, s->expert_begin, count,
                   starts, offsets, row_slot, slot_row);
  }
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
  const dim3 grid(moe_grid(s->tokens)), block(MOE_THREADS);
  const cudaError_t e = s->dtype == GRS_DTYPE_FP32
                            ? launch_pdl(moe_dispatch_kernel<float>, grid, block, 0, stream, static_cast<const float*>(x), slot_row,
                                       static_cast<float*>(xs), s->tokens, s->top_k, s->hidden)
                            : launch_pdl(moe_dispatch_kernel<uint16_t>, grid, block, 0, stream, static_cast<const uint16_t*>(x),
                                       slot_row, static_cast<uint16_t*>(xs), s->tokens, s->top_k, s->hidden);
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
  const dim3 grid(moe_grid(s->tokens)), block(MOE_THREADS);
  const cudaError_t e =
      s->dtype == GRS_DTYPE_FP32
          ? launch_pdl(moe_combine_kernel<float>, grid, block, 0, stream, static_cast<const float*>(ys), slot_row, weights,
                     static_cast<float*>(y), s->tokens, s->top_k, s->hidden)
          : launch_pdl(moe_combine_kernel<uint16_t>, grid, block, 0, stream, static_cast<const uint16_t*>(ys), slot_row, weights,
                     static_cast<uint16_t*>(y), s->tokens, s->top_k, s->hidden);
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
  const dim3 grid(moe_grid(s->tokens * s->top_k)), block(MOE_THREADS);
  const cudaError_t e =
      s->dtype == GRS_DTYPE_FP32
          ? launch_pdl(moe_combine_bwd_kernel<float>, grid, block, 0, stream, static_cast<const float*>(dy),
                     static_cast<const float*>(ys), slot_row, weights, static_cast<float*>(dys), dweights, s->tokens, s->top_k, s->hidden)
          : launch_pdl(moe_combine_bwd_kernel<uint16_t>, grid, block, 0, stream, static_cast<const uint16_t*>(dy),
                     static_cast<const uint16_t*>(ys), slot_row, weights, static_cast<uint16_t*>(dys), dweights, s->tokens, s->top_k,
                     s->hidden);
  return e == cudaSuccess ? GRS_OK : api_cuda_fail(e, who);
}

}  // extern "C"
