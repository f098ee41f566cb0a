// Device helpers of the experts' products.
#pragma once

#include <cstdint>

#include "device.cuh"
#include "experts.h"

namespace grs {

// An expert's rows, as the caller's offsets say within [0, rows].
struct ExpertRows {
  int32_t from, to;
  __device__ __forceinline__ ExpertRows(const int32_t* offsets, int e, int32_t rows) {
    from = __ldg(offsets + e);
    to = __ldg(offsets + e + 1);
    from = from < 0 ? 0 : from > rows ? rows : from;
    to = to < from ? from : to > rows ? rows : to;
  }
};

// first[e] = groups of G rows before expert e's, first[experts] all of them; by a whole block.
template <int G, int kThreads>
__device__ __forceinline__ void group_prefix(const int32_t* offsets, int32_t experts, int32_t rows, int32_t* first) {
  __shared__ int32_t sums[kThreads / 32];
  constexpr int EACH = (GRS_MOE_MAX_EXPERTS + kThreads - 1) / kThreads;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int32_t n[EACH], all = 0;
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int e = threadIdx.x * EACH + i;
    n[i] = 0;
    if (e < experts) {
      const ExpertRows r(offsets, e, rows);
      n[i] = (r.to - r.from) / G + ((r.to - r.from) % G != 0);
    }
    all += n[i];
  }
  int32_t s = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  if (lane == 31) sums[w] = s;
  __syncthreads();
  for (int i = 0; i < w; ++i) s += sums[i];
  s -= all;
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int e = threadIdx.x * EACH + i;
    if (e < experts) first[e] = s;
    s += n[i];
    if (e == experts - 1) first[experts] = s;
  }
}

// The expert that group g < first[experts] belongs to.
__device__ __forceinline__ int expert_of(const int32_t* first, int experts, int64_t g) {
  int lo = 0, hi = experts;  // first[lo] <= g < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (first[mid] <= g) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace grs
