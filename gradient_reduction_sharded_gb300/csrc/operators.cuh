// What the operators of kernels_experts, kernels_embedding and kernels_qk_norm
// share: elements of either type, device flags.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "device.cuh"
#include "packed.cuh"

namespace grs {

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(uint16_t x) { return __uint_as_float(uint32_t(x) << 16); }

template <typename T>
__device__ __forceinline__ T from_float(float x) {
  if constexpr (sizeof(T) == 4) return x;
  else return static_cast<uint16_t>(to_bf16_pair(make_float2(x, 0.0f)));
}

// N consecutive elements as fp32: 1, or 8 that start at a multiple of 16 bytes.
template <int N, typename T>
__device__ __forceinline__ void load_floats(const T* p, float (&o)[N]) {
  if constexpr (N == 1) {
    o[0] = to_float(__ldg(p));
  } else if constexpr (sizeof(T) == 2) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
    set_bf16x8(o, w);
  } else {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
    o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
  }
}

template <int N, typename T>
__device__ __forceinline__ void store_floats(T* p, const float (&v)[N]) {
  if constexpr (N == 1) {
    *p = from_float<T>(v[0]);
  } else if constexpr (sizeof(T) == 2) {
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(to_bf16_pair(make_float2(v[0], v[1])), to_bf16_pair(make_float2(v[2], v[3])),
                                                   to_bf16_pair(make_float2(v[4], v[5])), to_bf16_pair(make_float2(v[6], v[7]))));
  } else {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
  }
}

// The device flags (FLAG_COUNT ints) of each file on the current device.
cudaError_t experts_flags(int** at);
cudaError_t experts_mma_flags(int** at);
cudaError_t embedding_flags(int** at);
cudaError_t qk_norm_flags(int** at);

}  // namespace grs
