// Error and device helpers of the C entry points outside api.cu (internal).
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <string>

#include "internal.h"

namespace grs {

inline grs_status api_fail(grs_status s, const char* who, const char* msg) {
  try {
    set_last_error(std::string(who) + ": " + msg);
  } catch (...) {  // no memory for the message: the status still says what failed
  }
  return s;
}

inline grs_status api_cuda_fail(int e, const char* who) {
  return api_fail(GRS_ERR_CUDA, who, cudaGetErrorString(static_cast<cudaError_t>(e)));
}

inline bool api_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Makes `dev` current for the scope and restores the caller's device.
class ApiDevice {
 public:
  explicit ApiDevice(int dev) {
    ok_ = cudaGetDevice(&prev_) == cudaSuccess;
    if (ok_ && prev_ != dev) {
      ok_ = cudaSetDevice(dev) == cudaSuccess;
      switched_ = ok_;
    }
  }
  ~ApiDevice() {
    if (switched_) cudaSetDevice(prev_);
  }
  ApiDevice(const ApiDevice&) = delete;
  ApiDevice& operator=(const ApiDevice&) = delete;
  bool ok() const { return ok_; }

 private:
  int prev_ = 0;
  bool ok_ = false, switched_ = false;
};

// Lets `Kernel` use up to `bytes` of dynamic shared memory on the current
// device; asked once a device, so that a call does not pay for it again.
template <auto* Kernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_release);
  return e;
}

inline bool dtype_ok(int32_t t) { return t == GRS_DTYPE_BF16 || t == GRS_DTYPE_FP32; }
inline int dtype_size(int32_t t) { return t == GRS_DTYPE_FP32 ? 4 : 2; }

}  // namespace grs
