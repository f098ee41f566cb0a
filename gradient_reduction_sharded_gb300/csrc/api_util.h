// Error and device helpers of the C entry points outside api.cu (internal).
#pragma once

#include <cuda_runtime.h>

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

inline bool dtype_ok(int32_t t) { return t == GRS_DTYPE_BF16 || t == GRS_DTYPE_FP32; }
inline int dtype_size(int32_t t) { return t == GRS_DTYPE_FP32 ? 4 : 2; }

}  // namespace grs
