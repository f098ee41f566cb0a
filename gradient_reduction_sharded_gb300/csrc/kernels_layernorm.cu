// Layer norm over rows, forward and backward.
//
//   mean = sum x / C,  var = sum (x - mean)^2 / C,  r = 1 / sqrt(var + eps)
//   h = (x - mean) r,  y = h w + b
//   dh = dy w,  dx = r (dh - mean_C(dh) - h mean_C(dh h))
//   dw = sum over rows of dy h,  db = sum over rows of dy
//
// All arithmetic and every sum in fp32; one rounding to the output's type.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "api_util.h"
#include "device.cuh"
#include "internal.h"
#include "launch.cuh"

namespace grs {
namespace {

constexpr int LN_THREADS = 256;
constexpr int LN_PARTS = 304;  // partial rows of dw and db at most

__device__ __forceinline__ float ln_load(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }
__device__ __forceinline__ float ln_load(const float* p) { return *p; }
__device__ __forceinline__ void ln_store(uint16_t* p, float x) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
__device__ __forceinline__ void ln_store(float* p, float x) { *p = x; }

// Sum over the block, the same bits for every thread; `red` holds one float a warp.
__device__ __forceinline__ float ln_block_sum(float x, float* red) {
  x = warp_sum(x);
  __syncthreads();  // red may still be read from the sum before
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  float s = red[0];
  for (int k = 1; k < LN_THREADS / 32; ++k) s = __fadd_rn(s, red[k]);
  return s;
}

// ------------------------------------------------ any width, any alignment
// One block a row, the row read again for each pass (it is in L2 by then).
template <typename T, typename W>
__global__ void __launch_bounds__(LN_THREADS) ln_fwd_any_kernel(const T* __restrict__ x, int64_t ld_x, const W* __restrict__ w,
                                                                const W* __restrict__ b, T* __restrict__ y, int64_t ld_y,
                                                                float* __restrict__ mean_out, float* __restrict__ rstd_out,
                                                                int64_t rows, int32_t cols, float eps) {
  __shared__ float red[LN_THREADS / 32];
  pdl_wait();
  pdl_trigger();
  const float inv_c = 1.0f / static_cast<float>(cols);
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* xr = x + row * ld_x;
    float s = 0.0f;
    for (int c = threadIdx.x; c < cols; c += LN_THREADS) s += ln_load(xr + c);
    const float mean = ln_block_sum(s, red) * inv_c;
    s = 0.0f;
    for (int c = threadIdx.x; c < cols; c += LN_THREADS) {
      const float d = ln_load(xr + c) - mean;
      s = fmaf(d, d, s);
    }
    const float rstd = 1.0f / sqrtf(ln_block_sum(s, red) * inv_c + eps);
    T* yr = y + row * ld_y;
    for (int c = threadIdx.x; c < cols; c += LN_THREADS) {
      const float h = (ln_load(xr + c) - mean) * rstd;
      ln_store(yr + c, fmaf(h, w != nullptr ? ln_load(w + c) : 1.0f, b != nullptr ? ln_load(b + c) : 0.0f));
    }
    if (threadIdx.x == 0) {
      if (mean_out != nullptr) mean_out[row] = mean;
      if (rstd_out != nullptr) rstd_out[row] = rstd;
    }
  }
}

template <typename T, typename W>
__global__ void __launch_bounds__(LN_THREADS) ln_dx_any_kernel(const T* __restrict__ dy, int64_t ld_dy, const T* __restrict__ x,
                                                               int64_t ld_x, const W* __restrict__ w,
                                                               const float* __restrict__ mean_in,
                                                               const float* __restrict__ rstd_in, T* __restrict__ dx,
                                                               int64_t ld_dx, int64_t rows, int32_t cols) {
  __shared__ float red[LN_THREADS / 32];
  pdl_wait();
  pdl_trigger();
  const float inv_c = 1.0f / static_cast<float>(cols);
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T *gr = dy + row * ld_dy, *xr = x + row * ld_x;
    const float mean = mean_in[row], rstd = rstd_in[row];
    float s1 = 0.0f, s2 = 0.0f;
    for (int c = threadIdx.x; c < cols; c += LN_THREADS) {
      const float dh = ln_load(gr + c) * (w != nullptr ? ln_load(w + c) : 1.0f);
      s1 += dh;
      s2 = fmaf(dh, (ln_load(xr + c) - mean) * rstd, s2);
    }
    s1 = ln_block_sum(s1, red) * inv_c;
    s2 = ln_block_sum(s2, red) * inv_c;
    T* dr = dx + row * ld_dx;
    for (int c = threadIdx.x; c < cols; c += LN_THREADS) {
      const float dh = ln_load(gr + c) * (w != nullptr ? ln_load(w + c) : 1.0f);
      const float h = (ln_load(xr + c) - mean) * rstd;
      ln_store(dr + c, rstd * (dh - s1 - h * s2));
    }
  }
}

// Partial sums of dw and db: part blockIdx.y takes rows blockIdx.y,
// blockIdx.y + parts, ..., a thread one column.
template <typename T>
__global__ void __launch_bounds__(LN_THREADS) ln_dparam_any_kernel(const T* __restrict__ dy, int64_t ld_dy,
                                                                   const T* __restrict__ x, int64_t ld_x,
                                                                   const float* __restrict__ mean_in,
                                                                   const float* __restrict__ rstd_in,
                                                                   float* __restrict__ parts, int64_t rows, int32_t cols) {
  pdl_wait();
  pdl_trigger();
  const int64_t c = int64_t(blockIdx.x) * LN_THREADS + threadIdx.x;
  if (c >= cols) return;
  float dw = 0.0f, db = 0.0f;
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    const float g = ln_load(dy + row * ld_dy + c);
    dw = fmaf(g, (ln_load(x + row * ld_x + c) - mean_in[row]) * rstd_in[row], dw);
    db += g;
  }
  float* p = parts + int64_t(blockIdx.y) * 2 * cols;
  p[c] = dw;
  p[cols + c] = db;
}

// dw and db from the parts, in the parts' order.  A block takes 32 of the
// 2 C sums, warp k of it the parts k, k + 8, ...
template <typename D>
__global__ void __launch_bounds__(LN_THREADS) ln_dparam_sum_kernel(const float* __restrict__ parts, int32_t n_parts,
                                                                   int32_t cols, D* __restrict__ dw, D* __restrict__ db) {
  __shared__ float red[LN_THREADS / 32][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int64_t c = int64_t(blockIdx.x) * 32 + lane, width = 2 * int64_t(cols);
  float s = 0.0f;
  if (c < width)
    for (int p = k; p < n_parts; p += LN_THREADS / 32) s += parts[p * width + c];
  red[k][lane] = s;
  __syncthreads();
  if (k != 0 || c >= width) return;
  for (int j = 1; j < LN_THREADS / 32; ++j) s += red[j][lane];
  D* out = c < cols ? dw : db;
  if (out != nullptr) ln_store(out + (c < cols ? c : c - cols), s);
}

int32_t ln_parts(int64_t rows) { return static_cast<int32_t>(rows < LN_PARTS ? (rows > 0 ? rows : 1) : LN_PARTS); }

struct LnLd {
  int64_t x, y, dy, dx;
};

grs_status check_norm(const grs_norm* s, const char* who, LnLd* ld) {
  if (s == nullptr) return api_fail(GRS_ERR_INVALID_ARG, who, "shape is NULL");
  if (s->rows < 0 || s->cols < 1) return api_fail(GRS_ERR_SHAPE, who, "rows must be >= 0 and cols >= 1");
  if (!dtype_ok(s->dtype) || !dtype_ok(s->param_dtype) || !dtype_ok(s->grad_dtype))
    return api_fail(GRS_ERR_INVALID_ARG, who, "unknown element type");
  if (!(s->eps >= 0.0f) || std::isinf(s->eps)) return api_fail(GRS_ERR_INVALID_ARG, who, "eps must be finite and >= 0");
  *ld = {s->ld_x ? s->ld_x : s->cols, s->ld_y ? s->ld_y : s->cols, s->ld_dy ? s->ld_dy : s->cols,
         s->ld_dx ? s->ld_dx : s->cols};
  if (ld->x < s->cols || ld->y < s->cols || ld->dy < s->cols || ld->dx < s->cols)
    return api_fail(GRS_ERR_SHAPE, who, "a leading dimension is less than cols");
  return GRS_OK;
}

template <typename T, typename W>
cudaError_t ln_forward(const grs_norm* s, const LnLd& ld, const void* x, const void* w, const void* b, void* y, float* mean,
                       float* rstd, void* stream) {
  const unsigned grid = static_cast<unsigned>(s->rows < 1 << 20 ? s->rows : 1 << 20);
  return launch_k(ln_fwd_any_kernel<T, W>, dim3(grid), dim3(LN_THREADS), 0, stream, static_cast<const T*>(x), ld.x,
                  static_cast<const W*>(w), static_cast<const W*>(b), static_cast<T*>(y), ld.y, mean, rstd, s->rows, s->cols,
                  s->eps);
}

template <typename T, typename W>
cudaError_t ln_backward(const grs_norm* s, const LnLd& ld, const void* dy, const void* x, const void* w, const float* mean,
                        const float* rstd, void* dx, void* dw, void* db, float* ws, void* stream) {
  cudaError_t e = cudaSuccess;
  if (dx != nullptr && s->rows > 0) {
    const unsigned grid = static_cast<unsigned>(s->rows < 1 << 20 ? s->rows : 1 << 20);
    e = launch_k(ln_dx_any_kernel<T, W>, dim3(grid), dim3(LN_THREADS), 0, stream, static_cast<const T*>(dy), ld.dy,
                 static_cast<const T*>(x), ld.x, static_cast<const W*>(w), mean, rstd, static_cast<T*>(dx), ld.dx, s->rows,
                 s->cols);
  }
  if (e != cudaSuccess || (dw == nullptr && db == nullptr)) return e;
  const int32_t parts = ln_parts(s->rows);
  e = launch_k(ln_dparam_any_kernel<T>, dim3((unsigned(s->cols) + LN_THREADS - 1) / LN_THREADS, unsigned(parts)),
               dim3(LN_THREADS), 0, stream, static_cast<const T*>(dy), ld.dy, static_cast<const T*>(x), ld.x, mean, rstd, ws,
               s->rows, s->cols);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>((2 * int64_t(s->cols) + 31) / 32));
  const float* parts_in = ws;
  return s->grad_dtype == GRS_DTYPE_FP32
             ? launch_k(ln_dparam_sum_kernel<float>, grid, dim3(LN_THREADS), 0, stream, parts_in, parts, s->cols,
                        static_cast<float*>(dw), static_cast<float*>(db))
             : launch_k(ln_dparam_sum_kernel<uint16_t>, grid, dim3(LN_THREADS), 0, stream, parts_in, parts, s->cols,
                        static_cast<uint16_t*>(dw), static_cast<uint16_t*>(db));
}

}  // namespace
}  // namespace grs

using namespace grs;

extern "C" {

int64_t grs_layernorm_workspace_bytes(const grs_norm* s) {
  LnLd ld;
  if (check_norm(s, "grs_layernorm_workspace_bytes", &ld) != GRS_OK) return -1;
  return int64_t(ln_parts(s->rows)) * 2 * s->cols * 4;
}

grs_status grs_layernorm_forward(const grs_norm* s, const void* x, const void* w, const void* b, void* y, float* mean,
                                 float* rstd, void* stream) {
  static const char who[] = "grs_layernorm_forward";
  LnLd ld;
  const grs_status st = check_norm(s, who, &ld);
  if (st != GRS_OK) return st;
  if (s->rows == 0) return GRS_OK;
  if (x == nullptr || y == nullptr) return api_fail(GRS_ERR_INVALID_ARG, who, "NULL argument");
  const uintptr_t ea = dtype_size(s->dtype), pa = dtype_size(s->param_dtype);
  if (!api_aligned(x, ea) || !api_aligned(y, ea) || !api_aligned(w, pa) || !api_aligned(b, pa) || !api_aligned(mean, 4) ||
      !api_aligned(rstd, 4))
    return api_fail(GRS_ERR_ALIGNMENT, who, "a pointer is not aligned to its element");
  const bool f = s->dtype == GRS_DTYPE_FP32, pf = s->param_dtype == GRS_DTYPE_FP32;
  const cudaError_t e = f ? (pf ? ln_forward<float, float>(s, ld, x, w, b, y, mean, rstd, stream)
                                : ln_forward<float, uint16_t>(s, ld, x, w, b, y, mean, rstd, stream))
                          : (pf ? ln_forward<uint16_t, float>(s, ld, x, w, b, y, mean, rstd, stream)
                                : ln_forward<uint16_t, uint16_t>(s, ld, x, w, b, y, mean, rstd, stream));
  return e == cudaSuccess ? GRS_OK : api_cuda_fail(e, who);
}

grs_status grs_layernorm_backward(const grs_norm* s, const void* dy, const void* x, const void* w, const float* mean,
                                  const float* rstd, void* dx, void* dw, void* db, void* workspace, void* stream) {
  static const char who[] = "grs_layernorm_backward";
  LnLd ld;
  const grs_status st = check_norm(s, who, &ld);
  if (st != GRS_OK) return st;
  const bool params = dw != nullptr || db != nullptr;
  if (s->rows > 0 && (dy == nullptr || x == nullptr || mean == nullptr || rstd == nullptr))
    return api_fail(GRS_ERR_INVALID_ARG, who, "NULL argument");
  if (params && workspace == nullptr) return api_fail(GRS_ERR_INVALID_ARG, who, "dw and db need a workspace");
  const uintptr_t ea = dtype_size(s->dtype), pa = dtype_size(s->param_dtype), ga = dtype_size(s->grad_dtype);
  if (!api_aligned(dy, ea) || !api_aligned(x, ea) || !api_aligned(dx, ea) || !api_aligned(w, pa) || !api_aligned(dw, ga) ||
      !api_aligned(db, ga) || !api_aligned(mean, 4) || !api_aligned(rstd, 4))
    return api_fail(GRS_ERR_ALIGNMENT, who, "a pointer is not aligned to its element");
  if (params && !api_aligned(workspace, 16)) return api_fail(GRS_ERR_ALIGNMENT, who, "workspace not 16-byte aligned");
  const bool f = s->dtype == GRS_DTYPE_FP32, pf = s->param_dtype == GRS_DTYPE_FP32;
  float* ws = static_cast<float*>(workspace);
  const cudaError_t e = f ? (pf ? ln_backward<float, float>(s, ld, dy, x, w, mean, rstd, dx, dw, db, ws, stream)
                                : ln_backward<float, uint16_t>(s, ld, dy, x, w, mean, rstd, dx, dw, db, ws, stream))
                          : (pf ? ln_backward<uint16_t, float>(s, ld, dy, x, w, mean, rstd, dx, dw, db, ws, stream)
                                : ln_backward<uint16_t, uint16_t>(s, ld, dy, x, w, mean, rstd, dx, dw, db, ws, stream));
  return e == cudaSuccess ? GRS_OK : api_cuda_fail(e, who);
}

}  // extern "C"
