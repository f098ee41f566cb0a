// Products of the experts: one linear map for each expert on rows sorted by
// expert, with the gradients of the rows and of the weights.
//
// Every product is O[c][f] = sum over k of A[f][k] B[c][k] for each expert:
//   forward   f an output feature of w,  c a row, k an input feature
//   rows      f an input feature of w,   c a row, k an output feature
//   weights   f an input feature of xs,  c an output feature of dys, k a row
// so that f is what lies next to one another in the result and the expert's
// rows, of which only the device knows how many, are c or k.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "api_util.h"
#include "device.cuh"
#include "internal.h"
#include "launch.cuh"
#include "operators.cuh"

namespace grs {
namespace {

constexpr int EXP_THREADS = 256;
enum : int { SITE_EXP_ROW = 1 };

__device__ int exp_flags[FLAG_COUNT];

enum class Product { kForward, kRows, kWeights };

// An expert's rows, as the caller's offsets say within [0, rows].
struct Span2 {
  int32_t from, to;
};
__device__ __forceinline__ Span2 expert_rows(const int32_t* offsets, int e, int32_t rows) {
  int32_t a = __ldg(offsets + e), b = __ldg(offsets + e + 1);
  a = a < 0 ? 0 : a > rows ? rows : a;
  b = b < a ? a : b > rows ? rows : b;
  return {a, b};
}

// ------------------------------------------------------- any size and type
constexpr int GT = 64, GK = 16;  // tile of the result, elements of a step

template <typename T, typename O>
struct GeneralArgs {
  const T *a, *b;
  O* o;
  const int32_t* offsets;
  int64_t a_f, a_k, a_e;  // distances in A of features, of k, of experts
  int64_t b_c, b_k, b_e;
  int64_t o_c, o_e;
  int64_t f, c, k;        // extents; c or k of an expert's own are its rows
  int32_t rows, experts;
};

// Sums of 64 products are added up to the result's: shorter chains, errors
// that grow with 64 + k / 64 additions instead of k.
template <Product kP, typename T, typename O>
__global__ void __launch_bounds__(EXP_THREADS) exp_general_kernel(const __grid_constant__ GeneralArgs<T, O> p) {
  __shared__ float as[GK][GT + 4], bs[GK][GT + 4];
  __shared__ int32_t first[GRS_MOE_MAX_EXPERTS + 1];  // tiles of c before each expert's
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) {
    int32_t n = 0;
    for (int e = 0; e < p.experts; ++e) {
      first[e] = n;
      const Span2 r = expert_rows(p.offsets, e, p.rows);
      n += kP == Product::kWeights ? static_cast<int32_t>((p.c + GT - 1) / GT) : (r.to - r.from + GT - 1) / GT;
    }
    first[p.experts] = n;
  }
  __syncthreads();
  const int64_t ft = (p.f + GT - 1) / GT, tiles = ft * first[p.experts];
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;  // 4 features and 4 c of a thread
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int32_t ct = static_cast<int32_t>(tile / ft);
    const int64_t f0 = (tile - ct * ft) * GT;
    int lo = 0, hi = p.experts;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (first[mid] <= ct) lo = mid;
      else hi = mid;
    }
    while (first[lo + 1] <= ct) ++lo;
    const Span2 r = expert_rows(p.offsets, lo, p.rows);
    int64_t c0 = int64_t(ct - first[lo]) * GT, c1 = p.c, k0 = 0, k1 = p.k;
    if (kP == Product::kWeights) {
      k0 = r.from;
      k1 = r.to;
    } else {
      c0 += r.from;
      c1 = r.to;
    }
    const T *a = p.a + lo * p.a_e, *b = p.b + lo * p.b_e;
    float total[4][4] = {}, part[4][4] = {};
    int steps = 0;
    for (int64_t k = k0; k < k1; k += GK) {
      for (int i = threadIdx.x; i < GT * GK; i += EXP_THREADS) {
        // Neighbouring threads along what lies next to one another.
        const int fa = p.a_k == 1 ? i / GK : i % GT, ka = p.a_k == 1 ? i % GK : i / GT;
        as[ka][fa] = f0 + fa < p.f && k + ka < k1 ? to_float(a[(f0 + fa) * p.a_f + (k + ka) * p.a_k]) : 0.0f;
        const int cb = p.b_k == 1 ? i / GK : i % GT, kb = p.b_k == 1 ? i % GK : i / GT;
        bs[kb][cb] = c0 + cb < c1 && k + kb < k1 ? to_float(b[(c0 + cb) * p.b_c + (k + kb) * p.b_k]) : 0.0f;
      }
      __syncthreads();
#pragma unroll
      for (int q = 0; q < GK; ++q) {
        float u[4], v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          u[i] = as[q][tx * 4 + i];
          v[i] = bs[q][ty * 4 + i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) part[i][j] = __fmaf_rn(v[i], u[j], part[i][j]);
      }
      if (++steps % 4 == 0)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            total[i][j] += part[i][j];
            part[i][j] = 0.0f;
          }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t c = c0 + ty * 4 + i, f = f0 + tx * 4 + j;
        if (c < c1 && f < p.f && GRS_CHECK(kP == Product::kWeights || c < p.rows, exp_flags, SITE_EXP_ROW))
          p.o[lo * p.o_e + c * p.o_c + f] = from_float<O>(total[i][j] + part[i][j]);
      }
  }
}

// ------------------------------------------------------------------- host
struct ExpLd {
  int64_t x, y;
};

grs_status check_experts(const grs_experts* s, const char* who, ExpLd* ld) {
  if (s == nullptr) return api_fail(GRS_ERR_INVALID_ARG, who, "shape is NULL");
  if (s->rows < 0 || s->rows > INT32_MAX) return api_fail(GRS_ERR_SHAPE, who, "rows must be in [0, 2^31)");
  if (s->experts < 1 || s->experts > GRS_MOE_MAX_EXPERTS) return api_fail(GRS_ERR_SHAPE, who, "experts must be in [1, GRS_MOE_MAX_EXPERTS]");
  if (s->in_features < 1 || s->out_features < 1 || s->in_features > GRS_MAX_WIDTH || s->out_features > GRS_MAX_WIDTH)
    return api_fail(GRS_ERR_SHAPE, who, "in_features and out_features must be in [1, GRS_MAX_WIDTH]");
  if (!dtype_ok(s->dtype) || !dtype_ok(s->grad_dtype)) return api_fail(GRS_ERR_INVALID_ARG, who, "unknown element type");
  ld->x = s->ld_x == 0 ? s->in_features : s->ld_x;
  ld->y = s->ld_y == 0 ? s->out_features : s->ld_y;
  if (ld->x < s->in_features || ld->y < s->out_features || ld->x > GRS_MAX_WIDTH || ld->y > GRS_MAX_WIDTH)
    return api_fail(GRS_ERR_SHAPE, who, "a distance of rows below their width or above GRS_MAX_WIDTH");
  return GRS_OK;
}

template <Product kP, typename T, typename O>
cudaError_t exp_general(const grs_experts* s, const ExpLd& ld, const void* a, const void* b, const int32_t* offsets, void* o, void* stream) {
  const int64_t in = s->in_features, out = s->out_features;
  GeneralArgs<T, O> p{};
  p.a = static_cast<const T*>(a);
  p.b = static_cast<const T*>(b);
  p.o = static_cast<O*>(o);
  p.offsets = offsets;
  p.rows = static_cast<int32_t>(s->rows);
  p.experts = s->experts;
  if (kP == Product::kForward) {  // A = w, B = xs
    p.a_f = in, p.a_k = 1, p.a_e = in * out, p.b_c = ld.x, p.b_k = 1, p.o_c = ld.y, p.f = out, p.k = in;
  } else if (kP == Product::kRows) {  // A = w, B = dys
    p.a_f = 1, p.a_k = in, p.a_e = in * out, p.b_c = ld.y, p.b_k = 1, p.o_c = ld.x, p.f = in, p.k = out;
  } else {  // A = xs, B = dys
    p.a_f = 1, p.a_k = ld.x, p.b_c = 1, p.b_k = ld.y, p.o_c = in, p.o_e = in * out, p.f = in, p.c = out;
  }
  return launch_pdl(exp_general_kernel<kP, T, O>, dim3(152 * 8), dim3(EXP_THREADS), 0, stream, p);
}

template <Product kP>
cudaError_t exp_run(const grs_experts* s, const ExpLd& ld, const void* a, const void* b, const int32_t* offsets, void* o, void* stream) {
  const bool f = s->dtype == GRS_DTYPE_FP32, g = kP == Product::kWeights ? s->grad_dtype == GRS_DTYPE_FP32 : f;
  if (f) return g ? exp_general<kP, float, float>(s, ld, a, b, offsets, o, stream) : exp_general<kP, float, uint16_t>(s, ld, a, b, offsets, o, stream);
  return g ? exp_general<kP, uint16_t, float>(s, ld, a, b, offsets, o, stream) : exp_general<kP, uint16_t, uint16_t>(s, ld, a, b, offsets, o, stream);
}

}  // namespace

cudaError_t take_experts_flags(int (&total)[FLAG_COUNT], cudaStream_t st) { return take_flags(exp_flags, total, st); }

}  // namespace grs

using namespace grs;

extern "C" {

grs_status grs_operators_check_device_errors(void* stream) {
  static const char who[] = "grs_operators_check_device_errors";
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  int flags[FLAG_COUNT] = {};
  cudaError_t e = cudaStreamSynchronize(st);
  if (e == cudaSuccess) e = take_experts_flags(flags, st);
  if (e == cudaSuccess) e = take_embedding_flags(flags, st);
  if (e == cudaSuccess) e = take_qk_norm_flags(flags, st);
  if (e != cudaSuccess) return api_cuda_fail(e, who);
  if (flags[FLAG_BOUNDS] != 0) return api_fail(GRS_ERR_BOUNDS, who, "an index out of place");
  return flags[FLAG_TIMEOUT] != 0 ? api_fail(GRS_ERR_TIMEOUT, who, "a bounded device wait timed out") : GRS_OK;
}

int64_t grs_experts_workspace_bytes(const grs_experts* s) {
  ExpLd ld;
  if (check_experts(s, "grs_experts_workspace_bytes", &ld) != GRS_OK) return -1;
  return 0;
}

grs_status grs_experts_forward(const grs_experts* s, const void* xs, const void* w, const int32_t* offsets, void* ys, void* workspace,
                               void* stream) {
  static const char who[] = "grs_experts_forward";
  ExpLd ld;
  const grs_status st = check_experts(s, who, &ld);
  if (st != GRS_OK) return st;
  if (s->rows == 0) return GRS_OK;
  if (xs == nullptr || w == nullptr || offsets == nullptr || ys == nullptr) return api_fail(GRS_ERR_INVALID_ARG, who, "NULL argument");
  if (!api_aligned(xs, 16) || !api_aligned(w, 16) || !api_aligned(offsets, 4) || !api_aligned(ys, dtype_size(s->dtype)) ||
      !api_aligned(workspace, 16))
    return api_fail(GRS_ERR_ALIGNMENT, who, "a misaligned pointer");
  const cudaError_t e = exp_run<Product::kForward>(s, ld, w, xs, offsets, ys, stream);
  return e == cudaSuccess ? GRS_OK : api_cuda_fail(e, who);
}

grs_status grs_experts_backward(const grs_experts* s, const void* dys, const void* xs, const void* w, const int32_t* offsets, void* dxs,
                                void* dw, void* workspace, void* stream) {
  static const char who[] = "grs_experts_backward";
  ExpLd ld;
  const grs_status st = check_experts(s, who, &ld);
  if (st != GRS_OK) return st;
  if (!api_aligned(dys, 16) || !api_aligned(xs, 16) || !api_aligned(w, 16) || !api_aligned(offsets, 4) ||
      !api_aligned(dxs, dtype_size(s->dtype)) || !api_aligned(dw, dtype_size(s->grad_dtype)) || !api_aligned(workspace, 16))
    return api_fail(GRS_ERR_ALIGNMENT, who, "a misaligned pointer");
  if (s->rows == 0) {
    if (dw == nullptr) return GRS_OK;
    const size_t bytes = size_t(s->experts) * s->in_features * s->out_features * dtype_size(s->grad_dtype);
    const cudaError_t e = cudaMemsetAsync(dw, 0, bytes, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GRS_OK : api_cuda_fail(e, who);
  }
  if (offsets == nullptr || (dys == nullptr && (dxs != nullptr || dw != nullptr)) || (w == nullptr && dxs != nullptr) ||
      (xs == nullptr && dw != nullptr))
    return api_fail(GRS_ERR_INVALID_ARG, who, "NULL argument");
  cudaError_t e = cudaSuccess;
  if (dxs != nullptr) e = exp_run<Product::kRows>(s, ld, w, dys, offsets, dxs, stream);
  if (e == cudaSuccess && dw != nullptr) e = exp_run<Product::kWeights>(s, ld, xs, dys, offsets, dw, stream);
  return e == cudaSuccess ? GRS_OK : api_cuda_fail(e, who);
}

}  // extern "C"
