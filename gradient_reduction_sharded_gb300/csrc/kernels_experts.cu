// Products of the experts: one linear map for each expert on rows sorted by
// expert, with the gradients of the rows and of the weights.
//
// bf16 goes to the tensor cores (kernels_experts_mma.cu); operands whose row
// distance is not a multiple of 16 bytes, which TMA wants, are laid out anew
// in the workspace first.  fp32 goes to the kernel here.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "api_util.h"
#include "device.cuh"
#include "experts.h"
#include "internal.h"
#include "launch.cuh"
#include "operators.cuh"

namespace grs {
namespace {

constexpr int EXP_THREADS = 256;
enum : int { SITE_EXP_ROW = 1 };

__device__ int exp_flags[FLAG_COUNT];

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
  ld->w = s->in_features;
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
cudaError_t exp_general(const grs_experts* s, const ExpLd& ld, const void* a, const void* b, const int32_t* offsets, void* o, void* stream) {
  if (kP == Product::kWeights && s->grad_dtype == GRS_DTYPE_BF16) return exp_general<kP, float, uint16_t>(s, ld, a, b, offsets, o, stream);
  return exp_general<kP, float, float>(s, ld, a, b, offsets, o, stream);
}

// --------------------------------------------------- bf16, rows laid out anew
__global__ void __launch_bounds__(EXP_THREADS) exp_pad_kernel(const uint16_t* __restrict__ from, int64_t ld, uint16_t* __restrict__ to,
                                                              int64_t ld_to, int64_t rows, int32_t width) {
  pdl_wait();
  pdl_trigger();
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
    for (int32_t i = threadIdx.x; i < width; i += EXP_THREADS) to[r * ld_to + i] = from[r * ld + i];
}

int64_t round8(int64_t n) { return (n + 7) & ~int64_t(7); }

// Bytes of an operand's copy: none where its rows are whole 16-byte chunks apart.
int64_t pad_bytes(int64_t rows, int64_t ld, int64_t width) { return ld % 8 == 0 ? 0 : rows * round8(width) * 2; }

// `p` itself, or its copy at *ws; *ld becomes the copy's.
const void* pad_rows(const void* p, int64_t rows, int64_t* ld, int64_t width, uint8_t** ws, void* stream, cudaError_t* e) {
  const int64_t bytes = pad_bytes(rows, *ld, width);
  if (bytes == 0 || *e != cudaSuccess) return p;
  uint16_t* to = reinterpret_cast<uint16_t*>(*ws);
  *e = launch_pdl(exp_pad_kernel, dim3(static_cast<unsigned>(rows < 152 * 8 ? rows : 152 * 8)), dim3(EXP_THREADS), 0, stream,
                  static_cast<const uint16_t*>(p), *ld, to, round8(width), rows, static_cast<int32_t>(width));
  *ws += (bytes + 15) & ~int64_t(15);
  *ld = round8(width);
  return to;
}

int64_t exp_workspace(const grs_experts* s, const ExpLd& ld) {
  if (s->dtype == GRS_DTYPE_FP32) return 0;
  auto up = [](int64_t b) { return (b + 15) & ~int64_t(15); };
  return up(pad_bytes(s->rows, ld.x, s->in_features)) + up(pad_bytes(s->rows, ld.y, s->out_features)) +
         up(pad_bytes(int64_t(s->experts) * s->out_features, ld.w, s->in_features));
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
  if (e == cudaSuccess) e = take_experts_mma_flags(flags, st);
  if (e == cudaSuccess) e = take_embedding_flags(flags, st);
  if (e == cudaSuccess) e = take_qk_norm_flags(flags, st);
  if (e != cudaSuccess) return api_cuda_fail(e, who);
  if (flags[FLAG_BOUNDS] != 0) return api_fail(GRS_ERR_BOUNDS, who, "an index out of place");
  return flags[FLAG_TIMEOUT] != 0 ? api_fail(GRS_ERR_TIMEOUT, who, "a bounded device wait timed out") : GRS_OK;
}

int64_t grs_experts_workspace_bytes(const grs_experts* s) {
  ExpLd ld;
  if (check_experts(s, "grs_experts_workspace_bytes", &ld) != GRS_OK) return -1;
  return exp_workspace(s, ld);
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
  if (workspace == nullptr && exp_workspace(s, ld) > 0) return api_fail(GRS_ERR_INVALID_ARG, who, "these row distances need a workspace");
  cudaError_t e = cudaSuccess;
  if (s->dtype == GRS_DTYPE_FP32) {
    e = exp_general<Product::kForward>(s, ld, w, xs, offsets, ys, stream);
  } else {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const int64_t ld_y = ld.y;
    xs = pad_rows(xs, s->rows, &ld.x, s->in_features, &ws, stream, &e);
    w = pad_rows(w, int64_t(s->experts) * s->out_features, &ld.w, s->in_features, &ws, stream, &e);
    if (e == cudaSuccess) e = experts_mma(Product::kForward, s, ld, xs, w, nullptr, offsets, ys, ld_y, stream);
  }
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
  if (workspace == nullptr && exp_workspace(s, ld) > 0) return api_fail(GRS_ERR_INVALID_ARG, who, "these row distances need a workspace");
  cudaError_t e = cudaSuccess;
  if (s->dtype == GRS_DTYPE_FP32) {
    if (dxs != nullptr) e = exp_general<Product::kRows>(s, ld, w, dys, offsets, dxs, stream);
    if (e == cudaSuccess && dw != nullptr) e = exp_general<Product::kWeights>(s, ld, xs, dys, offsets, dw, stream);
  } else if (dxs != nullptr || dw != nullptr) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const int64_t ld_x = ld.x;
    dys = pad_rows(dys, s->rows, &ld.y, s->out_features, &ws, stream, &e);
    if (dxs != nullptr) {
      w = pad_rows(w, int64_t(s->experts) * s->out_features, &ld.w, s->in_features, &ws, stream, &e);
      if (e == cudaSuccess) e = experts_mma(Product::kRows, s, ld, nullptr, w, dys, offsets, dxs, ld_x, stream);
    }
    if (dw != nullptr) {
      xs = pad_rows(xs, s->rows, &ld.x, s->in_features, &ws, stream, &e);
      if (e == cudaSuccess) e = experts_mma(Product::kWeights, s, ld, xs, nullptr, dys, offsets, dw, s->in_features, stream);
    }
  }
  return e == cudaSuccess ? GRS_OK : api_cuda_fail(e, who);
}

}  // extern "C"
