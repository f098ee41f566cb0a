// Root-mean-square norms of query and key heads with the rotation by position
// in the same pass, forward and backward.
//
// A head x of D elements: r = 1 / sqrt(sum x^2 / D + eps), h = x r, u = h w,
// and the first elements of u in pairs (a, b) turned by the position's angle.
// Backward turns the gradient back, so du = R^T dy, and with dh = du w
//   dx = r (dh - h sum(dh h) / D),   dw = sum over tokens and heads of du h.
// r is computed again from x, which backward reads in any case.
//
// Angles: a frequency is a fraction of a turn in 64 bits, and a position times
// it modulo 2^64 the fraction of its angle, without rounding at any position;
// its upper 32 bits go to sincospi.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "api_util.h"
#include "device.cuh"
#include "internal.h"
#include "launch.cuh"
#include "operators.cuh"

namespace grs {
namespace {

constexpr int QK_THREADS = 256;
constexpr int QK_WARPS = QK_THREADS / 32;
constexpr int QK_BLOCKS = 4 * 152;  // of the backward pass at most: the parts of dwq and dwk
enum : int { SITE_QK_HEAD = 1 };

__device__ int qk_flags[FLAG_COUNT];

template <typename T, typename P>
struct QkArgs {
  const T *x[2], *dy[2];  // queries, keys; gradients of the outputs
  T* o[2];                // outputs, or dq and dk (may be null)
  const P* w[2];          // may be null
  const int32_t* positions;
  const uint64_t* turns;
  float* parts;           // [blocks][2][D], or null
  int64_t ld_x[2], ld_y[2];  // ld_y: of outputs and their gradients
  int64_t tokens;
  int32_t heads[2];
  int32_t d, rot, pairs;
  float eps, inv_d;
};

__device__ __forceinline__ float2 turn_of(int32_t position, uint64_t turns) {
  const uint64_t a = static_cast<uint64_t>(int64_t(position)) * turns + 0x80000000u;
  float2 cs;
  sincospif(static_cast<float>(static_cast<int32_t>(a >> 32)) * 0x1p-31f, &cs.y, &cs.x);
  return cs;
}

// A warp's head: which token, whether a query (0) or a key (1), and its place.
template <typename T, typename P>
struct Head {
  int64_t t;
  int which;
  const T* x;
  __device__ __forceinline__ Head(const QkArgs<T, P>& a, int64_t item) {
    const int32_t all = a.heads[0] + a.heads[1];
    t = item / all;
    int32_t h = static_cast<int32_t>(item - t * all);
    which = h >= a.heads[0];
    if (which) h -= a.heads[0];
    off_x = t * a.ld_x[which] + int64_t(h) * a.d;
    off_y = t * a.ld_y[which] + int64_t(h) * a.d;
    x = a.x[which] + off_x;
  }
  int64_t off_x, off_y;
};

// f(element, element, cos, sin) for each of the lane's pairs, then g(element) for each of its others.
template <typename T, typename P, typename F, typename G>
__device__ __forceinline__ void each(const QkArgs<T, P>& a, int64_t t, int lane, bool angles, F&& f, G&& g) {
  const int half = a.rot / 2;
  const int32_t pos = half > 0 && angles ? __ldg(a.positions + t) : 0;
  for (int p = lane; p < half; p += 32) {
    const float2 cs = angles ? turn_of(pos, __ldg(a.turns + p)) : make_float2(1.0f, 0.0f);
    const int i = a.pairs ? 2 * p : p, j = a.pairs ? 2 * p + 1 : p + half;
    f(i, j, cs.x, cs.y);
  }
  for (int i = a.rot + lane; i < a.d; i += 32) g(i);
}

template <typename T, typename P>
__device__ __forceinline__ float weight(const QkArgs<T, P>& a, int which, int i) {
  return a.w[which] != nullptr ? to_float(__ldg(a.w[which] + i)) : 1.0f;
}

template <typename T, typename P>
__device__ __forceinline__ float head_rstd(const QkArgs<T, P>& a, const T* x, int lane) {
  float s = 0.0f;
  for (int i = lane; i < a.d; i += 32) {
    const float v = to_float(x[i]);
    s = __fmaf_rn(v, v, s);
  }
  return 1.0f / sqrtf(__fmaf_rn(warp_sum(s), a.inv_d, a.eps));
}

// Any dimension and alignment: a warp a head.  A lane reads again and writes
// the elements that are its own, after the sum over all: so in place as well.
template <typename T, typename P>
__global__ void __launch_bounds__(QK_THREADS) qk_forward_kernel(const __grid_constant__ QkArgs<T, P> a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t item = int64_t(blockIdx.x) * QK_WARPS + (threadIdx.x >> 5);
  if (item >= a.tokens * (a.heads[0] + a.heads[1])) return;
  const Head<T, P> h(a, item);
  if (!GRS_CHECK(h.t >= 0 && h.t < a.tokens, qk_flags, SITE_QK_HEAD)) return;
  const T* x = h.x;
  T* y = a.o[h.which] + h.off_y;
  const float r = head_rstd(a, x, lane);
  each(
      a, h.t, lane, true,
      [&](int i, int j, float c, float s) {
        const float u = to_float(x[i]) * r * weight(a, h.which, i), v = to_float(x[j]) * r * weight(a, h.which, j);
        y[i] = from_float<T>(u * c - v * s);
        y[j] = from_float<T>(u * s + v * c);
      },
      [&](int i) { y[i] = from_float<T>(to_float(x[i]) * r * weight(a, h.which, i)); });
}

template <typename T, typename P>
__global__ void __launch_bounds__(QK_THREADS) qk_backward_kernel(const __grid_constant__ QkArgs<T, P> a) {
  extern __shared__ float sums[];  // [warps][2][D]: each warp's dwq and dwk, an element always by the same lane
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, d = a.d;
  float* mine = sums + w * 2 * d;
  for (int i = lane; i < 2 * d; i += 32) mine[i] = 0.0f;
  __syncwarp();
  const int64_t items = a.tokens * (a.heads[0] + a.heads[1]);
  for (int64_t item = int64_t(blockIdx.x) * QK_WARPS + w; item < items; item += int64_t(gridDim.x) * QK_WARPS) {
    const Head<T, P> h(a, item);
    if (!GRS_CHECK(h.t >= 0 && h.t < a.tokens, qk_flags, SITE_QK_HEAD)) continue;
    const T *x = h.x, *dy = a.dy[h.which] + h.off_y;
    const float r = head_rstd(a, x, lane);
    float* dw = mine + h.which * d;
    float dot = 0.0f;
    each(
        a, h.t, lane, true,
        [&](int i, int j, float c, float s) {
          const float p = to_float(dy[i]), q = to_float(dy[j]);
          const float du = p * c + q * s, dv = q * c - p * s, hu = to_float(x[i]) * r, hv = to_float(x[j]) * r;
          dw[i] += du * hu;
          dw[j] += dv * hv;
          dot += du * weight(a, h.which, i) * hu + dv * weight(a, h.which, j) * hv;
        },
        [&](int i) {
          const float du = to_float(dy[i]), hu = to_float(x[i]) * r;
          dw[i] += du * hu;
          dot += du * weight(a, h.which, i) * hu;
        });
    const float m = warp_sum(dot) * a.inv_d;
    if (a.o[h.which] == nullptr) continue;
    T* dx = a.o[h.which] + h.off_x;
    each(
        a, h.t, lane, true,
        [&](int i, int j, float c, float s) {
          const float p = to_float(dy[i]), q = to_float(dy[j]);
          const float du = p * c + q * s, dv = q * c - p * s, hu = to_float(x[i]) * r, hv = to_float(x[j]) * r;
          dx[i] = from_float<T>(r * (du * weight(a, h.which, i) - hu * m));
          dx[j] = from_float<T>(r * (dv * weight(a, h.which, j) - hv * m));
        },
        [&](int i) {
          dx[i] = from_float<T>(r * (to_float(dy[i]) * weight(a, h.which, i) - to_float(x[i]) * r * m));
        });
  }
  if (a.parts == nullptr) return;
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * d; i += QK_THREADS) {
    float s = sums[i];
    for (int k = 1; k < QK_WARPS; ++k) s += sums[k * 2 * d + i];
    a.parts[int64_t(blockIdx.x) * 2 * d + i] = s;
  }
}

// dwq and dwk: a warp an element, the blocks' parts in a fixed order.
template <typename G>
__global__ void __launch_bounds__(QK_THREADS) qk_weights_kernel(const float* __restrict__ parts, int n, int d, G* dwq, G* dwk) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, i = blockIdx.x * QK_WARPS + (threadIdx.x >> 5);
  if (i >= 2 * d) return;
  float s = 0.0f;
  for (int k = lane; k < n; k += 32) s += parts[int64_t(k) * 2 * d + i];
  s = warp_sum(s);
  G* o = i < d ? dwq : dwk;
  if (lane == 0 && o != nullptr) o[i < d ? i : i - d] = from_float<G>(s);
}

// ------------------------------------------------------------------- host
grs_status check_qk(const grs_qk_norm* s, const char* who, int64_t (&ld)[4]) {
  if (s == nullptr) return api_fail(GRS_ERR_INVALID_ARG, who, "shape is NULL");
  if (s->tokens < 0 || s->q_heads < 0 || s->k_heads < 0 || s->head_dim < 1 || s->head_dim > GRS_QK_MAX_DIM)
    return api_fail(GRS_ERR_SHAPE, who, "tokens and heads must be >= 0 and head_dim in [1, GRS_QK_MAX_DIM]");
  if ((int64_t(s->q_heads) + s->k_heads) * s->head_dim > GRS_MAX_WIDTH || s->tokens > (int64_t(1) << 40))
    return api_fail(GRS_ERR_SHAPE, who, "more than GRS_MAX_WIDTH elements a token, or 2^40 tokens");
  if (s->rotary_dim < 0 || s->rotary_dim > s->head_dim || s->rotary_dim % 2 != 0)
    return api_fail(GRS_ERR_SHAPE, who, "rotary_dim must be even and in [0, head_dim]");
  if (s->interleaved != 0 && s->interleaved != 1) return api_fail(GRS_ERR_INVALID_ARG, who, "interleaved must be 0 or 1");
  if (!(s->eps >= 0.0f)) return api_fail(GRS_ERR_INVALID_ARG, who, "eps must be >= 0");
  if (!dtype_ok(s->dtype) || !dtype_ok(s->param_dtype) || !dtype_ok(s->grad_dtype))
    return api_fail(GRS_ERR_INVALID_ARG, who, "unknown element type");
  const int64_t given[4] = {s->ld_q, s->ld_k, s->ld_qo, s->ld_ko};
  for (int i = 0; i < 4; ++i) {
    const int64_t row = int64_t(i % 2 == 0 ? s->q_heads : s->k_heads) * s->head_dim;
    ld[i] = given[i] == 0 ? row : given[i];
    if (ld[i] < row || ld[i] > (int64_t(1) << 40)) return api_fail(GRS_ERR_SHAPE, who, "a distance of tokens below their heads' elements");
  }
  return GRS_OK;
}

int qk_blocks(const grs_qk_norm* s) {
  const int64_t b = (s->tokens * (s->q_heads + s->k_heads) + QK_WARPS - 1) / QK_WARPS;
  return static_cast<int>(b < QK_BLOCKS ? b : QK_BLOCKS);
}

template <typename T, typename P>
QkArgs<T, P> qk_args(const grs_qk_norm* s, const int64_t (&ld)[4], const void* dqo, const void* dko, const void* q, const void* k,
                     const void* wq, const void* wk, const int32_t* positions, const uint64_t* turns, void* oq, void* ok, void* parts) {
  QkArgs<T, P> a{};
  a.x[0] = static_cast<const T*>(q);
  a.x[1] = static_cast<const T*>(k);
  a.dy[0] = static_cast<const T*>(dqo);
  a.dy[1] = static_cast<const T*>(dko);
  a.o[0] = static_cast<T*>(oq);
  a.o[1] = static_cast<T*>(ok);
  a.w[0] = static_cast<const P*>(wq);
  a.w[1] = static_cast<const P*>(wk);
  a.positions = positions;
  a.turns = turns;
  a.parts = static_cast<float*>(parts);
  a.ld_x[0] = ld[0];
  a.ld_x[1] = ld[1];
  a.ld_y[0] = ld[2];
  a.ld_y[1] = ld[3];
  a.tokens = s->tokens;
  a.heads[0] = s->q_heads;
  a.heads[1] = s->k_heads;
  a.d = s->head_dim;
  a.rot = s->rotary_dim;
  a.pairs = s->interleaved;
  a.eps = s->eps;
  a.inv_d = 1.0f / static_cast<float>(s->head_dim);
  return a;
}

template <typename T, typename P>
cudaError_t qk_forward(const grs_qk_norm* s, const QkArgs<T, P>& a, void* stream) {
  const int64_t blocks = (s->tokens * (s->q_heads + s->k_heads) + QK_WARPS - 1) / QK_WARPS;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  return launch_pdl(qk_forward_kernel<T, P>, dim3(static_cast<unsigned>(blocks)), dim3(QK_THREADS), 0, stream, a);
}

template <typename T, typename P>
cudaError_t qk_backward(const grs_qk_norm* s, const QkArgs<T, P>& a, void* dwq, void* dwk, void* stream) {
  const int blocks = qk_blocks(s);
  cudaError_t e = allow_smem<qk_backward_kernel<T, P>>(QK_WARPS * 2 * GRS_QK_MAX_DIM * 4);
  if (e == cudaSuccess)
    e = launch_pdl(qk_backward_kernel<T, P>, dim3(blocks), dim3(QK_THREADS), size_t(QK_WARPS) * 2 * s->head_dim * 4, stream, a);
  if (e != cudaSuccess || a.parts == nullptr) return e;
  const dim3 grid((2 * s->head_dim + QK_WARPS - 1) / QK_WARPS), block(QK_THREADS);
  return s->grad_dtype == GRS_DTYPE_FP32
             ? launch_pdl(qk_weights_kernel<float>, grid, block, 0, stream, static_cast<const float*>(a.parts), blocks, s->head_dim,
                          static_cast<float*>(dwq), static_cast<float*>(dwk))
             : launch_pdl(qk_weights_kernel<uint16_t>, grid, block, 0, stream, static_cast<const float*>(a.parts), blocks, s->head_dim,
                          static_cast<uint16_t*>(dwq), static_cast<uint16_t*>(dwk));
}

}  // namespace

cudaError_t take_qk_norm_flags(int (&total)[FLAG_COUNT], cudaStream_t st) { return take_flags(qk_flags, total, st); }

}  // namespace grs

using namespace grs;

extern "C" {

grs_status grs_rope_turns(const double* inv_freq, int32_t n, uint64_t* turns) {
  static const char who[] = "grs_rope_turns";
  if (n < 0 || (n > 0 && (inv_freq == nullptr || turns == nullptr))) return api_fail(GRS_ERR_INVALID_ARG, who, "NULL argument or n < 0");
  for (int32_t i = 0; i < n; ++i) {
    if (!std::isfinite(inv_freq[i])) return api_fail(GRS_ERR_INVALID_ARG, who, "a frequency that is not finite");
    double f = inv_freq[i] / 6.283185307179586476925;
    f -= std::floor(f);                          // exact for f >= 0; [0, 1], 1 by rounding of a tiny negative f
    const double hi = std::floor(f * 0x1p32);    // two halves: 2^64 itself does not fit
    turns[i] = (static_cast<uint64_t>(hi) << 32) + static_cast<uint64_t>(std::floor((f * 0x1p32 - hi) * 0x1p32 + 0.5));
  }
  return GRS_OK;
}

int64_t grs_qk_norm_workspace_bytes(const grs_qk_norm* s) {
  int64_t ld[4];
  if (check_qk(s, "grs_qk_norm_workspace_bytes", ld) != GRS_OK) return -1;
  return int64_t(qk_blocks(s)) * 2 * s->head_dim * 4;
}

grs_status grs_qk_norm_forward(const grs_qk_norm* s, const void* q, const void* k, const void* wq, const void* wk,
                               const int32_t* positions, const uint64_t* turns, void* qo, void* ko, void* stream) {
  static const char who[] = "grs_qk_norm_forward";
  int64_t ld[4];
  const grs_status st = check_qk(s, who, ld);
  if (st != GRS_OK) return st;
  if (s->tokens == 0 || s->q_heads + s->k_heads == 0) return GRS_OK;
  if ((s->q_heads > 0 && (q == nullptr || qo == nullptr)) || (s->k_heads > 0 && (k == nullptr || ko == nullptr)) ||
      (s->rotary_dim > 0 && (positions == nullptr || turns == nullptr)))
    return api_fail(GRS_ERR_INVALID_ARG, who, "NULL argument");
  if ((q == qo && s->q_heads > 0 && ld[0] != ld[2]) || (k == ko && s->k_heads > 0 && ld[1] != ld[3]))
    return api_fail(GRS_ERR_INVALID_ARG, who, "in place with two distances of tokens");
  const uintptr_t ea = dtype_size(s->dtype), pa = dtype_size(s->param_dtype);
  if (!api_aligned(q, ea) || !api_aligned(k, ea) || !api_aligned(qo, ea) || !api_aligned(ko, ea) || !api_aligned(wq, pa) ||
      !api_aligned(wk, pa) || !api_aligned(positions, 4) || !api_aligned(turns, 8))
    return api_fail(GRS_ERR_ALIGNMENT, who, "a pointer is not aligned to its element");
  const bool f = s->dtype == GRS_DTYPE_FP32, pf = s->param_dtype == GRS_DTYPE_FP32;
#define GRS_QK_CALL(T, P) qk_forward<T, P>(s, qk_args<T, P>(s, ld, nullptr, nullptr, q, k, wq, wk, positions, turns, qo, ko, nullptr), stream)
  const cudaError_t e = f ? (pf ? GRS_QK_CALL(float, float) : GRS_QK_CALL(float, uint16_t))
                          : (pf ? GRS_QK_CALL(uint16_t, float) : GRS_QK_CALL(uint16_t, uint16_t));
#undef GRS_QK_CALL
  return e == cudaSuccess ? GRS_OK : api_cuda_fail(e, who);
}

grs_status grs_qk_norm_backward(const grs_qk_norm* s, const void* dqo, const void* dko, const void* q, const void* k, const void* wq,
                                const void* wk, const int32_t* positions, const uint64_t* turns, void* dq, void* dk, void* dwq, void* dwk,
                                void* workspace, void* stream) {
  static const char who[] = "grs_qk_norm_backward";
  int64_t ld[4];
  const grs_status st = check_qk(s, who, ld);
  if (st != GRS_OK) return st;
  const bool some = s->tokens > 0 && s->q_heads + s->k_heads > 0, params = dwq != nullptr || dwk != nullptr;
  if (some && ((s->q_heads > 0 && (q == nullptr || dqo == nullptr)) || (s->k_heads > 0 && (k == nullptr || dko == nullptr)) ||
               (s->rotary_dim > 0 && (positions == nullptr || turns == nullptr)) || (params && workspace == nullptr)))
    return api_fail(GRS_ERR_INVALID_ARG, who, "NULL argument");
  if ((dq != nullptr && dq == dqo && ld[0] != ld[2]) || (dk != nullptr && dk == dko && ld[1] != ld[3]))
    return api_fail(GRS_ERR_INVALID_ARG, who, "in place with two distances of tokens");
  const uintptr_t ea = dtype_size(s->dtype), pa = dtype_size(s->param_dtype), ga = dtype_size(s->grad_dtype);
  if (!api_aligned(q, ea) || !api_aligned(k, ea) || !api_aligned(dqo, ea) || !api_aligned(dko, ea) || !api_aligned(dq, ea) ||
      !api_aligned(dk, ea) || !api_aligned(wq, pa) || !api_aligned(wk, pa) || !api_aligned(dwq, ga) || !api_aligned(dwk, ga) ||
      !api_aligned(positions, 4) || !api_aligned(turns, 8) || !api_aligned(workspace, 16))
    return api_fail(GRS_ERR_ALIGNMENT, who, "a misaligned pointer");
  cudaError_t e = cudaSuccess;
  if (!some) {
    const size_t bytes = size_t(s->head_dim) * ga;
    if (dwq != nullptr) e = cudaMemsetAsync(dwq, 0, bytes, static_cast<cudaStream_t>(stream));
    if (e == cudaSuccess && dwk != nullptr) e = cudaMemsetAsync(dwk, 0, bytes, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GRS_OK : api_cuda_fail(e, who);
  }
  void* parts = params ? workspace : nullptr;
  const bool f = s->dtype == GRS_DTYPE_FP32, pf = s->param_dtype == GRS_DTYPE_FP32;
#define GRS_QK_CALL(T, P) \
  qk_backward<T, P>(s, qk_args<T, P>(s, ld, dqo, dko, q, k, wq, wk, positions, turns, dq, dk, parts), dwq, dwk, stream)
  e = f ? (pf ? GRS_QK_CALL(float, float) : GRS_QK_CALL(float, uint16_t))
        : (pf ? GRS_QK_CALL(uint16_t, float) : GRS_QK_CALL(uint16_t, uint16_t));
#undef GRS_QK_CALL
  return e == cudaSuccess ? GRS_OK : api_cuda_fail(e, who);
}

}  // extern "C"
