// Products of the experts: one linear map for each expert on rows sorted by
// expert, with the gradients of the rows and of the weights.
//
// bf16 goes to the tensor cores (kernels_experts_mma.cu); operands whose row
// distance is not a multiple of 16 bytes, which TMA wants, are laid out anew
// in the workspace first.  fp32 goes to the kernel here.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "api_util.h"
#include "device.cuh"
#include "experts.cuh"
#include "internal.h"
#include "launch.cuh"
#include "operators.cuh"

namespace grs {
namespace {

constexpr int EXP_THREADS = 256;
enum : int { SITE_EXP_ROW = 1 };

__device__ int exp_flags[FLAG_COUNT];

// --------------------------------------------------------- fp32, any size
// A block has 128 features of 64 c, a thread eight by eight, as pairs of
// neighbouring features.  Operands are read as single numbers, which turns
// either layout into [k][feature or c] in shared memory; the next 16 of k are in
// registers, the ones after on their way, while 16 are multiplied.  3000 rows, 8
// experts, 1024 -> 1024: forward 166 us, rows' gradients 160, weights' gradients
// 136 (38 to 46 TFLOP/s); 16384 rows 45 to 50.  Bound by reads of shared memory:
// four a thread and k for 32 additions of pairs; eight by four (three for 16)
// took 224, 215 and 182, copies of single numbers past the registers the same,
// every c twice in shared memory instead of moves 17 % more.
constexpr int GF = 128, GC = 64, GK = 16, G_THREADS = 128, G_PER_SM = 2;

template <typename O>
struct GeneralArgs {
  const float *a, *b;
  O* o;
  const int32_t* offsets;
  int64_t a_f, a_k, a_e;  // distances in A of features, of k, of experts
  int64_t b_c, b_k;
  int64_t o_c, o_e, o_s;  // distances of c, of experts, of slices
  int64_t f, c, k;        // extents; c or k of an expert's own are its rows
  int32_t rows, experts, slices;
};

// One operand's next GK x N elements: where a thread's lie and go.
// Neighbouring threads along what lies next to one another, k with kAlongK.
template <int N, bool kAlongK>
struct Panel {
  static constexpr int EACH = N * GK / G_THREADS;
  static constexpr int PER_K = G_THREADS / GK, PER_N = G_THREADS / N;  // between a thread's elements: in N, in k
  static constexpr int DAT = kAlongK ? PER_K : PER_N * (N + 4);        // in shared memory
  const float* p;      // the thread's first element of the next step
  int64_t next, step;  // elements to its next one, to the next step's
  int32_t k;           // of its first element
  uint32_t on;         // which of its elements exist along N
  uint32_t at;         // in shared memory
  bool whole;          // all of the panel's N exist
  float v[EACH];
  __device__ __forceinline__ Panel(const float* base, int64_t n0, int64_t n1, int64_t k0, int64_t ld_n, int64_t ld_k)
      : whole(n0 + N <= n1) {
    const int tk = kAlongK ? threadIdx.x % GK : threadIdx.x / N, tn = kAlongK ? threadIdx.x / GK : threadIdx.x % N;
    p = base + (n0 + tn) * ld_n + (k0 + tk) * ld_k;
    k = tk;
    next = kAlongK ? PER_K * ld_n : PER_N * ld_k;
    step = GK * ld_k;
    at = tk * (N + 4) + tn;
    on = 0;
#pragma unroll
    for (int j = 0; j < EACH; ++j) on |= uint32_t(n0 + tn + (kAlongK ? j * PER_K : 0) < n1) << j;
  }
  // The step whose first k has `rest` left; what is not there is zero.
  __device__ __forceinline__ void load(int64_t rest) {
    const float* q = p;
    if (whole && rest >= GK) {
#pragma unroll
      for (int j = 0; j < EACH; ++j, q += next) v[j] = __ldg(q);
    } else {
#pragma unroll
      for (int j = 0; j < EACH; ++j, q += next) v[j] = (on >> j & 1) != 0 && k + (kAlongK ? 0 : j * PER_N) < rest ? __ldg(q) : 0.0f;
    }
    p += step;
  }
  __device__ __forceinline__ void put(float* stage) const {
#pragma unroll
    for (int j = 0; j < EACH; ++j) stage[at + j * DAT] = v[j];
  }
};

// Sums of 64 products are added up to the result's: shorter chains, errors
// that grow with 64 + k / 64 additions instead of k.
template <Product kP, typename O>
__global__ void __launch_bounds__(G_THREADS, G_PER_SM) exp_general_kernel(const __grid_constant__ GeneralArgs<O> p) {
  constexpr bool kWeights = kP == Product::kWeights;
  __shared__ __align__(16) float as[2][GK * (GF + 4)], bs[2][GK * (GC + 4)];
  __shared__ int32_t first[GRS_MOE_MAX_EXPERTS + 1];
  pdl_wait();
  pdl_trigger();
  if constexpr (!kWeights) {
    group_prefix<GC, G_THREADS>(p.offsets, p.experts, p.rows, first);
    __syncthreads();
  }
  const int64_t ft = (p.f + GF - 1) / GF, ct = (p.c + GC - 1) / GC;
  const int64_t tiles = ft * (kWeights ? ct * p.experts : first[p.experts]);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;  // features 4 tx.. and 64 + 4 tx.., c 4 ty.. and 32 + 4 ty..
  for (int64_t i = blockIdx.x; i < tiles * p.slices; i += gridDim.x) {
    const int64_t slice = i / tiles, tile = i - slice * tiles, ci = tile / ft, f0 = (tile - ci * ft) * GF;
    const int e = kWeights ? static_cast<int>(ci / ct) : expert_of(first, p.experts, ci);
    const ExpertRows r(p.offsets, e, p.rows);
    const int64_t c0 = kWeights ? (ci - e * ct) * GC : r.from + (ci - first[e]) * GC, c1 = kWeights ? p.c : r.to;
    int64_t k0 = kWeights ? r.from : 0, k1 = kWeights ? r.to : p.k;
    if (p.slices > 1) {
      const int64_t n = slice_length<64>(k1 - k0, p.slices);
      k0 = k0 + slice * n < k1 ? k0 + slice * n : k1;
      k1 = k1 - k0 < n ? k1 : k0 + n;
    }
    const float *a = p.a + e * p.a_e, *b = p.b;
    uint64_t total[8][4] = {}, part[8][4] = {};
    Panel<GF, kP == Product::kForward> pa(a, f0, p.f, k0, p.a_f, p.a_k);
    Panel<GC, !kWeights> pb(b, c0, c1, k0, p.b_c, p.b_k);
    pa.load(k1 - k0);
    pb.load(k1 - k0);
    __syncthreads();  // the tile before has been read
    pa.put(as[0]);
    pb.put(bs[0]);
    if (k1 - k0 > GK) {
      pa.load(k1 - k0 - GK);
      pb.load(k1 - k0 - GK);
    }
    int step = 0;
    for (int64_t k = k0; k < k1; k += GK, ++step) {
      __syncthreads();  // all have put this step's numbers, and are done with those of the step before
      if (k + GK < k1) {
        pa.put(as[(step + 1) & 1]);
        pb.put(bs[(step + 1) & 1]);
        if (k + 2 * GK < k1) {
          pa.load(k1 - k - 2 * GK);
          pb.load(k1 - k - 2 * GK);
        }
      }
      const float *sa = as[step & 1], *sb = bs[step & 1];
#pragma unroll
      for (int q = 0; q < GK; ++q) {
        const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(sa + q * (GF + 4) + 4 * tx), v = *reinterpret_cast<const ulonglong2*>(sa + q * (GF + 4) + 64 + 4 * tx);
        const float4 c = *reinterpret_cast<const float4*>(sb + q * (GC + 4) + 4 * ty), d = *reinterpret_cast<const float4*>(sb + q * (GC + 4) + 32 + 4 * ty);
        const uint64_t x[4] = {u.x, u.y, v.x, v.y};
        const float y[8] = {c.x, c.y, c.z, c.w, d.x, d.y, d.z, d.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) part[i][j] = fma2(x[j], pair_bits(both(y[i])), part[i][j]);
      }
      if (step % 4 == 3)
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            total[i][j] = add2(total[i][j], part[i][j]);
            part[i][j] = 0;
          }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t c = c0 + (i < 4 ? 4 * ty + i : 28 + 4 * ty + i);
      if (c >= c1 || !GRS_CHECK(kWeights || c < p.rows, exp_flags, SITE_EXP_ROW)) continue;
      O* o = p.o + e * p.o_e + slice * p.o_s + c * p.o_c;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = pair_floats(add2(total[i][j], part[i][j]));
        const int64_t f = f0 + (j < 2 ? 4 * tx + 2 * j : 64 + 4 * tx + 2 * (j - 2));
        if (f < p.f) o[f] = from_float<O>(v.x);
        if (f + 1 < p.f) o[f + 1] = from_float<O>(v.y);
      }
    }
  }
}

// ------------------------------------------------------------ bf16, few rows
// Forward of a token or two is a matter of reading the weights, and the tensor
// cores' tiles of 128 features are too few for the SMs.  A warp has two
// features and a group of up to four rows, its lanes the same 8 of k of all,
// products in fp32.
constexpr int FEW = 4;        // rows of a group
constexpr int FEW_AHEAD = 4;  // loads of each feature on their way
constexpr int FEW_ROWS = 8;   // 2048 -> 768, 32 experts: 4 rows 6.2 us and 11.7 on the tensor cores, 8 rows 7.8 and 11.5, 20 rows 14.4 and 11.8

struct FewArgs {
  const uint16_t *x, *w;
  uint16_t* y;
  const int32_t* offsets;
  int64_t ld_x, ld_y;
  int32_t rows, experts, in, out;
};

__global__ void __launch_bounds__(EXP_THREADS) exp_few_kernel(const __grid_constant__ FewArgs a) {
  __shared__ int32_t first[GRS_MOE_MAX_EXPERTS + 1];
  pdl_wait();
  pdl_trigger();
  group_prefix<FEW, EXP_THREADS>(a.offsets, a.experts, a.rows, first);
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const int64_t pairs = (int64_t(a.out) + 1) / 2, items = pairs * first[a.experts], warps = int64_t(gridDim.x) * (EXP_THREADS / 32);
  for (int64_t it = int64_t(threadIdx.x >> 5) * gridDim.x + blockIdx.x; it < items; it += warps) {
    const int64_t g = it / pairs;
    const int32_t f = static_cast<int32_t>(it - g * pairs) * 2;
    const int e = expert_of(first, a.experts, g);
    const ExpertRows r(a.offsets, e, a.rows);
    const int32_t row = r.from + static_cast<int32_t>(g - first[e]) * FEW, n = r.to - row < FEW ? r.to - row : FEW;
    const uint16_t *w0 = a.w + (int64_t(e) * a.out + f) * a.in, *w1 = f + 1 < a.out ? w0 + a.in : w0, *x = a.x + row * a.ld_x;
    float2 sum[FEW][2];
#pragma unroll
    for (int i = 0; i < FEW; ++i) sum[i][0] = sum[i][1] = both(0.0f);
    for (int32_t k0 = lane * 8; k0 < a.in; k0 += 256 * FEW_AHEAD) {
      uint4 u[FEW_AHEAD], v[FEW_AHEAD];
#pragma unroll
      for (int j = 0; j < FEW_AHEAD; ++j) {
        const int32_t k = k0 + 256 * j;
        u[j] = v[j] = make_uint4(0, 0, 0, 0);
        if (k < a.in) {
          u[j] = __ldcs(reinterpret_cast<const uint4*>(w0 + k));
          v[j] = __ldcs(reinterpret_cast<const uint4*>(w1 + k));
        }
      }
#pragma unroll
      for (int j = 0; j < FEW_AHEAD; ++j) {
        const int32_t k = k0 + 256 * j;
        if (k >= a.in) break;
        const float2 p[4] = {bf16_pair(u[j].x), bf16_pair(u[j].y), bf16_pair(u[j].z), bf16_pair(u[j].w)};
        const float2 q[4] = {bf16_pair(v[j].x), bf16_pair(v[j].y), bf16_pair(v[j].z), bf16_pair(v[j].w)};
#pragma unroll
        for (int i = 0; i < FEW; ++i) {
          if (i >= n) break;
          const uint4 d = __ldg(reinterpret_cast<const uint4*>(x + i * a.ld_x + k));
          const float2 y[4] = {bf16_pair(d.x), bf16_pair(d.y), bf16_pair(d.z), bf16_pair(d.w)};
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            sum[i][0] = fma2(p[h], y[h], sum[i][0]);
            sum[i][1] = fma2(q[h], y[h], sum[i][1]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < FEW; ++i) {
      if (i >= n) break;
      const float s = warp_sum(sum[i][0].x + sum[i][0].y), t = warp_sum(sum[i][1].x + sum[i][1].y);
      uint16_t* y = a.y + (row + i) * a.ld_y + f;
      if (lane == 0 && GRS_CHECK(row + i < a.rows, exp_flags, SITE_EXP_ROW)) {
        y[0] = from_float<uint16_t>(s);
        if (f + 1 < a.out) y[1] = from_float<uint16_t>(t);
      }
    }
  }
}

// ------------------------------------------------------------------- host
grs_status check_experts(const grs_experts* s, const char* who, ExpLd* ld) {
  if (s == nullptr) return api_fail(GRS_ERR_INVALID_ARG, who, "shape is NULL");
  if (s->rows < 0 || s->rows > GRS_MAX_ROWS) return api_fail(GRS_ERR_SHAPE, who, "rows must be in [0, GRS_MAX_ROWS]");
  if (s->experts < 1 || s->experts > GRS_MOE_MAX_EXPERTS) return api_fail(GRS_ERR_SHAPE, who, "experts must be in [1, GRS_MOE_MAX_EXPERTS]");
  if (s->in_features < 1 || s->out_features < 1 || s->in_features > GRS_MAX_WIDTH || s->out_features > GRS_MAX_WIDTH)
    return api_fail(GRS_ERR_SHAPE, who, "in_features and out_features must be in [1, GRS_MAX_WIDTH]");
  if (!dtype_ok(s->dtype) || !dtype_ok(s->grad_dtype)) return api_fail(GRS_ERR_INVALID_ARG, who, "unknown element type");
  ld->x = s->ld_x == 0 ? s->in_features : s->ld_x;
  ld->y = s->ld_y == 0 ? s->out_features : s->ld_y;
  if (ld->x < s->in_features || ld->y < s->out_features || ld->x > GRS_MAX_WIDTH || ld->y > GRS_MAX_WIDTH)
    return api_fail(GRS_ERR_SHAPE, who, "a distance of rows below their width or above GRS_MAX_WIDTH");
  ld->w = s->in_features;
  // (so that bytes of anything here fit 64 bits)
  const int64_t wide = ld->x > ld->y ? ld->x : ld->y;
  if (int64_t(s->in_features) * s->out_features > GRS_MAX_ELEMENTS / s->experts || s->rows > GRS_MAX_ELEMENTS / wide)
    return api_fail(GRS_ERR_SHAPE, who, "more than GRS_MAX_ELEMENTS elements of a matrix or of all weights");
  return GRS_OK;
}

// Tiles of a product, n of them where experts have equal numbers of rows, `most` at most.
struct GeneralTiles {
  int64_t n, most, k;
};
GeneralTiles exp_general_tiles(Product p, const grs_experts* s) {
  const int64_t in = s->in_features, out = s->out_features, some = s->rows < s->experts ? s->rows : s->experts;
  auto up = [](int64_t n, int64_t to) { return (n + to - 1) / to; };
  if (p == Product::kWeights) {
    const int64_t n = s->experts * up(in, GF) * up(out, GC);
    return {n, n, s->rows / s->experts};
  }
  const int64_t ft = up(p == Product::kForward ? out : in, GF);
  return {some * up(s->rows / some, GC) * ft, (s->rows / GC + some) * ft, p == Product::kForward ? in : out};
}

// Slices of such a product, of 64 at least: those that end first, by the measured
// 1.8 us of a step with two blocks an SM and 4 us and 5 TB/s of the joining
// kernel.  749 rows, 9 experts, 1251 -> 1208: forward 134 us whole, 93 so; 138
// rows, 2 experts, 507 -> 120 35 and 15; 2048 rows, one expert, 64 x 64, weights'
// gradient 39 (in slices of 512) and 16.
int exp_general_slices(const GeneralTiles& t, int64_t outputs) {
  const int64_t slots = G_PER_SM * 152;
  double best = 1e30;
  int n = 1;
  for (int i = 1; i <= 64 && (i == 1 || i * 64 <= t.k); i += i < 8 ? 1 : i / 4) {
    const double us = double((t.n * i + slots - 1) / slots) * ((t.k + i - 1) / i) * (1.8 / GK) + (i > 1 ? 4.0 + 8e-6 / 5 * outputs * i : 0.0);
    if (us < 0.95 * best) {
      best = us;
      n = i;
    }
  }
  return n;
}

template <Product kP, typename O>
cudaError_t exp_general(const grs_experts* s, const ExpLd& ld, const void* a, const void* b, const int32_t* offsets, void* o,
                        const ExpSlices& sl, void* stream) {
  const int64_t in = s->in_features, out = s->out_features;
  GeneralArgs<O> p{};
  p.a = static_cast<const float*>(a);
  p.b = static_cast<const float*>(b);
  p.o = static_cast<O*>(sl.n > 1 ? static_cast<void*>(sl.parts) : o);
  p.offsets = offsets;
  p.rows = static_cast<int32_t>(s->rows);
  p.experts = s->experts;
  p.slices = sl.n;
  p.o_s = sl.distance;
  if (kP == Product::kForward) {  // A = w, B = xs
    p.a_f = in, p.a_k = 1, p.a_e = in * out, p.b_c = ld.x, p.b_k = 1, p.o_c = ld.y, p.f = out, p.k = in;
  } else if (kP == Product::kRows) {  // A = w, B = dys
    p.a_f = 1, p.a_k = in, p.a_e = in * out, p.b_c = ld.y, p.b_k = 1, p.o_c = ld.x, p.f = in, p.k = out;
  } else {  // A = xs, B = dys
    p.a_f = 1, p.a_k = ld.x, p.b_c = 1, p.b_k = ld.y, p.o_c = in, p.o_e = in * out, p.f = in, p.c = out;
  }
  if (sl.n > 1) p.o_c = sl.ld;
  const int64_t tiles = exp_general_tiles(kP, s).most * sl.n;
  return launch_pdl(exp_general_kernel<kP, O>, dim3(static_cast<unsigned>(tiles < 152 * G_PER_SM ? tiles : 152 * G_PER_SM)), dim3(G_THREADS), 0, stream, p);
}

// ------------------------------------------------------------------ slices
// The sum of the slices' results, in their order.  With offsets only the
// experts' rows; an expert without rows has no product, its slices are zeros.
template <typename O>
__global__ void __launch_bounds__(EXP_THREADS) exp_join_kernel(const float* __restrict__ parts, int32_t slices, int64_t distance, int64_t rows,
                                                               int32_t width, O* o, int64_t ld, const int32_t* offsets, int32_t experts) {
  pdl_wait();
  pdl_trigger();
  int64_t from = 0, to = rows;
  if (offsets != nullptr) {
    from = ExpertRows(offsets, 0, static_cast<int32_t>(rows)).from;
    to = ExpertRows(offsets, experts - 1, static_cast<int32_t>(rows)).to;
  }
  for (int64_t i = from * width + int64_t(blockIdx.x) * EXP_THREADS + threadIdx.x; i < to * width; i += int64_t(gridDim.x) * EXP_THREADS) {
    float s = 0.0f;
#pragma unroll 4
    for (int32_t k = 0; k < slices; ++k) s = __fadd_rn(s, __ldcs(parts + k * distance + i));
    const int64_t r = i / width;
    if (GRS_CHECK(r < rows, exp_flags, SITE_EXP_ROW)) o[r * ld + (i - r * width)] = from_float<O>(s);
  }
}

// How a product on the tensor cores is cut: as far as its tiles leave SMs
// without any, in slices of 1024 at least.  20 rows, 32 experts, 2048 -> 768:
// 12.7 us whole, 11.7 in two slices; 16 rows, 8 experts, 8192 -> 1024 32 and 16.5.
// Twice as many slices: 512 rows 17.2 -> 21.1.
ExpSlices exp_slices(Product p, const grs_experts* s) {
  ExpSlices sl;
  sl.ld = p == Product::kForward ? s->out_features : s->in_features;
  sl.distance = (p == Product::kWeights ? int64_t(s->experts) * s->out_features : s->rows) * sl.ld;
  if (s->rows == 0) return sl;
  if (s->dtype == GRS_DTYPE_FP32) {
    sl.n = exp_general_slices(exp_general_tiles(p, s), sl.distance);
    return sl;
  }
  const ExpTiles t = experts_mma_tiles(p, s);
  const int64_t slots = t.columns == 256 ? 0 : t.columns <= 64 && p != Product::kWeights ? 2 * 152 : 152;
  int64_t n = t.n > 0 ? slots / t.n : 0, most = t.k / 1024;
  if (n > most) n = most;
  if (n >= 2) sl.n = static_cast<int>(n);
  return sl;
}

int64_t slices_bytes(const ExpSlices& sl) { return sl.n > 1 ? sl.n * sl.distance * 4 : 0; }

template <typename O>
cudaError_t exp_join(Product p, const grs_experts* s, const ExpSlices& sl, const int32_t* offsets, void* o, int64_t ld, void* stream) {
  const int64_t blocks = (sl.distance + EXP_THREADS - 1) / EXP_THREADS;
  return launch_pdl(exp_join_kernel<O>, dim3(static_cast<unsigned>(blocks < 8 * 152 ? blocks : 8 * 152)), dim3(EXP_THREADS), 0, stream,
                    static_cast<const float*>(sl.parts), sl.n, sl.distance, sl.distance / sl.ld, static_cast<int32_t>(sl.ld), static_cast<O*>(o), ld,
                    p == Product::kWeights ? nullptr : offsets, s->experts);
}

// One product to `o`, rows o_ld apart; parts: room for its slices.
template <Product kP>
cudaError_t exp_product(const grs_experts* s, const ExpLd& ld, const void* xs, const void* w, const void* dys, const int32_t* offsets, void* o,
                        int64_t o_ld, void* parts, const ExpQuit& quit, void* stream) {
  ExpSlices sl = exp_slices(kP, s);
  sl.parts = static_cast<float*>(parts);
  const bool fp32 = (kP == Product::kWeights ? s->grad_dtype : s->dtype) == GRS_DTYPE_FP32;
  cudaError_t e;
  if (s->dtype == GRS_DTYPE_BF16) {
    e = experts_mma(kP, s, ld, xs, w, dys, offsets, o, o_ld, sl, quit, stream);
  } else {
    const void *a = kP == Product::kWeights ? xs : w, *b = kP == Product::kForward ? xs : dys;
    if constexpr (kP == Product::kWeights) {  // only gradients may be of another type
      e = fp32 || sl.n > 1 ? exp_general<kP, float>(s, ld, a, b, offsets, o, sl, stream)
                           : exp_general<kP, uint16_t>(s, ld, a, b, offsets, o, sl, stream);
    } else {
      e = exp_general<kP, float>(s, ld, a, b, offsets, o, sl, stream);
    }
  }
  if (e != cudaSuccess || sl.n == 1) return e;
  return fp32 ? exp_join<float>(kP, s, sl, offsets, o, o_ld, stream) : exp_join<uint16_t>(kP, s, sl, offsets, o, o_ld, stream);
}

// Whether forward is left to exp_few_kernel.
bool exp_few(const grs_experts* s, const ExpLd& ld) { return s->rows <= FEW_ROWS && s->in_features % 8 == 0 && ld.x % 8 == 0; }

cudaError_t exp_few_forward(const grs_experts* s, const ExpLd& ld, const void* xs, const void* w, const int32_t* offsets, void* ys, void* stream) {
  const FewArgs a{static_cast<const uint16_t*>(xs), static_cast<const uint16_t*>(w), static_cast<uint16_t*>(ys), offsets, ld.x, ld.y,
                  static_cast<int32_t>(s->rows), s->experts, s->in_features, s->out_features};
  return launch_pdl(exp_few_kernel, dim3(152 * 2), dim3(EXP_THREADS), 0, stream, a);
}

// --------------------------------------------------- bf16, rows laid out anew
// Up to three matrices to rows that are whole 16-byte chunks apart, a thread
// eight elements: from the two aligned chunks that they lie in, or one by one
// where these reach behind the matrix.  What comes after a row's last element
// in the copy is never read.
struct PadArgs {
  const uint16_t* from[3];
  uint16_t* to[3];
  int64_t ld[3], end[3], chunks[4];  // end: elements up to the matrix's last; chunks[i]: of the matrices before
  int32_t per[3];                    // chunks of a row
};

constexpr int PAD_EACH = 4;  // chunks of a thread, their loads on their way together

__global__ void __launch_bounds__(EXP_THREADS) exp_pad_kernel(const __grid_constant__ PadArgs a) {
  pdl_wait();
  pdl_trigger();
  const int64_t i0 = int64_t(blockIdx.x) * (EXP_THREADS * PAD_EACH) + threadIdx.x;
  uint4 x[PAD_EACH], y[PAD_EACH];
  int shift[PAD_EACH];  // elements
#pragma unroll
  for (int u = 0; u < PAD_EACH; ++u) {
    const int64_t i = i0 + u * EXP_THREADS;
    shift[u] = -1;
    if (i >= a.chunks[3]) continue;
    const int m = i >= a.chunks[2] ? 2 : i >= a.chunks[1] ? 1 : 0;
    const int64_t c = i - a.chunks[m], r = c <= UINT32_MAX ? static_cast<uint32_t>(c) / static_cast<uint32_t>(a.per[m]) : c / a.per[m];
    const int64_t at = r * a.ld[m] + (c - r * a.per[m]) * 8, low = at & ~int64_t(7);
    const uint16_t* p = a.from[m];
    if (low + 16 <= a.end[m]) {
      shift[u] = static_cast<int>(at - low);
      x[u] = __ldg(reinterpret_cast<const uint4*>(p + low));
      y[u] = __ldg(reinterpret_cast<const uint4*>(p + low) + 1);
    } else if (GRS_CHECK(at < a.end[m], exp_flags, SITE_EXP_ROW)) {
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        w[q] = (at + 2 * q < a.end[m] ? uint32_t(__ldg(p + at + 2 * q)) : 0u) |
               (at + 2 * q + 1 < a.end[m] ? uint32_t(__ldg(p + at + 2 * q + 1)) << 16 : 0u);
      *reinterpret_cast<uint4*>(a.to[m] + c * 8) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
#pragma unroll
  for (int u = 0; u < PAD_EACH; ++u) {
    if (shift[u] < 0) continue;
    const int64_t i = i0 + u * EXP_THREADS;
    const int m = i >= a.chunks[2] ? 2 : i >= a.chunks[1] ? 1 : 0;
    uint32_t w[8] = {x[u].x, x[u].y, x[u].z, x[u].w, y[u].x, y[u].y, y[u].z, y[u].w};
#pragma unroll
    for (int q = 0; q < 6; ++q) w[q] = (shift[u] & 4) != 0 ? w[q + 2] : w[q];
#pragma unroll
    for (int q = 0; q < 5; ++q) w[q] = (shift[u] & 2) != 0 ? w[q + 1] : w[q];
#pragma unroll
    for (int q = 0; q < 4; ++q) w[q] = (shift[u] & 1) != 0 ? __funnelshift_r(w[q], w[q + 1], 16) : w[q];
    *reinterpret_cast<uint4*>(a.to[m] + (i - a.chunks[m]) * 8) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

int64_t round8(int64_t n) { return (n + 7) & ~int64_t(7); }

// Bytes of an operand's copy: none where its rows are whole 16-byte chunks apart.
int64_t pad_bytes(int64_t rows, int64_t ld, int64_t width) { return ld % 8 == 0 ? 0 : rows * round8(width) * 2; }

// Copies to be made, at *ws one after another.
struct Pads {
  PadArgs a{};
  int n = 0;
  uint8_t* ws;
  explicit Pads(void* ws_) : ws(static_cast<uint8_t*>(ws_)) {}
  // `p` itself, or where its copy will be; *ld becomes the copy's.
  const void* add(const void* p, int64_t rows, int64_t* ld, int64_t width) {
    const int64_t bytes = pad_bytes(rows, *ld, width);
    if (bytes == 0) return p;
    a.from[n] = static_cast<const uint16_t*>(p);
    a.to[n] = reinterpret_cast<uint16_t*>(ws);
    a.ld[n] = *ld;
    a.end[n] = (rows - 1) * *ld + width;
    a.per[n] = static_cast<int32_t>(round8(width) / 8);
    const int64_t all = a.chunks[n] + rows * a.per[n];
    for (int i = ++n; i < 4; ++i) a.chunks[i] = all;
    *ld = round8(width);
    void* here = ws;
    ws += bytes;  // (whole 16-byte chunks)
    return here;
  }
  cudaError_t run(void* stream) const {
    if (n == 0) return cudaSuccess;
    const int64_t per = EXP_THREADS * PAD_EACH, blocks = (a.chunks[3] + per - 1) / per;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_pdl(exp_pad_kernel, dim3(static_cast<unsigned>(blocks)), dim3(EXP_THREADS), 0, stream, a);
  }
};

// The copies of operands, then the slices of one product after another.
int64_t exp_workspace(const grs_experts* s, const ExpLd& ld, int64_t* pads) {
  *pads = s->dtype == GRS_DTYPE_FP32 ? 0
                                     : pad_bytes(s->rows, ld.x, s->in_features) + pad_bytes(s->rows, ld.y, s->out_features) +
                                           pad_bytes(int64_t(s->experts) * s->out_features, ld.w, s->in_features);
  int64_t most = 0;
  for (Product p : {Product::kForward, Product::kRows, Product::kWeights}) {
    const int64_t b = slices_bytes(exp_slices(p, s));
    if (b > most) most = b;
  }
  return *pads + ((most + 15) & ~int64_t(15));
}

grs_status experts_backward(const grs_experts* s, const void* dys, const void* xs, const void* w, const int32_t* offsets, void* dxs, void* dw,
                            void* workspace, const ExpQuit& quit, void* stream, const char* who) {
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
  int64_t pad = 0;
  if (exp_workspace(s, ld, &pad) > 0 && workspace == nullptr) return api_fail(GRS_ERR_INVALID_ARG, who, "this shape needs a workspace");
  cudaError_t e = cudaSuccess;
  if (dxs != nullptr || dw != nullptr) {
    const int64_t ld_x = ld.x;
    uint8_t* parts = static_cast<uint8_t*>(workspace) + pad;
    if (s->dtype == GRS_DTYPE_BF16) {
      Pads pads(workspace);
      dys = pads.add(dys, s->rows, &ld.y, s->out_features);
      if (dxs != nullptr) w = pads.add(w, int64_t(s->experts) * s->out_features, &ld.w, s->in_features);
      if (dw != nullptr) xs = pads.add(xs, s->rows, &ld.x, s->in_features);
      e = pads.run(stream);
    }
    if (e == cudaSuccess && dxs != nullptr) e = exp_product<Product::kRows>(s, ld, nullptr, w, dys, offsets, dxs, ld_x, parts, quit, stream);
    if (e == cudaSuccess && dw != nullptr) e = exp_product<Product::kWeights>(s, ld, xs, nullptr, dys, offsets, dw, s->in_features, parts, quit, stream);
  }
  return e == cudaSuccess ? GRS_OK : api_cuda_fail(e, who);
}

// ------------------------------------------------------------------ flags
// Kernels of other streams may raise a flag at any time, so each is read and
// cleared in one step: what is raised afterwards stays for the next look.
constexpr int FLAG_FILES = 4;
struct FlagFiles {
  int* at[FLAG_FILES];
};

__device__ int flags_taken[FLAG_COUNT];

__global__ void take_flags_kernel(const __grid_constant__ FlagFiles files) {
  pdl_wait();
  if (threadIdx.x >= FLAG_COUNT) return;
  int x = 0;
  for (int f = 0; f < FLAG_FILES; ++f) {
    const int y = atomicExch(files.at[f] + threadIdx.x, 0);
    if (x == 0) x = y;
  }
  flags_taken[threadIdx.x] = x;
}

cudaError_t take_flags(const FlagFiles& files, int (&flags)[FLAG_COUNT], cudaStream_t st) try {
  static std::mutex one;  // flags_taken holds one look's
  const std::lock_guard<std::mutex> lock(one);
  void* at = nullptr;
  cudaError_t e = cudaGetSymbolAddress(&at, flags_taken);
  if (e != cudaSuccess) return e;
  e = launch_pdl(take_flags_kernel, dim3(1), dim3(32), 0, st, files);
  if (e == cudaSuccess) e = cudaMemcpyAsync(flags, at, sizeof(flags), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  return e;
} catch (...) {  // the lock's
  return cudaErrorUnknown;
}

}  // namespace

cudaError_t experts_flags(int** at) { return cudaGetSymbolAddress(reinterpret_cast<void**>(at), exp_flags); }

}  // namespace grs

using namespace grs;

extern "C" {

grs_status grs_operators_check_device_errors(void* stream) {
  static const char who[] = "grs_operators_check_device_errors";
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  int flags[FLAG_COUNT] = {};
  FlagFiles files{};
  cudaError_t e = cudaStreamSynchronize(st);
  if (e == cudaSuccess) e = experts_flags(&files.at[0]);
  if (e == cudaSuccess) e = experts_mma_flags(&files.at[1]);
  if (e == cudaSuccess) e = embedding_flags(&files.at[2]);
  if (e == cudaSuccess) e = qk_norm_flags(&files.at[3]);
  if (e == cudaSuccess) e = take_flags(files, flags, st);
  if (e != cudaSuccess) return api_cuda_fail(e, who);
  if (flags[FLAG_BOUNDS] != 0) return api_fail(GRS_ERR_BOUNDS, who, "an index out of place");
  return flags[FLAG_TIMEOUT] != 0 ? api_fail(GRS_ERR_TIMEOUT, who, "a bounded device wait timed out") : GRS_OK;
}

int64_t grs_experts_workspace_bytes(const grs_experts* s) {
  ExpLd ld;
  if (check_experts(s, "grs_experts_workspace_bytes", &ld) != GRS_OK) return -1;
  int64_t pads;
  return exp_workspace(s, ld, &pads);
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
  int64_t pad = 0;
  if (workspace == nullptr && exp_workspace(s, ld, &pad) > 0) return api_fail(GRS_ERR_INVALID_ARG, who, "this shape needs a workspace");
  cudaError_t e = cudaSuccess;
  if (s->dtype == GRS_DTYPE_BF16 && exp_few(s, ld)) {
    e = exp_few_forward(s, ld, xs, w, offsets, ys, stream);
  } else {
    exp_workspace(s, ld, &pad);
    const int64_t ld_y = ld.y;
    if (s->dtype == GRS_DTYPE_BF16) {
      Pads pads(workspace);
      xs = pads.add(xs, s->rows, &ld.x, s->in_features);
      w = pads.add(w, int64_t(s->experts) * s->out_features, &ld.w, s->in_features);
      e = pads.run(stream);
    }
    if (e == cudaSuccess) e = exp_product<Product::kForward>(s, ld, xs, w, nullptr, offsets, ys, ld_y, static_cast<uint8_t*>(workspace) + pad, ExpQuit{}, stream);
  }
  return e == cudaSuccess ? GRS_OK : api_cuda_fail(e, who);
}

grs_status grs_experts_backward(const grs_experts* s, const void* dys, const void* xs, const void* w, const int32_t* offsets, void* dxs,
                                void* dw, void* workspace, void* stream) {
  return experts_backward(s, dys, xs, w, offsets, dxs, dw, workspace, ExpQuit{}, stream, "grs_experts_backward");
}

grs_status grs_selftest_experts_wait(const grs_experts* s, const void* dys, const void* xs, const void* w, const int32_t* offsets, void* dxs,
                                     void* dw, void* workspace, int32_t quitter, int32_t quit_tile, void* stream) {
  static const char who[] = "grs_selftest_experts_wait";
  if (quitter < 0 || quit_tile < 0) return api_fail(GRS_ERR_INVALID_ARG, who, "quitter and quit_tile must be >= 0");
  if (s != nullptr && s->dtype != GRS_DTYPE_BF16) return api_fail(GRS_ERR_INVALID_ARG, who, "only products in bf16 have such waits");
  return experts_backward(s, dys, xs, w, offsets, dxs, dw, workspace, ExpQuit{quitter, quit_tile}, stream, who);
}

}  // extern "C"
