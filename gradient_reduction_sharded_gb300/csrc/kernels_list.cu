// AdamW over a list of separate tensors (grs_tensors_*): the deterministic
// gradient norm, the fused clip + AdamW + bf16 cast with states in 32 or in
// 8 bits, and the conversion between the two.
//
// The step and the conversions walk tiles of LIST_T elements, each inside one
// tensor; a device table gives a tile's tensor, its first element there and
// its place in the state arrays.  A thread handles 8 consecutive elements, a
// warp therefore one block of the 8-bit states (256 elements): the block's
// largest magnitude is one warp reduction and no state crosses a warp.  One
// tile a block of 256 threads: blocks that stay and loop over tiles cost
// registers, spills and 20 % (1.10B elements, 8 bits, bf16 gradients).
//
// What bounds them, on a GB300 that copies 6.78 TB/s:
//   step, 32 bits  memory: 28 or 30 bytes an element; 61.8M at 6.9 TB/s
//                  (248 us with bf16, 265 with fp32 gradients)
//   step, 8 bits   memory and instruction issue alike: 16 or 18 bytes and 80
//                  instructions an element; 61.8M fp32 in 172 us (6.5 TB/s),
//                  1.10B bf16 in 2.92 ms (6.0 TB/s).  Hence the hardware's
//                  8-bit decoding, the codes rounded by one product and one
//                  addition, and the folded hash.
//   norm           memory for long lists (61.8M fp32: 5.8 TB/s; bf16, whose
//                  sums take as many instructions for half the bytes, 4.0),
//                  latency for short ones (12 tensors: 6 us)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "api_util.h"
#include "device.cuh"
#include "internal.h"
#include "launch.cuh"
#include "packed.cuh"
#include "shifted.cuh"

namespace grs {
namespace {

constexpr int LIST_THREADS = 256;
constexpr int64_t LIST_T = 2048;
static_assert(LIST_T == LIST_THREADS * 8, "one 8-element group per thread per tile");
static_assert(GRS_STATE_BLOCK == 32 * 8, "one warp per block of the 8-bit states");

struct alignas(16) ListTile {
  int64_t state0;  // first element in the state arrays
  int64_t e0;      // first element in the tensor
  int32_t tensor;
  int32_t n;       // elements of the tensor in the tile
  int64_t rest;    // elements of the tensor from e0 on
};
static_assert(sizeof(ListTile) == 32, "two 16-byte loads");

}  // namespace
}  // namespace grs

struct grs_tensors {
  std::vector<int64_t> numel, offset;
  int64_t n_elements = 0, n_state = 0, n_tiles = 0;
  int device = -1;
  grs::ListTile* d_tiles = nullptr;
  int* d_flags = nullptr;
};

namespace grs {
namespace {

__device__ __forceinline__ ListTile load_tile(const ListTile* p) {
  const int4 a = __ldg(reinterpret_cast<const int4*>(p));
  const int4 b = __ldg(reinterpret_cast<const int4*>(p) + 1);
  ListTile t;
  t.state0 = (int64_t(a.y) << 32) | uint32_t(a.x);
  t.e0 = (int64_t(a.w) << 32) | uint32_t(a.z);
  t.tensor = b.x;
  t.n = b.y;
  t.rest = (int64_t(b.w) << 32) | uint32_t(b.z);
  return t;
}

__device__ __forceinline__ void load_state8(const float* p, float2 (&o)[4]) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
  const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  o[0] = make_float2(a.x, a.y);
  o[1] = make_float2(a.z, a.w);
  o[2] = make_float2(b.x, b.y);
  o[3] = make_float2(b.z, b.w);
}

// Zeros in the place of elements n, n + 1, ...: state padding may hold anything.
__device__ __forceinline__ void clear_beyond(int n, float2 (&o)[4]) {
  if (n >= 8) return;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (2 * q >= n) o[q].x = 0.0f;
    if (2 * q + 1 >= n) o[q].y = 0.0f;
  }
}

__device__ __forceinline__ void store_state8(float* p, const float2 (&o)[4]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(o[0].x, o[0].y, o[1].x, o[1].y));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(o[2].x, o[2].y, o[3].x, o[3].y));
}

// ------------------------------------------------------------------- norm
// Sums held as unevaluated pairs hi + lo of floats (Knuth's TwoSum keeps each
// addition's rounding error), about 48 bits, two elements at a time: S is
// then as exact as a sum in fp64, whose additions would take several times
// the time of the loads.
struct Sums {
  float2 hi, lo;
};

__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return fma2(b, both(-1.0f), a); }

__device__ __forceinline__ void two_sum(Sums& a, float2 x) {
  const float2 t = add2(a.hi, x), z = sub2(t, a.hi);
  a.lo = add2(a.lo, add2(sub2(a.hi, sub2(t, z)), sub2(x, z)));
  a.hi = t;
}

// x * x: exact for bf16 numbers; for fp32 ones its rounding error goes to lo.
__device__ __forceinline__ void add_square(Sums& a, float2 x, float minus_zero, uint16_t) { two_sum(a, mul2_rounded(x, x, minus_zero)); }
__device__ __forceinline__ void add_square(Sums& a, float2 x, float minus_zero, float) {
  const float2 sq = mul2_rounded(x, x, minus_zero);
  two_sum(a, sq);
  a.lo = add2(a.lo, fma2(x, x, make_float2(-sq.x, -sq.y)));
}

// An infinite or NaN sum has no error term (inf - inf is NaN).
__device__ __forceinline__ double sum_value(float hi, float lo) {
  return isfinite(hi) ? static_cast<double>(hi) + static_cast<double>(lo) : static_cast<double>(hi);
}

// Every sum over the block's warps in a fixed order, in fp64.
__device__ __forceinline__ double block_sum(double x, double* red) {
  x = warp_sum(x);
  __syncthreads();  // red may still be read from the sum before
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  double s = red[0];
  for (int k = 1; k < LIST_THREADS / 32; ++k) s = __dadd_rn(s, red[k]);
  return s;
}

// A warp takes the tiles w, w + (all warps), ..., each as the 16-byte chunks
// that it starts in (a tensor that starts off a 16-byte boundary has its
// tiles' ends moved back to one; the order of a sum is free), half a tile's
// loads in flight at once and the next tile's record already there.  A lane
// keeps its sums in fp32 pairs over a tile and in fp64 over its tiles.  Each
// block leaves one fp64 sum, and the block that is last (the ticket) adds
// those up.  The grid is the same everywhere (or goes by the number of
// tiles), so every addition has its fixed place.
constexpr int LIST_NORM_BLOCKS = 608;  // four blocks an SM

__device__ __forceinline__ void add_chunk(Sums& s, uint4 v, float minus_zero, uint16_t tag) {
  add_square(s, bf16_pair(v.x), minus_zero, tag);
  add_square(s, bf16_pair(v.y), minus_zero, tag);
  add_square(s, bf16_pair(v.z), minus_zero, tag);
  add_square(s, bf16_pair(v.w), minus_zero, tag);
}
__device__ __forceinline__ void add_chunk(Sums& s, uint4 v, float minus_zero, float tag) {
  add_square(s, make_float2(__uint_as_float(v.x), __uint_as_float(v.y)), minus_zero, tag);
  add_square(s, make_float2(__uint_as_float(v.z), __uint_as_float(v.w)), minus_zero, tag);
}

template <typename G>
__global__ void __launch_bounds__(LIST_THREADS, 4) list_norm_kernel(const ListTile* __restrict__ tiles, int64_t n_tiles,
                                                                    const G* const* __restrict__ grads, int32_t n_tensors,
                                                                    double* __restrict__ partials,
                                                                    unsigned int* __restrict__ ticket, double inv_m2,
                                                                    float minus_zero, double* __restrict__ out,
                                                                    int* __restrict__ flags) {
  __shared__ double red[LIST_THREADS / 32];
  __shared__ bool last;
  constexpr int EL = 16 / sizeof(G), CHUNKS = static_cast<int>(LIST_T) / EL / 32, BATCH = 8;
  const int lane = threadIdx.x & 31;
  const int64_t warps = int64_t(gridDim.x) * (LIST_THREADS / 32);
  double total = 0.0;
  int64_t tile = int64_t(blockIdx.x) * (LIST_THREADS / 32) + (threadIdx.x >> 5);
  ListTile t{};
  if (tile < n_tiles) t = load_tile(tiles + tile);
  pdl_wait();  // the table above is the list's own and does not change
  pdl_trigger();
  const auto gradient = [&](int64_t at) -> const G* {
    if (at >= n_tiles || !GRS_CHECK(t.tensor >= 0 && t.tensor < n_tensors && t.n > 0 && t.n <= LIST_T, flags, SITE_LIST_NORM))
      return nullptr;
    return grads[t.tensor];
  };
  const G* g = gradient(tile);
  while (tile < n_tiles) {
    const ListTile now = t;
    const G* p = g;
    tile += warps;
    if (tile < n_tiles) t = load_tile(tiles + tile);
    g = gradient(tile);
    if (p == nullptr) continue;
    p += now.e0;
    const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15) / static_cast<int>(sizeof(G));
    // Elements of the tensor from the tile's first chunk on, as far as one
    // tile and chunk reach; its own first is `head`, 0 inside the tensor.
    const int head = now.e0 > 0 ? 0 : mis;
    const int64_t rest = now.rest + mis;
    const int end = rest < 2 * LIST_T ? static_cast<int>(rest) : static_cast<int>(2 * LIST_T);
    p -= mis;
    Sums s = {both(0.0f), both(0.0f)};
#pragma unroll
    for (int half = 0; half < CHUNKS; half += BATCH) {
      if (half * 32 * EL >= end) break;
      uint4 x[BATCH];
#pragma unroll
      for (int r = 0; r < BATCH; ++r) {
        const int c = ((half + r) * 32 + lane) * EL;
        x[r] = c < end ? load_chunk(p + c, head - c, end - c) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int r = 0; r < BATCH; ++r) add_chunk(s, x[r], minus_zero, G());
    }
    // A last tile may have a few elements left after its last whole chunk.
    if (lane == 0 && now.rest <= LIST_T && end > LIST_T) add_chunk(s, load_chunk(p + LIST_T, 0, end - static_cast<int>(LIST_T)), minus_zero, G());
    total = __dadd_rn(total, __dadd_rn(sum_value(s.hi.x, s.lo.x), sum_value(s.hi.y, s.lo.y)));
  }
  total = block_sum(total, red);
  if (threadIdx.x == 0) {
    partials[blockIdx.x] = total;
    __threadfence();
    last = atomicAdd(ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  total = 0.0;
  for (int i = threadIdx.x; i < static_cast<int>(gridDim.x); i += LIST_THREADS) total = __dadd_rn(total, __ldcg(partials + i));
  total = block_sum(total, red);
  if (threadIdx.x == 0) {
    total = __dmul_rn(total, inv_m2);
    *out = total;
    if (!isfinite(total)) atomicOr(flags + FLAG_NONFINITE, 1);
    *ticket = 0u;
  }
}

// Workspace of the norm: [LIST_NORM_BLOCKS doubles][ticket].
constexpr int64_t LIST_WS_TICKET = LIST_NORM_BLOCKS * 8;
constexpr int64_t LIST_WS_BYTES = LIST_WS_TICKET + 256;

// ---------------------------------------------------------- 8-bit format
// Counter-based random bits: an integer hash of the element's index under
// two keys made from the seed.  Each round folds the high half down and
// multiplies by an odd number (the golden ratio's and the square roots of 2
// and 3's fractional bits), so every index bit reaches every output bit.
constexpr uint32_t MIX_A = 0x9E3779B9u, MIX_B = 0x6A09E667u, MIX_C = 0xBB67AE85u;

inline uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= MIX_A;
  x ^= x >> 15;
  x *= MIX_C;
  return x ^ (x >> 16);
}

struct Keys {
  uint32_t k0, k1;
};

Keys make_keys(uint64_t seed) {
  Keys k;
  k.k0 = mix32(static_cast<uint32_t>(seed) + MIX_A);
  k.k1 = mix32(k.k0 ^ static_cast<uint32_t>(seed >> 32));
  return k;
}

// The number of element `index` is x ^ (x >> 16) for
//   x = lo ^ k0 ^ hi * MIX_B (index = hi : lo), x = (x ^ (x >> 16)) * MIX_A ^ k1, x = (x ^ (x >> 15)) * MIX_C;
// this is the part after the first fold and without the last.
__device__ __forceinline__ uint32_t random_rest(uint32_t folded, uint32_t k1) {
  const uint32_t x = folded * MIX_A ^ k1;
  return (x ^ (x >> 15)) * MIX_C;
}

// The scale of a block whose largest magnitude has the bits `top`:
// 2^(ceil(log2 x) - 8), at least 2^-126, NaN when x is not finite.  ceil, so
// that a largest magnitude that was rounded up to a power of two keeps its
// scale when it is packed again.
struct Scale {
  float scale;
  float to_code;  // 1 / scale * 2^-120, if that is a normal number
  float inv;      // 1 / scale
  bool bad;       // not finite
  bool plain;     // to_code holds
};
__device__ __forceinline__ Scale block_scale(uint32_t top) {
  Scale s;
  s.bad = top >= 0x7f800000u;
  int e = static_cast<int>((top + 0x7fffffu) >> 23) - 8;
  e = e < 1 ? 1 : e;
  s.plain = e <= 133;
  s.scale = s.bad ? __uint_as_float(0x7fc00000u) : __uint_as_float(static_cast<uint32_t>(e) << 23);
  s.inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
  s.to_code = __uint_as_float(static_cast<uint32_t>(134 - e) << 23);
  return s;
}

// Largest of three, NaN if one is NaN (fmaxf would drop it).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Largest magnitude of the warp's 256 values, as bits (ordered like the
// values, NaN above infinity).
__device__ __forceinline__ uint32_t warp_absmax(const float2 (&x)[4]) {
  float top = 0.0f;
#pragma unroll
  for (int q = 0; q < 4; ++q) top = max_nan(max_nan(top, fabsf(x[q].x)), fabsf(x[q].y));
  return __reduce_max_sync(0xffffffffu, __float_as_uint(top));
}

// Times 2^-120 an E4M3 number (bias 7) has its own exponent and subnormals
// as binary32 (bias 127), so the code of x / scale is the top of that
// binary32 pattern, and adding to the 20 bits below it before they are cut
// off rounds: a random number below 2^20 stochastically, the usual
// half-minus-one plus the last bit kept to nearest even.  The pattern is below
// 2^27 (no code is above 0x78), the sign stays in bit 31.
__device__ __forceinline__ void code_patterns(const float2 (&x)[4], const Scale& s, uint32_t (&t)[8]) {
  float2 y[4];
  // The scale is a power of two: one product gives the same number where its
  // factor is normal (magnitudes up to 2^14; the same for the whole warp).
  if (s.plain) {
#pragma unroll
    for (int q = 0; q < 4; ++q) y[q] = mul2(x[q], both(s.to_code));
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) y[q] = mul2(mul2(x[q], both(s.inv)), both(0x1p-120f));
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    t[2 * q] = __float_as_uint(y[q].x);
    t[2 * q + 1] = __float_as_uint(y[q].y);
  }
}

// Bytes of sign (if there is one) and code from the rounded patterns; zeros for a bad block.
template <bool kSigned>
__device__ __forceinline__ uint2 code_bytes(const uint32_t (&t)[8], bool bad) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t u[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) u[q] = t[4 * h + q] << 4 | (kSigned ? t[4 * h + q] & 0x80000000u : 0u);  // the code in the top byte
    w[h] = bad ? 0u : __byte_perm(__byte_perm(u[0], u[1], 0x0073), __byte_perm(u[2], u[3], 0x0073), 0x5410);
  }
  return make_uint2(w[0], w[1]);
}

// A positive sqrt(v) never becomes zero.  (sqrt of a positive fp32 number is
// normal, so its bits are above 2^20.)
__device__ __forceinline__ void keep_positive(const float2 (&s)[4], uint32_t (&t)[8]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    t[2 * q] = max(t[2 * q], min(__float_as_uint(s[q].x), 1u << 20));
    t[2 * q + 1] = max(t[2 * q + 1], min(__float_as_uint(s[q].y), 1u << 20));
  }
}

__device__ __forceinline__ void to_nearest(uint32_t (&t)[8]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) t[q] += 0x7ffffu + (t[q] >> 20 & 1u);
}

// The numbers of 8 codes times the block's scale.
__device__ __forceinline__ void decode8(uint2 w, float scale, float2 (&o)[4]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t two = (q & 2 ? w.y : w.x) >> (q & 1 ? 16 : 0);
    uint32_t h;
    asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(h) : "r"(two));
    float lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
    o[q] = mul2(make_float2(lo, hi), both(scale));
  }
}

// ------------------------------------------------------------------- step
struct ListArgs {
  const ListTile* tiles;
  const void* const* grads;
  float* master;
  float *m, *v;                // 32-bit states
  uint8_t *m8, *s8;            // 8-bit states
  float *m_scale, *s_scale;
  uint16_t* const* params;
  const double* norm_sq;
  int* flags;
  int64_t n_tiles, n_state;
  int32_t n_tensors;
  AdamwK k;
  float step_size, inv_bc2_sqrt, max_norm, inv_m;
  Keys keys;
};

__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// AdamW on one element.  What the next state comes from (m, v, sqrt(v)) is
// rounded product by product and sum by sum; the parameter's own step, which
// no state depends on, takes fused products and the fast reciprocal (1 unit in
// the last place; the step's error is about 2^-22 of itself), which takes a
// denominator below the normal numbers for zero: lift_denominator() keeps it
// above them.  V comes in as v and leaves as sqrt(v).  Scalar on purpose: a factor from the constant bank costs a
// scalar product nothing, a paired one two moves.
__device__ __forceinline__ void adamw_elem_sep(float g, const ListArgs& a, float& P, float& M, float& V) {
  const AdamwK& k = a.k;
  M = __fadd_rn(__fmul_rn(M, k.b1), __fmul_rn(g, k.omb1));
  V = __fsqrt_rn(__fadd_rn(__fmul_rn(V, k.b2), __fmul_rn(__fmul_rn(g, k.omb2), g)));
  P = fmaf(M * reciprocal(fmaf(V, a.inv_bc2_sqrt, k.eps)), -a.step_size, P * k.decay);
}

template <typename G, bool k8>
__global__ void __launch_bounds__(LIST_THREADS, 5) list_step_kernel(const __grid_constant__ ListArgs a) {
  const int64_t tile = blockIdx.x;
  const ListTile t = load_tile(a.tiles + tile);
  pdl_wait();
  pdl_trigger();
  if (!GRS_CHECK(tile < a.n_tiles && t.tensor >= 0 && t.tensor < a.n_tensors && t.n > 0 && t.n <= LIST_T &&
                     t.state0 >= 0 && t.state0 + (t.n + 255) / 256 * 256 <= a.n_state,
                 a.flags, SITE_LIST_STEP))
    return;
  const int at = threadIdx.x * 8, first = at & ~255;  // the warp's first element
  if (first >= t.n) return;                           // whole warps beyond the tensor's last block
  const int n = t.n - at;                             // elements of this thread's 8 (may be <= 0 or > 8)
  const G* g = static_cast<const G*>(a.grads[t.tensor]);
  uint16_t* p16 = a.params != nullptr ? a.params[t.tensor] : nullptr;
  const int64_t i = t.state0 + at;
  // The state's loads do not wait for the gradient's pointer.
  float2 P[4], M[4], V[4];
  uint2 mw, sw;
  float m_scale, s_scale;
  load_state8(a.master + i, P);
  if constexpr (k8) {
    mw = __ldcs(reinterpret_cast<const uint2*>(a.m8 + i));
    sw = __ldcs(reinterpret_cast<const uint2*>(a.s8 + i));
    m_scale = a.m_scale[i >> 8];
    s_scale = a.s_scale[i >> 8];
  } else {
    load_state8(a.m + i, M);
    load_state8(a.v + i, V);
  }
  if (g == nullptr) return;
  float2 G2[4];
  g += t.e0 + at;
  load8(g, run_of(g, t.e0 + first, t.rest - first), n, G2);
  const float gscale = a.max_norm > 0.0f ? clip_gscale(*a.norm_sq, a.max_norm, a.inv_m) : a.inv_m;
  if constexpr (k8) {
    decode8(mw, m_scale, M);
    decode8(sw, s_scale, V);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      V[q] = mul2(V[q], V[q]);
      adamw_elem_sep(__fmul_rn(G2[q].x, gscale), a, P[q].x, M[q].x, V[q].x);
      adamw_elem_sep(__fmul_rn(G2[q].y, gscale), a, P[q].y, M[q].y, V[q].y);
    }
    clear_beyond(n, M);
    clear_beyond(n, V);
    const Scale ms = block_scale(warp_absmax(M)), ss = block_scale(warp_absmax(V));
    const uint32_t k0 = a.keys.k0 ^ static_cast<uint32_t>(i >> 32) * MIX_B;
    uint32_t mt[8], st[8];
    code_patterns(M, ms, mt);
    code_patterns(V, ss, st);
    // random_bits() of i ... i + 7, i a multiple of 8: the first fold is the
    // same for all.  m takes the low half of a number, sqrt(v) the high one.
    const uint32_t x0 = static_cast<uint32_t>(i) ^ k0, base = x0 ^ (x0 >> 16);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const uint32_t x = random_rest(base ^ q, a.keys.k1), hi = x >> 12;
      mt[q] += ((x << 4 ^ hi) & 0xffff0u) + 8u;
      st[q] += (hi & 0xffff0u) + 8u;
    }
    keep_positive(V, st);
    __stcs(reinterpret_cast<uint2*>(a.m8 + i), code_bytes<true>(mt, ms.bad));
    __stcs(reinterpret_cast<uint2*>(a.s8 + i), code_bytes<false>(st, ss.bad));
    if ((threadIdx.x & 31) == 0) {
      a.m_scale[i >> 8] = ms.scale;
      a.s_scale[i >> 8] = ss.scale;
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      adamw_elem(G2[q].x, gscale, a.step_size, a.inv_bc2_sqrt, a.k, P[q].x, M[q].x, V[q].x);
      adamw_elem(G2[q].y, gscale, a.step_size, a.inv_bc2_sqrt, a.k, P[q].y, M[q].y, V[q].y);
    }
    clear_beyond(n, M);
    clear_beyond(n, V);
    store_state8(a.m + i, M);
    store_state8(a.v + i, V);
  }
  clear_beyond(n, P);
  store_state8(a.master + i, P);
  if (p16 != nullptr) {
    p16 += t.e0 + at;
    store8(p16, run_of(p16, t.e0 + first, t.rest - first), n, P);
  }
}

// ---------------------------------------------------------- pack / unpack
struct ConvertArgs {
  const ListTile* tiles;
  float *m, *v;
  uint8_t *m8, *s8;
  float *m_scale, *s_scale;
  int* flags;
  int64_t n_tiles, n_state;
};

// The thread's elements of its tile: the place in the state arrays, or -1
// for a warp beyond the tensor's last block; *n = elements of its 8 that the
// tensor has.
__device__ __forceinline__ int64_t convert_at(const ConvertArgs& a, int* n) {
  const int64_t tile = blockIdx.x;
  const ListTile t = load_tile(a.tiles + tile);
  const int at = threadIdx.x * 8;
  *n = t.n - at;
  if (!GRS_CHECK(tile < a.n_tiles && t.n > 0 && t.n <= LIST_T && t.state0 >= 0 &&
                     t.state0 + (t.n + 255) / 256 * 256 <= a.n_state,
                 a.flags, SITE_LIST_STEP))
    return -1;
  return (at & ~255) >= t.n ? -1 : t.state0 + at;
}

__global__ void __launch_bounds__(LIST_THREADS) list_pack8_kernel(const __grid_constant__ ConvertArgs a) {
  pdl_wait();
  pdl_trigger();
  int n;
  const int64_t i = convert_at(a, &n);
  if (i < 0) return;
  float2 M[4], V[4];
  load_state8(a.m + i, M);
  load_state8(a.v + i, V);
#pragma unroll
  for (int q = 0; q < 4; ++q) V[q] = add2(make_float2(__fsqrt_rn(V[q].x), __fsqrt_rn(V[q].y)), both(0.0f));  // -0 to 0
  clear_beyond(n, M);
  clear_beyond(n, V);
  const Scale ms = block_scale(warp_absmax(M)), ss = block_scale(warp_absmax(V));
  uint32_t mt[8], st[8];
  code_patterns(M, ms, mt);
  code_patterns(V, ss, st);
  to_nearest(mt);
  to_nearest(st);
  keep_positive(V, st);
  __stcs(reinterpret_cast<uint2*>(a.m8 + i), code_bytes<true>(mt, ms.bad));
  __stcs(reinterpret_cast<uint2*>(a.s8 + i), code_bytes<false>(st, ss.bad));
  if ((threadIdx.x & 31) == 0) {
    a.m_scale[i >> 8] = ms.scale;
    a.s_scale[i >> 8] = ss.scale;
  }
}

__global__ void __launch_bounds__(LIST_THREADS) list_unpack8_kernel(const __grid_constant__ ConvertArgs a) {
  pdl_wait();
  pdl_trigger();
  int n;
  const int64_t i = convert_at(a, &n);
  if (i < 0) return;
  float2 M[4], V[4];
  decode8(__ldcs(reinterpret_cast<const uint2*>(a.m8 + i)), a.m_scale[i >> 8], M);
  decode8(__ldcs(reinterpret_cast<const uint2*>(a.s8 + i)), a.s_scale[i >> 8], V);
#pragma unroll
  for (int q = 0; q < 4; ++q) V[q] = mul2(V[q], V[q]);
  clear_beyond(n, M);
  clear_beyond(n, V);
  store_state8(a.m + i, M);
  store_state8(a.v + i, V);
}

grs_status check_list(const grs_tensors* l, const char* who) {
  if (l == nullptr) return api_fail(GRS_ERR_INVALID_ARG, who, "list is NULL");
  if (l->device < 0) return api_fail(GRS_ERR_NO_DEVICE, who, "list was created with GRS_PLAN_HOST_ONLY");
  return GRS_OK;
}

grs_status check_step(const grs_tensors* l, const grs_adamw* hp, const double* d_norm_sq, const void* const* d_grads,
                      int32_t grad_dtype, const float* master, uint16_t* const* d_params, const char* who) {
  const grs_status st = check_list(l, who);
  if (st != GRS_OK) return st;
  if (hp == nullptr || d_grads == nullptr || master == nullptr) return api_fail(GRS_ERR_INVALID_ARG, who, "NULL argument");
  if (!dtype_ok(grad_dtype)) return api_fail(GRS_ERR_INVALID_ARG, who, "unknown gradient type");
  if (hp->step < 1 || hp->n_micro < 1) return api_fail(GRS_ERR_INVALID_ARG, who, "step and n_micro must be >= 1");
  if (hp->max_norm > 0.0f && d_norm_sq == nullptr) return api_fail(GRS_ERR_INVALID_ARG, who, "clipping needs d_norm_sq");
  if (!api_aligned(d_grads, 8) || !api_aligned(d_params, 8) || !api_aligned(d_norm_sq, 8) || !api_aligned(master, 16))
    return api_fail(GRS_ERR_ALIGNMENT, who, "misaligned pointer");
  return GRS_OK;
}

ListArgs list_args(const grs_tensors* l, const grs_adamw* hp, const double* d_norm_sq, const void* const* d_grads,
                   float* master, uint16_t* const* d_params) {
  ListArgs a{};
  a.tiles = l->d_tiles;
  a.grads = d_grads;
  a.master = master;
  a.params = d_params;
  a.norm_sq = d_norm_sq;
  a.flags = l->d_flags;
  a.n_tiles = l->n_tiles;
  a.n_state = l->n_state;
  a.n_tensors = static_cast<int32_t>(l->numel.size());
  a.k = adamw_consts(hp);
  bias_factors(hp, hp->step, &a.step_size, &a.inv_bc2_sqrt);
  a.max_norm = hp->max_norm > 0.0f ? hp->max_norm : 0.0f;
  a.inv_m = static_cast<float>(1.0 / static_cast<double>(hp->n_micro));
  return a;
}

// Where eps is so small that it may leave the normal numbers, the denominator
// and the step are both 2^30 as large: powers of two, so the quotient is the
// same.  (The smallest eps is 2^-149, the smallest positive sqrt(v) 2^-75.)
void lift_denominator(ListArgs* a) {
  if (a->k.eps >= 0x1p-100f) return;
  a->k.eps *= 0x1p30f;
  a->inv_bc2_sqrt *= 0x1p30f;
  a->step_size *= 0x1p30f;
}

template <bool k8>
grs_status launch_list_step(const grs_tensors* l, const ListArgs& a, int32_t grad_dtype, void* stream, const char* who) {
  if (l->n_tiles == 0) return GRS_OK;
  ApiDevice dev(l->device);
  if (!dev.ok()) return api_fail(GRS_ERR_CUDA, who, "cannot select the list's device");
  const dim3 grid(static_cast<unsigned>(l->n_tiles)), block(LIST_THREADS);
  const cudaError_t e = grad_dtype == GRS_DTYPE_FP32 ? launch_pdl(list_step_kernel<float, k8>, grid, block, 0, stream, a)
                                                     : launch_pdl(list_step_kernel<uint16_t, k8>, grid, block, 0, stream, a);
  return e == cudaSuccess ? GRS_OK : api_cuda_fail(e, who);
}

}  // namespace
}  // namespace grs

using namespace grs;

extern "C" {

grs_status grs_tensors_create(const int64_t* numels, int32_t n_tensors, uint32_t flags, grs_tensors** out) {
  static const char who[] = "grs_tensors_create";
  if (numels == nullptr || out == nullptr) return api_fail(GRS_ERR_INVALID_ARG, who, "NULL argument");
  if (n_tensors <= 0) return api_fail(GRS_ERR_INVALID_ARG, who, "n_tensors must be >= 1");
  if ((flags & ~GRS_PLAN_HOST_ONLY) != 0) return api_fail(GRS_ERR_INVALID_ARG, who, "unknown flag bits");
  int64_t tiles = 0;
  for (int32_t i = 0; i < n_tensors; ++i) {
    if (numels[i] < 0) return api_fail(GRS_ERR_SHAPE, who, "negative numel");
    // Tiles are blocks of one grid, and offsets stay far inside 64 bits.
    if (numels[i] > int64_t(INT32_MAX) * LIST_T) return api_fail(GRS_ERR_SHAPE, who, "tensor too large");
    tiles += (numels[i] + LIST_T - 1) / LIST_T;
    if (tiles > INT32_MAX) return api_fail(GRS_ERR_SHAPE, who, "list too large");
  }
  grs_tensors* l = nullptr;
  cudaError_t e = cudaSuccess;
  try {
    l = new grs_tensors();
    l->numel.assign(numels, numels + n_tensors);
    std::vector<ListTile> host;
    if ((flags & GRS_PLAN_HOST_ONLY) == 0) host.reserve(static_cast<size_t>(tiles));
    for (int32_t i = 0; i < n_tensors; ++i) {
      l->offset.push_back(l->n_state);
      if ((flags & GRS_PLAN_HOST_ONLY) == 0)
        for (int64_t e0 = 0; e0 < numels[i]; e0 += LIST_T) {
          const int64_t rem = numels[i] - e0;
          host.push_back(ListTile{l->n_state + e0, e0, i, static_cast<int32_t>(rem < LIST_T ? rem : LIST_T), rem});
        }
      l->n_elements += numels[i];
      l->n_state += (numels[i] + GRS_STATE_BLOCK - 1) / GRS_STATE_BLOCK * GRS_STATE_BLOCK;
    }
    l->n_tiles = tiles;
    if ((flags & GRS_PLAN_HOST_ONLY) == 0) {
      int dev = -1;
      e = cudaGetDevice(&dev);
      const size_t bytes = (host.empty() ? 1 : host.size()) * sizeof(ListTile);
      if (e == cudaSuccess) e = cudaMalloc(reinterpret_cast<void**>(&l->d_tiles), bytes);
      if (e == cudaSuccess && !host.empty()) e = cudaMemcpy(l->d_tiles, host.data(), bytes, cudaMemcpyHostToDevice);
      if (e == cudaSuccess) e = cudaMalloc(reinterpret_cast<void**>(&l->d_flags), FLAG_COUNT * sizeof(int));
      if (e == cudaSuccess) e = cudaMemsetAsync(l->d_flags, 0, FLAG_COUNT * sizeof(int), nullptr);
      if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);  // cleared before any launch on any stream
      if (e == cudaSuccess) l->device = dev;
    }
  } catch (...) {  // no memory for the tables
    if (l != nullptr) {
      cudaFree(l->d_tiles);
      cudaFree(l->d_flags);
      delete l;
    }
    return api_fail(GRS_ERR_INVALID_ARG, who, "host allocation failed");
  }
  if (e != cudaSuccess) {
    cudaFree(l->d_tiles);
    cudaFree(l->d_flags);
    delete l;
    return api_cuda_fail(e, who);
  }
  *out = l;
  return GRS_OK;
}

void grs_tensors_destroy(grs_tensors* l) {
  if (l == nullptr) return;
  if (l->device >= 0) {
    ApiDevice dev(l->device);
    cudaFree(l->d_tiles);
    cudaFree(l->d_flags);
  }
  delete l;
}

grs_status grs_tensors_query(const grs_tensors* l, grs_tensors_info* o) {
  if (l == nullptr || o == nullptr) return api_fail(GRS_ERR_INVALID_ARG, "grs_tensors_query", "NULL argument");
  std::memset(o, 0, sizeof(*o));
  o->n_tensors = static_cast<int32_t>(l->numel.size());
  o->device = l->device;
  o->n_elements = l->n_elements;
  o->n_state = l->n_state;
  o->n_blocks = l->n_state / GRS_STATE_BLOCK;
  o->workspace_bytes = LIST_WS_BYTES;
  return GRS_OK;
}

grs_status grs_tensors_offset(const grs_tensors* l, int32_t i, int64_t* out) {
  if (l == nullptr || out == nullptr) return api_fail(GRS_ERR_INVALID_ARG, "grs_tensors_offset", "NULL argument");
  if (i < 0 || i >= static_cast<int32_t>(l->numel.size()))
    return api_fail(GRS_ERR_INVALID_ARG, "grs_tensors_offset", "tensor index out of range");
  *out = l->offset[i];
  return GRS_OK;
}

grs_status grs_tensors_norm_sq(const grs_tensors* l, const void* const* d_grads, int32_t grad_dtype, int32_t n_micro,
                               void* workspace, double* d_norm_sq, void* stream) {
  static const char who[] = "grs_tensors_norm_sq";
  const grs_status st = check_list(l, who);
  if (st != GRS_OK) return st;
  if (d_grads == nullptr || workspace == nullptr || d_norm_sq == nullptr)
    return api_fail(GRS_ERR_INVALID_ARG, who, "NULL argument");
  if (!dtype_ok(grad_dtype)) return api_fail(GRS_ERR_INVALID_ARG, who, "unknown gradient type");
  if (n_micro < 1) return api_fail(GRS_ERR_INVALID_ARG, who, "n_micro must be >= 1");
  if (!api_aligned(d_grads, 8) || !api_aligned(d_norm_sq, 8) || !api_aligned(workspace, 16))
    return api_fail(GRS_ERR_ALIGNMENT, who, "misaligned pointer");
  ApiDevice dev(l->device);
  if (!dev.ok()) return api_fail(GRS_ERR_CUDA, who, "cannot select the list's device");
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  double* partials = reinterpret_cast<double*>(ws);
  unsigned int* ticket = reinterpret_cast<unsigned int*>(ws + LIST_WS_TICKET);
  const int32_t nt = static_cast<int32_t>(l->numel.size());
  const ListTile* tiles = l->d_tiles;
  const int64_t need = (l->n_tiles + LIST_THREADS / 32 - 1) / (LIST_THREADS / 32);
  const dim3 grid(static_cast<unsigned>(need < 1 ? 1 : need < LIST_NORM_BLOCKS ? need : LIST_NORM_BLOCKS)), block(LIST_THREADS);
  const double inv_m = 1.0 / static_cast<double>(n_micro);
  const cudaError_t e =
      grad_dtype == GRS_DTYPE_FP32
          ? launch_pdl(list_norm_kernel<float>, grid, block, 0, stream, tiles, l->n_tiles,
                       reinterpret_cast<const float* const*>(d_grads), nt, partials, ticket, inv_m * inv_m, -0.0f, d_norm_sq,
                       l->d_flags)
          : launch_pdl(list_norm_kernel<uint16_t>, grid, block, 0, stream, tiles, l->n_tiles,
                       reinterpret_cast<const uint16_t* const*>(d_grads), nt, partials, ticket, inv_m * inv_m, -0.0f, d_norm_sq,
                       l->d_flags);
  return e == cudaSuccess ? GRS_OK : api_cuda_fail(e, who);
}

grs_status grs_tensors_adamw_step(const grs_tensors* l, const grs_adamw* hp, const double* d_norm_sq,
                                  const void* const* d_grads, int32_t grad_dtype, float* master, float* m, float* v,
                                  uint16_t* const* d_params_bf16, void* stream) {
  static const char who[] = "grs_tensors_adamw_step";
  const grs_status st = check_step(l, hp, d_norm_sq, d_grads, grad_dtype, master, d_params_bf16, who);
  if (st != GRS_OK) return st;
  if (m == nullptr || v == nullptr) return api_fail(GRS_ERR_INVALID_ARG, who, "NULL argument");
  if (!api_aligned(m, 16) || !api_aligned(v, 16)) return api_fail(GRS_ERR_ALIGNMENT, who, "misaligned pointer");
  ListArgs a = list_args(l, hp, d_norm_sq, d_grads, master, d_params_bf16);
  a.m = m;
  a.v = v;
  return launch_list_step<false>(l, a, grad_dtype, stream, who);
}

grs_status grs_tensors_adamw8_step(const grs_tensors* l, const grs_adamw* hp, uint64_t seed, const double* d_norm_sq,
                                   const void* const* d_grads, int32_t grad_dtype, float* master, uint8_t* m8,
                                   float* m_scale, uint8_t* s8, float* s_scale, uint16_t* const* d_params_bf16,
                                   void* stream) {
  static const char who[] = "grs_tensors_adamw8_step";
  const grs_status st = check_step(l, hp, d_norm_sq, d_grads, grad_dtype, master, d_params_bf16, who);
  if (st != GRS_OK) return st;
  if (m8 == nullptr || s8 == nullptr || m_scale == nullptr || s_scale == nullptr)
    return api_fail(GRS_ERR_INVALID_ARG, who, "NULL argument");
  if (!api_aligned(m8, 16) || !api_aligned(s8, 16) || !api_aligned(m_scale, 4) || !api_aligned(s_scale, 4))
    return api_fail(GRS_ERR_ALIGNMENT, who, "misaligned pointer");
  ListArgs a = list_args(l, hp, d_norm_sq, d_grads, master, d_params_bf16);
  a.m8 = m8;
  a.s8 = s8;
  a.m_scale = m_scale;
  a.s_scale = s_scale;
  a.keys = make_keys(seed);
  lift_denominator(&a);
  return launch_list_step<true>(l, a, grad_dtype, stream, who);
}

static grs_status convert(const grs_tensors* l, float* m, float* v, uint8_t* m8, float* m_scale, uint8_t* s8,
                          float* s_scale, bool pack, void* stream, const char* who) {
  const grs_status st = check_list(l, who);
  if (st != GRS_OK) return st;
  if (m == nullptr || v == nullptr || m8 == nullptr || m_scale == nullptr || s8 == nullptr || s_scale == nullptr)
    return api_fail(GRS_ERR_INVALID_ARG, who, "NULL argument");
  if (!api_aligned(m, 16) || !api_aligned(v, 16) || !api_aligned(m8, 16) || !api_aligned(s8, 16) ||
      !api_aligned(m_scale, 4) || !api_aligned(s_scale, 4))
    return api_fail(GRS_ERR_ALIGNMENT, who, "misaligned pointer");
  if (l->n_tiles == 0) return GRS_OK;
  ApiDevice dev(l->device);
  if (!dev.ok()) return api_fail(GRS_ERR_CUDA, who, "cannot select the list's device");
  const ConvertArgs a{l->d_tiles, m, v, m8, s8, m_scale, s_scale, l->d_flags, l->n_tiles, l->n_state};
  const cudaError_t e = launch_pdl(pack ? list_pack8_kernel : list_unpack8_kernel, dim3(static_cast<unsigned>(l->n_tiles)),
                                 dim3(LIST_THREADS), 0, stream, a);
  return e == cudaSuccess ? GRS_OK : api_cuda_fail(e, who);
}

grs_status grs_tensors_pack8(const grs_tensors* l, const float* m, const float* v, uint8_t* m8, float* m_scale,
                             uint8_t* s8, float* s_scale, void* stream) {
  return convert(l, const_cast<float*>(m), const_cast<float*>(v), m8, m_scale, s8, s_scale, true, stream,
                 "grs_tensors_pack8");
}

grs_status grs_tensors_unpack8(const grs_tensors* l, const uint8_t* m8, const float* m_scale, const uint8_t* s8,
                               const float* s_scale, float* m, float* v, void* stream) {
  return convert(l, m, v, const_cast<uint8_t*>(m8), const_cast<float*>(m_scale), const_cast<uint8_t*>(s8),
                 const_cast<float*>(s_scale), false, stream, "grs_tensors_unpack8");
}

grs_status grs_tensors_check_device_errors(const grs_tensors* l, void* stream) {
  static const char who[] = "grs_tensors_check_device_errors";
  const grs_status st = check_list(l, who);
  if (st != GRS_OK) return st;
  ApiDevice dev(l->device);
  if (!dev.ok()) return api_fail(GRS_ERR_CUDA, who, "cannot select the list's device");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  int h[FLAG_COUNT] = {};
  cudaError_t e = cudaStreamSynchronize(s);
  if (e == cudaSuccess) e = cudaMemcpy(h, l->d_flags, sizeof(h), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaMemsetAsync(l->d_flags, 0, sizeof(h), s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return api_cuda_fail(e, who);
  if (h[FLAG_BOUNDS]) return api_fail(GRS_ERR_BOUNDS, who, "checked build: an index left its buffer");
  if (h[FLAG_NONFINITE]) return api_fail(GRS_ERR_NONFINITE, who, "global gradient norm is not finite");
  return GRS_OK;
}

}  // extern "C"
