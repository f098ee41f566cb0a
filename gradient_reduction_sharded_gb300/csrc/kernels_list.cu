// AdamW over a list of separate tensors (grs_tensors_*): the deterministic
// gradient norm, the fused clip + AdamW + bf16 cast with states in 32 or in
// 8 bits, and the conversion between the two.
//
// Every kernel walks tiles of LIST_T elements, each inside one tensor; a
// device table gives a tile's tensor, its first element there and its place
// in the state arrays.  A thread handles 8 consecutive elements, a warp
// therefore one block of the 8-bit states (256 elements): the block's largest
// magnitude is one warp reduction and no state crosses a warp.
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
  int64_t pad_;
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
  t.pad_ = 0;
  return t;
}

__device__ __forceinline__ float as_float(uint16_t bits) { return __uint_as_float(uint32_t(bits) << 16); }
__device__ __forceinline__ float as_float(float x) { return x; }

// Elements [0, n) of the 8 at p (zeros beyond), one by one.
template <typename G>
__device__ __forceinline__ void load8_slow(const G* p, int n, float (&o)[8]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) o[q] = q < n ? as_float(p[q]) : 0.0f;
}

__device__ __forceinline__ void load8(const uint16_t* p, int n, float (&o)[8]) {
  if (n >= 8 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
    const uint4 w = __ldcs(reinterpret_cast<const uint4*>(p));
    set_bf16x8(o, w);
  } else {
    load8_slow(p, n, o);
  }
}

__device__ __forceinline__ void load8(const float* p, int n, float (&o)[8]) {
  if (n >= 8 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
    o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
  } else {
    load8_slow(p, n, o);
  }
}

__device__ __forceinline__ void load_state8(const float* p, int n, float (&o)[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
  const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
  o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
  if (n < 8) {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q >= n) o[q] = 0.0f;  // state padding may hold anything
  }
}

__device__ __forceinline__ void store_state8(float* p, const float (&o)[8]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(o[0], o[1], o[2], o[3]));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(o[4], o[5], o[6], o[7]));
}

__device__ __forceinline__ void store_bf16x8(uint16_t* p, int n, const float (&o)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * q], o[2 * q + 1]);
    w[q] = *reinterpret_cast<const uint32_t*>(&h);
  }
  if (n >= 8 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < n) p[q] = static_cast<uint16_t>(w[q >> 1] >> (16 * (q & 1)));
  }
}

// ------------------------------------------------------------------- norm
// A sum held as the unevaluated pair hi + lo of floats (Knuth's TwoSum keeps
// each addition's rounding error), about 48 bits: S is then as exact as a sum
// in fp64, whose additions would take several times the time of the loads.
struct Pair {
  float hi, lo;
};

__device__ __forceinline__ void pair_add(Pair& a, float x, float x_lo) {
  const float t = __fadd_rn(a.hi, x);
  const float z = __fsub_rn(t, a.hi);
  const float err = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(t, z)), __fsub_rn(x, z));
  a.lo = __fadd_rn(__fadd_rn(a.lo, x_lo), err);
  a.hi = t;
}

// Sum over 2 * `from` neighbouring lanes; both sides of each exchange compute the same pair.
__device__ __forceinline__ void pair_reduce(Pair& a, int from) {
  for (int o = from; o > 0; o >>= 1) {
    const float h = __shfl_xor_sync(0xffffffffu, a.hi, o), l = __shfl_xor_sync(0xffffffffu, a.lo, o);
    pair_add(a, h, l);
  }
}

// The square's own rounding error; a bf16 number's square is exact.
__device__ __forceinline__ float square_err(float x, float sq, float) { return __fmaf_rn(x, x, -sq); }
__device__ __forceinline__ float square_err(float, float, uint16_t) { return 0.0f; }

// partials[tile] = sum of squares of the tile, in a fixed order.
template <typename G>
__global__ void __launch_bounds__(LIST_THREADS) list_norm_kernel(const ListTile* __restrict__ tiles, int64_t n_tiles,
                                                                 const G* const* __restrict__ grads, int32_t n_tensors,
                                                                 double* __restrict__ partials, int* __restrict__ flags) {
  __shared__ Pair red[LIST_THREADS / 32];
  const int64_t tile = blockIdx.x;
  const ListTile t = load_tile(tiles + tile);
  pdl_wait();
  pdl_trigger();
  const bool ok = GRS_CHECK(tile < n_tiles && t.tensor >= 0 && t.tensor < n_tensors && t.n >= 0 && t.n <= LIST_T,
                            flags, SITE_LIST_NORM);
  const G* g = ok ? grads[t.tensor] : nullptr;
  const int at = threadIdx.x * 8;
  Pair s = {0.0f, 0.0f};
  if (g != nullptr && at < t.n) {
    float x[8];
    load8(g + t.e0 + at, t.n - at, x);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float sq = __fmul_rn(x[q], x[q]);
      pair_add(s, sq, square_err(x[q], sq, G()));
    }
  }
  pair_reduce(s, 16);
  const int lane = threadIdx.x & 31;
  if (lane == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  s = red[lane & (LIST_THREADS / 32 - 1)];
  pair_reduce(s, LIST_THREADS / 64);
  // An infinite or NaN sum has no error term (inf - inf is NaN).
  if (lane == 0) partials[tile] = isfinite(s.hi) ? static_cast<double>(s.hi) + static_cast<double>(s.lo) : static_cast<double>(s.hi);
}

// *out = inv_m2 * the sum of the partials in fp64: block b of NORM_L2_BLOCKS
// sums a contiguous range, the block that is last (the ticket) the blocks'
// sums, every addition in a fixed order.
__device__ __forceinline__ double block_sum(double x, double* red) {
  x = warp_sum(x);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  double s = red[0];
  for (int k = 1; k < LIST_THREADS / 32; ++k) s = __dadd_rn(s, red[k]);
  return s;
}

__global__ void __launch_bounds__(LIST_THREADS) list_norm_finish_kernel(const double* __restrict__ partials, int64_t n,
                                                                        double* __restrict__ level2,
                                                                        unsigned int* __restrict__ ticket, double inv_m2,
                                                                        double* __restrict__ out, int* __restrict__ flags) {
  __shared__ double red[LIST_THREADS / 32];
  __shared__ bool last;
  pdl_wait();
  pdl_trigger();
  const int64_t chunk = (n + NORM_L2_BLOCKS - 1) / NORM_L2_BLOCKS;
  const int64_t lo = blockIdx.x * chunk, hi = lo + chunk < n ? lo + chunk : n;
  double s = 0.0;
  for (int64_t i = lo + threadIdx.x; i < hi; i += LIST_THREADS) s = __dadd_rn(s, partials[i]);
  s = block_sum(s, red);
  if (threadIdx.x == 0) {
    level2[blockIdx.x] = s;
    __threadfence();
    last = atomicAdd(ticket, 1u) == NORM_L2_BLOCKS - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  s = block_sum(threadIdx.x < NORM_L2_BLOCKS ? __ldcg(level2 + threadIdx.x) : 0.0, red);
  if (threadIdx.x == 0) {
    s = __dmul_rn(s, inv_m2);
    *out = s;
    if (!isfinite(s)) atomicOr(flags + FLAG_NONFINITE, 1);
    *ticket = 0u;
  }
}

// Workspace of the norm: [n_tiles doubles][NORM_L2_BLOCKS doubles][ticket].
int64_t list_ws_level2(int64_t n_tiles) { return (n_tiles * 8 + 255) / 256 * 256; }
int64_t list_ws_ticket(int64_t n_tiles) { return list_ws_level2(n_tiles) + NORM_L2_BLOCKS * 8; }
int64_t list_ws_bytes(int64_t n_tiles) { return list_ws_ticket(n_tiles) + 256; }

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

// `lo`: low word of the element's index; k0 carries the high word's part.
__device__ __forceinline__ uint32_t random_bits(uint32_t lo, uint32_t k0, uint32_t k1) {
  uint32_t x = lo ^ k0;
  x = (x ^ (x >> 16)) * MIX_A ^ k1;
  x = (x ^ (x >> 15)) * MIX_C;
  return x ^ (x >> 16);
}

// The scale of a block whose largest magnitude has the bits `top`:
// 2^(ceil(log2 x) - 8), at least 2^-126, NaN when x is not finite.  ceil, so
// that a largest magnitude that was rounded up to a power of two keeps its
// scale when it is packed again.
struct Scale {
  float scale, inv;
  bool bad;
};
__device__ __forceinline__ Scale block_scale(uint32_t top) {
  Scale s;
  s.bad = top >= 0x7f800000u;
  int e = static_cast<int>((top + 0x7fffffu) >> 23) - 8;
  e = e < 1 ? 1 : e;
  s.inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
  s.scale = s.bad ? __uint_as_float(0x7fc00000u) : __uint_as_float(static_cast<uint32_t>(e) << 23);
  if (s.bad) s.inv = 0.0f;
  return s;
}

// Largest magnitude of the warp's 256 values, as bits (ordered like the
// values, NaN above infinity).
__device__ __forceinline__ uint32_t warp_absmax(const float (&x)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) top = max(top, __float_as_uint(x[q]) & 0x7fffffffu);
  return __reduce_max_sync(0xffffffffu, top);
}

// E4M3 code of x / scale.  Times 2^-120 an E4M3 number (bias 7) has its own
// exponent and subnormals as binary32 (bias 127), so the code is the top of
// the binary32 pattern, and adding to the 20 bits below it before they are
// cut off rounds: a random number below 2^20 stochastically, the usual
// half-minus-one plus the last bit kept to nearest even.
__device__ __forceinline__ uint32_t code_bits(float x, float inv) {
  return __float_as_uint(__fmul_rn(__fmul_rn(fabsf(x), inv), 0x1p-120f));
}
__device__ __forceinline__ uint32_t sign_bit(float x) { return (__float_as_uint(x) >> 24) & 0x80u; }

// The value of a code (in the low byte of `code`) in units of 1.
__device__ __forceinline__ float code_value(uint32_t code) {
  const float y = __uint_as_float((code & 0x7fu) << 20) * 0x1p120f;
  return __uint_as_float(__float_as_uint(y) | (code & 0x80u) << 24);
}

__device__ __forceinline__ void decode8(uint2 w, float scale, float (&o)[8]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) o[q] = __fmul_rn(code_value((q < 4 ? w.x : w.y) >> (8 * (q & 3))), scale);
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

// AdamW on one element with every product and sum rounded by itself;
// returns sqrt(v).
__device__ __forceinline__ float adamw_elem_sep(float g, float step_size, float inv_bc2_sqrt, const AdamwK& k,
                                                float& P, float& M, float V) {
  M = __fadd_rn(__fmul_rn(M, k.b1), __fmul_rn(g, k.omb1));
  V = __fadd_rn(__fmul_rn(V, k.b2), __fmul_rn(__fmul_rn(g, k.omb2), g));
  const float s = __fsqrt_rn(V);
  const float upd = __fdiv_rn(M, __fadd_rn(__fmul_rn(s, inv_bc2_sqrt), k.eps));
  P = __fsub_rn(__fmul_rn(P, k.decay), __fmul_rn(upd, step_size));
  return s;
}

template <typename G, bool k8>
__global__ void __launch_bounds__(LIST_THREADS) list_step_kernel(const __grid_constant__ ListArgs a) {
  const int64_t tile = blockIdx.x;
  const ListTile t = load_tile(a.tiles + tile);
  pdl_wait();
  pdl_trigger();
  if (!GRS_CHECK(tile < a.n_tiles && t.tensor >= 0 && t.tensor < a.n_tensors && t.n > 0 && t.n <= LIST_T &&
                     t.state0 >= 0 && t.state0 + (t.n + 255) / 256 * 256 <= a.n_state,
                 a.flags, SITE_LIST_STEP))
    return;
  const G* g = static_cast<const G*>(a.grads[t.tensor]);
  if (g == nullptr) return;
  const int at = threadIdx.x * 8;
  if ((at & ~255) >= t.n) return;  // whole warps beyond the tensor's last block
  const int n = t.n - at;          // elements of this thread's 8 (may be <= 0 or > 8)
  uint16_t* p16 = a.params != nullptr ? a.params[t.tensor] : nullptr;
  const float gscale = a.max_norm > 0.0f ? clip_gscale(*a.norm_sq, a.max_norm, a.inv_m) : a.inv_m;
  const int64_t i = t.state0 + at;
  float G8[8], P[8], M[8], V[8];
  load8(g + t.e0 + at, n, G8);
  load_state8(a.master + i, n, P);
  if (k8) {
    const uint2 mw = __ldcs(reinterpret_cast<const uint2*>(a.m8 + i));
    const uint2 sw = __ldcs(reinterpret_cast<const uint2*>(a.s8 + i));
    decode8(mw, a.m_scale[i >> 8], M);
    decode8(sw, a.s_scale[i >> 8], V);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      V[q] = __fmul_rn(V[q], V[q]);
      V[q] = adamw_elem_sep(__fmul_rn(G8[q], gscale), a.step_size, a.inv_bc2_sqrt, a.k, P[q], M[q], V[q]);
      if (q >= n) P[q] = M[q] = V[q] = 0.0f;
    }
    const Scale ms = block_scale(warp_absmax(M)), ss = block_scale(warp_absmax(V));
    const uint32_t k0 = a.keys.k0 ^ static_cast<uint32_t>(i >> 32) * MIX_B;
    uint32_t mo[2] = {0, 0}, so[2] = {0, 0};
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const uint32_t r = random_bits(static_cast<uint32_t>(i) + q, k0, a.keys.k1);
      uint32_t mc = (code_bits(M[q], ms.inv) + ((r & 0xffffu) << 4 | 8u)) >> 20 | sign_bit(M[q]);
      uint32_t sc = (code_bits(V[q], ss.inv) + ((r >> 16) << 4 | 8u)) >> 20;
      if (V[q] > 0.0f && sc == 0) sc = 1;
      if (ms.bad) mc = 0;
      if (ss.bad) sc = 0;
      mo[q >> 2] |= mc << (8 * (q & 3));
      so[q >> 2] |= sc << (8 * (q & 3));
    }
    __stcs(reinterpret_cast<uint2*>(a.m8 + i), make_uint2(mo[0], mo[1]));
    __stcs(reinterpret_cast<uint2*>(a.s8 + i), make_uint2(so[0], so[1]));
    if ((threadIdx.x & 31) == 0) {
      a.m_scale[i >> 8] = ms.scale;
      a.s_scale[i >> 8] = ss.scale;
    }
  } else {
    load_state8(a.m + i, n, M);
    load_state8(a.v + i, n, V);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      adamw_elem(G8[q], gscale, a.step_size, a.inv_bc2_sqrt, a.k, P[q], M[q], V[q]);
      if (q >= n) P[q] = M[q] = V[q] = 0.0f;
    }
    store_state8(a.m + i, M);
    store_state8(a.v + i, V);
  }
  store_state8(a.master + i, P);
  if (p16 != nullptr && n > 0) store_bf16x8(p16 + t.e0 + at, n, P);
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
  float M[8], V[8];
  load_state8(a.m + i, n, M);
  load_state8(a.v + i, n, V);
#pragma unroll
  for (int q = 0; q < 8; ++q) V[q] = __fsqrt_rn(V[q]);
  const Scale ms = block_scale(warp_absmax(M)), ss = block_scale(warp_absmax(V));
  uint32_t mo[2] = {0, 0}, so[2] = {0, 0};
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint32_t mb = code_bits(M[q], ms.inv), sb = code_bits(V[q], ss.inv);
    uint32_t mc = (mb + 0x7ffffu + (mb >> 20 & 1u)) >> 20 | sign_bit(M[q]);
    uint32_t sc = (sb + 0x7ffffu + (sb >> 20 & 1u)) >> 20;
    if (V[q] > 0.0f && sc == 0) sc = 1;
    if (ms.bad) mc = 0;
    if (ss.bad) sc = 0;
    mo[q >> 2] |= mc << (8 * (q & 3));
    so[q >> 2] |= sc << (8 * (q & 3));
  }
  __stcs(reinterpret_cast<uint2*>(a.m8 + i), make_uint2(mo[0], mo[1]));
  __stcs(reinterpret_cast<uint2*>(a.s8 + i), make_uint2(so[0], so[1]));
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
  float M[8], V[8];
  decode8(__ldcs(reinterpret_cast<const uint2*>(a.m8 + i)), a.m_scale[i >> 8], M);
  decode8(__ldcs(reinterpret_cast<const uint2*>(a.s8 + i)), a.s_scale[i >> 8], V);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    V[q] = __fmul_rn(V[q], V[q]);
    if (q >= n) M[q] = V[q] = 0.0f;
  }
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
          host.push_back(ListTile{l->n_state + e0, e0, i, static_cast<int32_t>(rem < LIST_T ? rem : LIST_T), 0});
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
  } catch (const std::bad_alloc&) {
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
  o->workspace_bytes = list_ws_bytes(l->n_tiles);
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
  double* level2 = reinterpret_cast<double*>(ws + list_ws_level2(l->n_tiles));
  unsigned int* ticket = reinterpret_cast<unsigned int*>(ws + list_ws_ticket(l->n_tiles));
  const int32_t nt = static_cast<int32_t>(l->numel.size());
  cudaError_t e = cudaSuccess;
  if (l->n_tiles > 0) {
    const dim3 grid(static_cast<unsigned>(l->n_tiles)), block(LIST_THREADS);
    const ListTile* tiles = l->d_tiles;
    e = grad_dtype == GRS_DTYPE_FP32
            ? launch_pdl(list_norm_kernel<float>, grid, block, 0, stream, tiles, l->n_tiles,
                       reinterpret_cast<const float* const*>(d_grads), nt, partials, l->d_flags)
            : launch_pdl(list_norm_kernel<uint16_t>, grid, block, 0, stream, tiles, l->n_tiles,
                       reinterpret_cast<const uint16_t* const*>(d_grads), nt, partials, l->d_flags);
  }
  if (e != cudaSuccess) return api_cuda_fail(e, who);
  const double inv_m = 1.0 / static_cast<double>(n_micro);
  e = launch_pdl(list_norm_finish_kernel, dim3(NORM_L2_BLOCKS), dim3(LIST_THREADS), 0, stream, partials, l->n_tiles, level2,
               ticket, inv_m * inv_m, d_norm_sq, l->d_flags);
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
