// Root-mean-square norms of query and key heads with the rotation by position
// in the same pass, forward and backward.
//
// A head x of D elements: r = 1 / sqrt(sum x^2 / D + eps), h = x r, u = h w,
// and the first elements of u in pairs (a, b) turned by the position's angle.
// Backward turns the gradient back, so du = R^T dy, and with dh = du w
//   dx = r (dh - h sum(dh h) / D),   dw = sum over tokens and heads of du h.
// r is computed again from x, which backward reads in any case.
//
// Heads of whole 16-byte chunks are bound by memory and instruction issue
// together: 16384 tokens, 16 + 16 heads of 128 bf16, forward 48 us (5.6 TB/s,
// issue 71 %); 32 + 4 heads of 64, backward 43 (5.2 TB/s, issue 56 %; reads 151
// MB).  Others go a warp a head, element by element (forward 203, backward 331
// for the same).  Pairs kept in 64-bit registers changed nothing (50 and 45).
//
// Angles: a frequency is a fraction of a turn, rounded to 64 bits, and a position
// times it modulo 2^64 the fraction of its angle: the product adds no rounding,
// and the frequency's grows to 2^-33 of a turn at position 2^31.  Its upper 32
// bits go to sincospi.
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

// kExact: to two units; otherwise, where every result is rounded to bf16, to
// 2^-21 (a half step of bf16 is 2^-8).
template <bool kExact>
__device__ __forceinline__ float2 turn_of(int32_t position, uint64_t turns) {
  const uint64_t a = static_cast<uint64_t>(int64_t(position)) * turns + 0x80000000u;
  const float half_turns = static_cast<float>(static_cast<int32_t>(a >> 32)) * 0x1p-31f;
  float2 cs;
  if constexpr (kExact) sincospif(half_turns, &cs.y, &cs.x);
  else __sincosf(half_turns * 3.14159265358979f, &cs.y, &cs.x);
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
    const float2 cs = angles ? turn_of<true>(pos, __ldg(a.turns + p)) : make_float2(1.0f, 0.0f);
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

// ------------------------------------------------- heads of whole 16-byte chunks
// A head is shared by LANES lanes, 16 of its elements each: with the pairs (i,
// i + rot / 2) eight from either half, so that a lane has both of a pair, with
// neighbouring pairs 16 in a row.  A block takes the heads of a few tokens: it
// puts the tokens' sines and cosines into shared memory, each computed once
// for all heads, and its lane groups take the heads in turn, the next head's
// loads on their way while one is computed.
constexpr int QK_MAX_UNITS = 32;       // 16-element units of a head
// Measured, us (forward of 16384 tokens, 16 + 16 heads of 128; backward of 32 + 4 heads of 64): forward with 4, 6 and 12
// heads of a group in a tile 49, 47.8, 48.8; backward with 4, 8 and 12 48.7, 44.6, 43.2, with three blocks an SM
// (80 registers) and 8 48.5.
constexpr int QK_FWD_ROUNDS = 6;       // heads of a lane group in a tile of tokens
constexpr int QK_BWD_ROUNDS = 12;
constexpr int QK_FWD_BLOCKS = 4;       // an SM
constexpr int QK_BWD_BLOCKS = 2;
constexpr int QK_FWD_DEPTH = 4;        // heads of a thread on their way
template <typename T>
constexpr int qk_bwd_depth = sizeof(T) == 2 ? 4 : 2;
constexpr int QK_TABLE = 32 * 1024;    // bytes of sines and cosines at most
constexpr int QK_MAX_TOKENS = 128;     // of a block
constexpr int64_t QK_MAX_LD = 1 << 22; // elements between tokens: those of a block, and one step further, lie within 2^31

struct QkShape {
  int units, turned, lanes;  // units of a head, of them with a rotated part; lanes that share a head (a power of 2)
  int tokens;                // of a block
  int slots;                 // lane groups of a block
  int dt[2], dh[2];          // tokens and heads from one of a group's queries, keys, to its next
};

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 shared16(uint32_t from) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(from) : "memory");
  return v;
}

template <typename T>
__device__ __forceinline__ void store_chunk(T* p, const float2* v) {
  if constexpr (sizeof(T) == 2) {
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(to_bf16_pair(v[0]), to_bf16_pair(v[1]), to_bf16_pair(v[2]), to_bf16_pair(v[3])));
  } else {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0].x, v[0].y, v[1].x, v[1].y));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[2].x, v[2].y, v[3].x, v[3].y));
  }
}

// The lane's 16 elements: eight from i0, eight from i1 (-1: none), and whether
// these are turned.  Neighbouring lanes have neighbouring chunks in either half.
template <bool kPairs>
struct Unit {
  int i0, i1;
  bool r0, r1;
  __device__ __forceinline__ Unit(int u, int units, int d, int rot) {
    const int halves = kPairs ? 0 : rot / 16, from = kPairs ? 0 : rot;  // units of two turned halves, and what comes behind them
    if (u >= units) {
      i0 = i1 = -1;
      r0 = r1 = false;
    } else if (u >= halves) {
      i0 = from + 8 * (u - halves);
      i1 = i0 + 8 * (units - halves);
      if (i1 >= d) i1 = -1;
      r0 = kPairs && i0 < rot;
      r1 = kPairs && i1 >= 0 && i1 < rot;
    } else {
      i0 = 8 * u;
      i1 = 8 * u + rot / 2;
      r0 = r1 = true;
    }
  }
  // Where angle p of a token is in the table: entry [q][u], its place there.
  static __device__ __forceinline__ int angle_at(int p, int turned) {
    if constexpr (kPairs) {
      const int c = p / 4, h = c >= turned;
      return ((2 * h + p % 4 / 2) * turned + c - h * turned) * 4 + p % 2;
    }
    return (p % 8 / 2 * turned + p / 8) * 4 + p % 2;
  }
  // v turned by the unit's eight angles, or back: entry q has (cos, cos, sin, sin) of its angles 2 q and 2 q + 1.
  template <bool kBack>
  __device__ __forceinline__ void turn(float2 (&v)[8], const float4* table, int turned) const {
    if (!r0) return;  // (r1 without r0 there is not)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (kPairs && q >= 2 && !r1) break;
      const float4 t = table[q * turned];
      if constexpr (kPairs) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float c = k == 0 ? t.x : t.y, s = kBack ? -(k == 0 ? t.z : t.w) : (k == 0 ? t.z : t.w);
          const float2 a = v[2 * q + k];
          v[2 * q + k] = make_float2(__fmaf_rn(a.x, c, -(a.y * s)), __fmaf_rn(a.x, s, a.y * c));
        }
      } else {
        const float2 c = make_float2(t.x, t.y), s = make_float2(t.z, t.w), m = make_float2(-t.z, -t.w), a = v[q], b = v[q + 4];
        v[q] = fma2(b, kBack ? s : m, mul2(a, c));
        v[q + 4] = fma2(a, kBack ? m : s, mul2(b, c));
      }
    }
  }
};

__device__ __forceinline__ float lanes_sum(float x, int lanes) {
#pragma unroll
  for (int o = 1; o < 32; o *= 2)
    if (o < lanes) x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// Shared memory of a block: the angles of its tokens, [token][4][turned] of
// (cos, cos, sin, sin), and the weights, [2][4][units] of four.
template <typename T, typename P, bool kPairs>
__device__ __forceinline__ void qk_weights_to_smem(const QkArgs<T, P>& a, const QkShape& s, float* w) {
  for (int i = threadIdx.x; i < 2 * 16 * s.units; i += QK_THREADS) {
    const int which = i >= 16 * s.units, k = i - which * 16 * s.units, u = k / 16, j = k % 16;
    const Unit<kPairs> x(u, s.units, a.d, a.rot);
    const int at = j < 8 ? x.i0 + j : x.i1 + j - 8;
    const bool on = (j < 8 || x.i1 >= 0) && a.heads[which] > 0;
    w[((which * 4 + j / 4) * s.units + u) * 4 + j % 4] = on ? weight(a, which, at) : 0.0f;
  }
}
// A thread's angles, the i-th with i = its number plus a multiple of the
// block's threads: the first one's position can be asked for ahead.
template <typename T, typename P, bool kPairs, bool kExact>
struct Angles {
  const QkArgs<T, P>& a;
  const QkShape& s;
  int t, p;
  int32_t ahead = 0;
  __device__ __forceinline__ Angles(const QkArgs<T, P>& a_, const QkShape& s_) : a(a_), s(s_) {
    const int half = a.rot / 2;
    t = half > 0 ? threadIdx.x / half : 0;
    p = threadIdx.x - t * half;
  }
  __device__ __forceinline__ void ask(int64_t t0, int tokens) {
    if (a.rot > 0 && t < tokens) ahead = __ldg(a.positions + t0 + t);
  }
  __device__ __forceinline__ void put(float* table, int ti, int pi, int32_t position) const {
    const float2 cs = turn_of<kExact>(position, __ldg(a.turns + pi));
    float* o = table + ti * 16 * s.turned + Unit<kPairs>::angle_at(pi, s.turned);
    o[0] = cs.x;
    o[2] = cs.y;
  }
  __device__ __forceinline__ void store(int64_t t0, int tokens, float* table) const {
    const int half = a.rot / 2;
    if (half == 0) return;
    if (t < tokens) put(table, t, p, ahead);
    for (int i = threadIdx.x + QK_THREADS; i < tokens * half; i += QK_THREADS) {
      const int ti = i / half, pi = i - ti * half;
      put(table, ti, pi, __ldg(a.positions + t0 + ti));
    }
  }
};

// A lane group's way through the heads of a block's tokens, queries or keys:
// every slots-th, and where they lie in the inputs and in the outputs.
struct Way {
  int t, h;
  int32_t x, y;  // from the block's first token on; QK_MAX_LD keeps them in 32 bits
  template <typename T, typename P>
  __device__ __forceinline__ Way(const QkArgs<T, P>& a, int w, int slot) {
    const int n = a.heads[w];
    t = n > 0 ? slot / n : 0;
    h = slot - t * n;
    x = t * static_cast<int32_t>(a.ld_x[w]) + h * a.d;
    y = t * static_cast<int32_t>(a.ld_y[w]) + h * a.d;
  }
  template <typename T, typename P>
  __device__ __forceinline__ void step(const QkArgs<T, P>& a, const QkShape& s, int w) {
    const int n = a.heads[w], ld_x = static_cast<int32_t>(a.ld_x[w]), ld_y = static_cast<int32_t>(a.ld_y[w]);
    t += s.dt[w];
    h += s.dh[w];
    x += s.dt[w] * ld_x + s.dh[w] * a.d;
    y += s.dt[w] * ld_y + s.dh[w] * a.d;
    if (h >= n) {
      h -= n;
      ++t;
      x += ld_x - n * a.d;
      y += ld_y - n * a.d;
    }
  }
};

// The heads that a thread's copies are under way for: ahead of those that it
// computes, in the same order (queries of a tile of tokens, keys, the next
// tile), so that the memory is busy across all of these ends.  A thread copies
// what it reads itself; what has no place in memory stays zeros.
template <typename T, typename P, int kInputs, int kDepth>
struct Stream {
  static_assert((kDepth & (kDepth - 1)) == 0, "a power of two");
  static constexpr int N = static_cast<int>(sizeof(T)) / 2;  // 16-byte pieces of 8 elements
  static constexpr int PIECE = 16 * QK_THREADS, SLOT = kInputs * 2 * N * PIECE, BYTES = kDepth * SLOT;
  const QkArgs<T, P>& a;
  const QkShape& s;
  uint32_t ring;    // [kDepth][input][half][piece][threads] of 16 bytes, this thread's
  int64_t t0, end;  // of the tile, of the block's tokens
  int slot, i0, i1, tokens, which, left, at;  // at: bytes into the ring
  Way way;
  const T *x, *dy;                     // of the tile's queries or keys
  int n, dt, dh, dx, dy_, wrap_x, wrap_y;  // and the steps of their way

  __device__ __forceinline__ Stream(const QkArgs<T, P>& a_, const QkShape& s_, uint4* ring_, int64_t first, int64_t end_, int slot_, int i0_, int i1_)
      : a(a_), s(s_), ring(smem_addr(ring_ + threadIdx.x)), t0(first), end(end_), slot(slot_), i0(i0_), i1(i1_), which(-1), at(0), way(a_, 0, slot_) {
#pragma unroll
    for (int i = 0; i < BYTES / PIECE; ++i) ring_[i * QK_THREADS + threadIdx.x] = make_uint4(0, 0, 0, 0);
    tokens = count(t0);
    next_part();
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) ask();
  }
  __device__ __forceinline__ int count(int64_t t) const { return t >= end ? 0 : end - t < s.tokens ? static_cast<int>(end - t) : s.tokens; }
  __device__ __forceinline__ int rounds(int w, int of) const { return (of * a.heads[w] + s.slots - 1) / s.slots; }
  __device__ __forceinline__ void next_part() {
    if (tokens == 0) return;
    do {
      if (++which == 2) {
        which = 0;
        t0 += s.tokens;
        tokens = count(t0);
        if (tokens == 0) return;
      }
      left = rounds(which, tokens);
    } while (left == 0);
    const int32_t ld_x = static_cast<int32_t>(a.ld_x[which]), ld_y = static_cast<int32_t>(a.ld_y[which]);
    way = Way(a, which, slot);
    n = a.heads[which];
    dt = s.dt[which];
    dh = s.dh[which];
    dx = dt * ld_x + dh * a.d;
    dy_ = dt * ld_y + dh * a.d;
    wrap_x = ld_x - n * a.d;
    wrap_y = ld_y - n * a.d;
    x = a.x[which] + t0 * a.ld_x[which];
    if constexpr (kInputs == 2) dy = a.dy[which] + t0 * a.ld_y[which];
  }
  __device__ __forceinline__ void ask() {
    if (tokens > 0) {
      if (way.t < tokens) {
        copy(ring + at, x + way.x);
        if constexpr (kInputs == 2) copy(ring + at + 2 * N * PIECE, dy + way.y);
      }
      way.t += dt;
      way.h += dh;
      way.x += dx;
      if constexpr (kInputs == 2) way.y += dy_;
      if (way.h >= n) {
        way.h -= n;
        ++way.t;
        way.x += wrap_x;
        if constexpr (kInputs == 2) way.y += wrap_y;
      }
      if (--left == 0) next_part();
    }
    copies_commit();
    at = (at + SLOT) & (BYTES - 1);
  }
  __device__ __forceinline__ void copy(uint32_t to, const T* from) const {
    if (i0 >= 0)
#pragma unroll
      for (int k = 0; k < N; ++k) copy16(to + k * PIECE, reinterpret_cast<const uint4*>(from + i0) + k);
    if (i1 >= 0)
#pragma unroll
      for (int k = 0; k < N; ++k) copy16(to + (N + k) * PIECE, reinterpret_cast<const uint4*>(from + i1) + k);
  }
  // The next head: asks for a later one, waits for this one's copies.
  __device__ __forceinline__ uint32_t next() {
    const uint32_t from = ring + ((at + SLOT) & (BYTES - 1));
    ask();
    copies_wait<kDepth - 1>();
    return from;
  }
  template <int kInput>
  static __device__ __forceinline__ void get(uint32_t from, float2 (&v)[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const uint4 c = shared16(from + ((kInput * 2 + h) * N + k) * PIECE);
        if constexpr (sizeof(T) == 2) {
          v[4 * h] = bf16_pair(c.x);
          v[4 * h + 1] = bf16_pair(c.y);
          v[4 * h + 2] = bf16_pair(c.z);
          v[4 * h + 3] = bf16_pair(c.w);
        } else {
          v[4 * h + 2 * k] = make_float2(__uint_as_float(c.x), __uint_as_float(c.y));
          v[4 * h + 2 * k + 1] = make_float2(__uint_as_float(c.z), __uint_as_float(c.w));
        }
      }
  }
};

// A block's tokens follow one another: [block_token(b), block_token(b + 1)).
__device__ __forceinline__ int64_t block_token(int64_t tokens, unsigned b) {
  const int64_t each = tokens / gridDim.x, more = tokens % gridDim.x;
  return each * b + (more < b ? more : b);
}

__device__ __forceinline__ float squares_sum(const float2 (&v)[8]) {
  float2 s = mul2(v[0], v[0]);
#pragma unroll
  for (int q = 1; q < 8; ++q) s = fma2(v[q], v[q], s);
  return s.x + s.y;
}

// The heads of one kind of a block's tokens.
template <int W, typename T, typename P, bool kPairs, typename S>
__device__ __forceinline__ void qk_forward_heads(const QkArgs<T, P>& a, const QkShape& s, int64_t t0, int tokens, const Unit<kPairs>& unit, int u,
                                                 const float4* table, const float4* weights, S& stream) {
  const int rounds = stream.rounds(W, tokens);  // whole warps stay together for the sums
  T* const o = a.o[W] + t0 * a.ld_y[W];
  Way way(a, W, stream.slot);
#pragma unroll 1
  for (int r = 0; r < rounds; ++r) {
    float2 v[8];
    S::template get<0>(stream.next(), v);
    const float rs = rsqrtf(__fmaf_rn(lanes_sum(squares_sum(v), s.lanes), a.inv_d, a.eps));
    if (way.t < tokens && unit.i0 >= 0 && GRS_CHECK(way.h < a.heads[W], qk_flags, SITE_QK_HEAD)) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 k = weights[(W * 4 + q) * s.units + u];
        v[2 * q] = mul2(mul2(v[2 * q], both(rs)), make_float2(k.x, k.y));
        v[2 * q + 1] = mul2(mul2(v[2 * q + 1], both(rs)), make_float2(k.z, k.w));
      }
      unit.template turn<false>(v, table + way.t * 4 * s.turned + u, s.turned);
      store_chunk(o + way.y + unit.i0, v);
      if (unit.i1 >= 0) store_chunk(o + way.y + unit.i1, v + 4);
    }
    way.step(a, s, W);
  }
}

template <typename T, typename P, bool kPairs>
__global__ void __launch_bounds__(QK_THREADS, QK_FWD_BLOCKS) qk_forward_whole_kernel(const __grid_constant__ QkArgs<T, P> a, const __grid_constant__ QkShape s) {
  extern __shared__ float4 shared[];
  const int entries = s.tokens * 4 * s.turned;  // of a table of angles; there are two
  float4* weights = shared + 2 * entries;
  pdl_wait();
  pdl_trigger();
  const int slot = threadIdx.x / s.lanes, u = threadIdx.x - slot * s.lanes;
  const Unit<kPairs> unit(u, s.units, a.d, a.rot);
  const int64_t end = block_token(a.tokens, blockIdx.x + 1);
  int64_t t0 = block_token(a.tokens, blockIdx.x);
  Angles<T, P, kPairs, sizeof(T) == 4> angles(a, s);  // (exact for bf16 too: 47.9 -> 48.4 us)
  Stream<T, P, 1, QK_FWD_DEPTH> stream(a, s, reinterpret_cast<uint4*>(weights + 8 * s.units), t0, end, slot, unit.i0, unit.i1);
  qk_weights_to_smem<T, P, kPairs>(a, s, reinterpret_cast<float*>(weights));
  angles.ask(t0, stream.count(t0));
  for (int flip = 0; t0 < end; t0 += s.tokens, flip ^= 1) {
    const int tokens = stream.count(t0);
    float4* table = shared + flip * entries;
    angles.store(t0, tokens, reinterpret_cast<float*>(table));
    angles.ask(t0 + s.tokens, stream.count(t0 + s.tokens));
    __syncthreads();  // (the other table is free: all are done with the tile before)
    if (a.heads[0] > 0) qk_forward_heads<0>(a, s, t0, tokens, unit, u, table, weights, stream);
    if (a.heads[1] > 0) qk_forward_heads<1>(a, s, t0, tokens, unit, u, table, weights, stream);
  }
}

// Backward, likewise; dw: the lane's share of the weight's gradient.
template <int W, typename T, typename P, bool kPairs, typename S>
__device__ __forceinline__ void qk_backward_heads(const QkArgs<T, P>& a, const QkShape& s, int64_t t0, int tokens, const Unit<kPairs>& unit, int u,
                                                  const float4* table, const float4* weights, S& stream, float2 (&dw)[8]) {
  const int rounds = stream.rounds(W, tokens);
  T* const o = a.o[W] != nullptr ? a.o[W] + t0 * a.ld_x[W] : nullptr;
  Way way(a, W, stream.slot);
#pragma unroll 1
  for (int r = 0; r < rounds; ++r) {
    const bool on = way.t < tokens && unit.i0 >= 0;
    float2 x[8], g[8];
    const uint32_t from = stream.next();
    S::template get<0>(from, x);
    S::template get<1>(from, g);
    const float rs = rsqrtf(__fmaf_rn(lanes_sum(squares_sum(x), s.lanes), a.inv_d, a.eps));
    float2 dot = both(0.0f);
    if (on && GRS_CHECK(way.h < a.heads[W], qk_flags, SITE_QK_HEAD)) {
      unit.template turn<true>(g, table + way.t * 4 * s.turned + u, s.turned);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        x[q] = mul2(x[q], both(rs));
        dw[q] = fma2(g[q], x[q], dw[q]);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 k = weights[(W * 4 + q) * s.units + u];
        g[2 * q] = mul2(g[2 * q], make_float2(k.x, k.y));
        g[2 * q + 1] = mul2(g[2 * q + 1], make_float2(k.z, k.w));
        dot = fma2(g[2 * q], x[2 * q], dot);
        dot = fma2(g[2 * q + 1], x[2 * q + 1], dot);
      }
    }
    const float m = -lanes_sum(dot.x + dot.y, s.lanes) * a.inv_d;
    if (on && o != nullptr) {
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = mul2(fma2(x[q], both(m), g[q]), both(rs));
      store_chunk(o + way.x + unit.i0, x);
      if (unit.i1 >= 0) store_chunk(o + way.x + unit.i1, x + 4);
    }
    way.step(a, s, W);
  }
}

// Eight pairs of a thread in shared memory, [4][threads].
__device__ __forceinline__ void park(float4* at, const float2 (&v)[8]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) at[q * QK_THREADS + threadIdx.x] = make_float4(v[2 * q].x, v[2 * q].y, v[2 * q + 1].x, v[2 * q + 1].y);
}
__device__ __forceinline__ void unpark(const float4* at, float2 (&v)[8]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float4 k = at[q * QK_THREADS + threadIdx.x];
    v[2 * q] = make_float2(k.x, k.y);
    v[2 * q + 1] = make_float2(k.z, k.w);
  }
}

// Blocks stay and take tiles of tokens in turn.  The shares of dwq and dwk are
// in registers while their heads are computed and in shared memory (each
// thread its own) while the others' are.
template <typename T, typename P, bool kPairs>
__global__ void __launch_bounds__(QK_THREADS, QK_BWD_BLOCKS)
    qk_backward_whole_kernel(const __grid_constant__ QkArgs<T, P> a, const __grid_constant__ QkShape s) {
  extern __shared__ float4 shared[];
  const int entries = s.tokens * 4 * s.turned;  // of a table of angles; there are two
  float4 *weights = shared + 2 * entries, *parked = weights + 8 * s.units;
  pdl_wait();
  pdl_trigger();
  const int slot = threadIdx.x / s.lanes, u = threadIdx.x - slot * s.lanes, slots = s.slots;
  const Unit<kPairs> unit(u, s.units, a.d, a.rot);
  Angles<T, P, kPairs, true> angles(a, s);  // the weights' gradients may leave in fp32; 43.2 -> 43.4 us
  const int64_t end = block_token(a.tokens, blockIdx.x + 1);
  int64_t t0 = block_token(a.tokens, blockIdx.x);
  Stream<T, P, 2, qk_bwd_depth<T>> stream(a, s, reinterpret_cast<uint4*>(parked + 8 * QK_THREADS), t0, end, slot, unit.i0, unit.i1);
  float2 dw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = both(0.0f);
  park(parked, dw);
  park(parked + 4 * QK_THREADS, dw);
  qk_weights_to_smem<T, P, kPairs>(a, s, reinterpret_cast<float*>(weights));
  angles.ask(t0, stream.count(t0));
  for (int flip = 0; t0 < end; t0 += s.tokens, flip ^= 1) {
    const int tokens = stream.count(t0);
    float4* table = shared + flip * entries;
    angles.store(t0, tokens, reinterpret_cast<float*>(table));
    angles.ask(t0 + s.tokens, stream.count(t0 + s.tokens));
    __syncthreads();  // (the other table is free: all are done with the tile before)
    if (a.heads[0] > 0) {
      unpark(parked, dw);
      qk_backward_heads<0>(a, s, t0, tokens, unit, u, table, weights, stream, dw);
      park(parked, dw);
    }
    if (a.heads[1] > 0) {
      unpark(parked + 4 * QK_THREADS, dw);
      qk_backward_heads<1>(a, s, t0, tokens, unit, u, table, weights, stream, dw);
      park(parked + 4 * QK_THREADS, dw);
    }
  }
  if (a.parts == nullptr) return;
  // The block's dwq and dwk: the lane groups' sums, in order.
  __syncthreads();
  const float* red = reinterpret_cast<const float*>(parked);
  for (int i = threadIdx.x; i < 2 * 16 * s.units; i += QK_THREADS) {
    const int which = i >= 16 * s.units, n = i - which * 16 * s.units, v = n / 16, j = n % 16;
    const Unit<kPairs> x(v, s.units, a.d, a.rot);
    if (j >= 8 && x.i1 < 0) continue;
    float sum = 0.0f;
    for (int g = 0; g < slots; ++g) sum += red[((which * 4 + j / 4) * QK_THREADS + g * s.lanes + v) * 4 + j % 4];
    a.parts[(int64_t(blockIdx.x) * 2 + which) * a.d + (j < 8 ? x.i0 + j : x.i1 + j - 8)] = sum;
  }
}

// dwq and dwk: 32 elements a block, the blocks' parts in a fixed order.
template <typename G>
__global__ void __launch_bounds__(1024) qk_weights_kernel(const float* __restrict__ parts, int n, int d, G* dwq, G* dwk) {
  __shared__ float red[32][33];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (i < 2 * d)
    for (int k = w; k < n; k += 32) s += parts[int64_t(k) * 2 * d + i];
  red[lane][w] = s;
  __syncthreads();
  s = warp_sum(red[w][lane]);
  const int o = blockIdx.x * 32 + w;
  if (lane != 0 || o >= 2 * d) return;
  G* to = o < d ? dwq : dwk;
  if (to != nullptr) to[o < d ? o : o - d] = from_float<G>(s);
}

// ------------------------------------------------------------------- host
grs_status check_qk(const grs_qk_norm* s, const char* who, int64_t (&ld)[4]) {
  if (s == nullptr) return api_fail(GRS_ERR_INVALID_ARG, who, "shape is NULL");
  if (s->tokens < 0 || s->q_heads < 0 || s->k_heads < 0 || s->head_dim < 1 || s->head_dim > GRS_QK_MAX_DIM)
    return api_fail(GRS_ERR_SHAPE, who, "tokens and heads must be >= 0 and head_dim in [1, GRS_QK_MAX_DIM]");
  const int64_t all = (int64_t(s->q_heads) + s->k_heads) * s->head_dim;
  if (all > GRS_MAX_WIDTH || s->tokens > GRS_MAX_ELEMENTS / (all > 0 ? all : 1))
    return api_fail(GRS_ERR_SHAPE, who, "more than GRS_MAX_WIDTH elements a token, or GRS_MAX_ELEMENTS in all");
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
    if (ld[i] < row || ld[i] > GRS_MAX_ELEMENTS / (s->tokens > 1 ? s->tokens - 1 : 1))
      return api_fail(GRS_ERR_SHAPE, who, "a distance of tokens below their heads' elements, or GRS_MAX_ELEMENTS from the first to the last");
  }
  return GRS_OK;
}

// x modulo 1 in units of 2^-64, rounded to the nearest.
uint64_t fraction64(double x) {
  const double a = std::fabs(x), f = a - std::floor(a), hi = std::floor(f * 0x1p32);  // (all exact; two halves: 2^64 does not fit)
  const uint64_t t = (static_cast<uint64_t>(hi) << 32) + static_cast<uint64_t>(std::floor((f * 0x1p32 - hi) * 0x1p32 + 0.5));
  return x < 0 ? 0 - t : t;
}

// Blocks of the backward pass and so parts of dwq and dwk: what any of its kernels has at most.
int qk_blocks(const grs_qk_norm* s) {
  const int64_t b = (s->tokens * (s->q_heads + s->k_heads) + QK_WARPS - 1) / QK_WARPS;
  return static_cast<int>(b < QK_BLOCKS ? b : QK_BLOCKS);
}

// Whether heads are whole 16-byte chunks whose turned parts are whole chunks too.
bool qk_whole(const grs_qk_norm* s, const int64_t (&ld)[4], const void* a, const void* b, const void* c, const void* d, const void* e,
              const void* f) {
  const int64_t chunk = 16 / dtype_size(s->dtype);
  if (s->head_dim % 8 != 0 || s->rotary_dim % (s->interleaved ? 8 : 16) != 0 || (s->head_dim + 15) / 16 > QK_MAX_UNITS) return false;
  for (int i = 0; i < 4; ++i)
    if (ld[i] % chunk != 0 || ld[i] > QK_MAX_LD) return false;
  return api_aligned(a, 16) && api_aligned(b, 16) && api_aligned(c, 16) && api_aligned(d, 16) && api_aligned(e, 16) && api_aligned(f, 16);
}

QkShape qk_shape(const grs_qk_norm* s, int rounds) {
  QkShape q;
  const int d = s->head_dim, r = s->rotary_dim;
  q.units = s->interleaved ? (d + 15) / 16 : r / 16 + (d - r + 15) / 16;
  q.turned = s->interleaved ? (r > 0 ? q.units : 0) : r / 16;
  q.lanes = 1;
  while (q.lanes < q.units) q.lanes *= 2;
  // Tokens of a block: enough for `rounds` heads a lane group, as far as the table goes and every SM has blocks.
  const int64_t heads = s->q_heads + s->k_heads, slots = QK_THREADS / q.lanes;
  int64_t t = (rounds * slots + heads - 1) / heads;
  if (q.turned > 0 && t > QK_TABLE / (64 * q.turned)) t = QK_TABLE / (64 * q.turned);
  if (t > QK_MAX_TOKENS) t = QK_MAX_TOKENS;
  q.tokens = static_cast<int>(t < 1 ? 1 : t);
  q.slots = static_cast<int>(slots);
  for (int w = 0; w < 2; ++w) {
    const int n = w == 0 ? s->q_heads : s->k_heads;
    q.dt[w] = n > 0 ? q.slots / n : 0;
    q.dh[w] = n > 0 ? q.slots - q.dt[w] * n : 0;
  }
  return q;
}

// Shared memory: tables of angles, weights, backward the parked shares, and the heads under way.
template <typename T, typename P>
int qk_forward_smem(const QkShape& q) {
  return 2 * q.tokens * 64 * q.turned + 2 * 64 * q.units + Stream<T, P, 1, QK_FWD_DEPTH>::BYTES;
}
template <typename T, typename P>
int qk_backward_smem(const QkShape& q) {
  return 2 * q.tokens * 64 * q.turned + 2 * 64 * q.units + 2 * 64 * QK_THREADS + Stream<T, P, 2, qk_bwd_depth<T>>::BYTES;
}

template <typename T, typename P, bool kPairs>
cudaError_t qk_forward_whole(const grs_qk_norm* s, const QkArgs<T, P>& a, void* stream) {
  const QkShape q = qk_shape(s, QK_FWD_ROUNDS);
  const int64_t blocks = s->tokens < QK_FWD_BLOCKS * 152 ? s->tokens : QK_FWD_BLOCKS * 152;
  const QkShape most{QK_MAX_UNITS, 0, 0, 0, 0, {}, {}};
  const cudaError_t e = allow_smem<qk_forward_whole_kernel<T, P, kPairs>>(2 * QK_TABLE + qk_forward_smem<T, P>(most));
  if (e != cudaSuccess) return e;
  return launch_pdl(qk_forward_whole_kernel<T, P, kPairs>, dim3(static_cast<unsigned>(blocks)), dim3(QK_THREADS), qk_forward_smem<T, P>(q),
                    stream, a, q);
}

// *blocks: at most, and then how many it has.
template <typename T, typename P, bool kPairs>
cudaError_t qk_backward_whole(const grs_qk_norm* s, const QkArgs<T, P>& a, int* blocks, void* stream) {
  const QkShape q = qk_shape(s, QK_BWD_ROUNDS);
  if (*blocks > QK_BWD_BLOCKS * 152) *blocks = QK_BWD_BLOCKS * 152;
  if (*blocks > s->tokens) *blocks = static_cast<int>(s->tokens);
  const QkShape most{QK_MAX_UNITS, 0, 0, 0, 0, {}, {}};
  const cudaError_t e = allow_smem<qk_backward_whole_kernel<T, P, kPairs>>(2 * QK_TABLE + qk_backward_smem<T, P>(most));
  if (e != cudaSuccess) return e;
  return launch_pdl(qk_backward_whole_kernel<T, P, kPairs>, dim3(*blocks), dim3(QK_THREADS), qk_backward_smem<T, P>(q), stream, a, q);
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
cudaError_t qk_forward(const grs_qk_norm* s, const int64_t (&ld)[4], const QkArgs<T, P>& a, void* stream) {
  if (qk_whole(s, ld, a.x[0], a.x[1], a.o[0], a.o[1], nullptr, nullptr)) {
    return s->interleaved ? qk_forward_whole<T, P, true>(s, a, stream) : qk_forward_whole<T, P, false>(s, a, stream);
  }
  const int64_t blocks = (s->tokens * (s->q_heads + s->k_heads) + QK_WARPS - 1) / QK_WARPS;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  return launch_pdl(qk_forward_kernel<T, P>, dim3(static_cast<unsigned>(blocks)), dim3(QK_THREADS), 0, stream, a);
}

template <typename T, typename P>
cudaError_t qk_backward(const grs_qk_norm* s, const int64_t (&ld)[4], const QkArgs<T, P>& a, void* dwq, void* dwk, void* stream) {
  int blocks = qk_blocks(s);
  cudaError_t e;
  if (qk_whole(s, ld, a.x[0], a.x[1], a.dy[0], a.dy[1], a.o[0], a.o[1])) {
    e = s->interleaved ? qk_backward_whole<T, P, true>(s, a, &blocks, stream) : qk_backward_whole<T, P, false>(s, a, &blocks, stream);
  } else {
    e = allow_smem<qk_backward_kernel<T, P>>(QK_WARPS * 2 * GRS_QK_MAX_DIM * 4);
    if (e == cudaSuccess)
      e = launch_pdl(qk_backward_kernel<T, P>, dim3(blocks), dim3(QK_THREADS), size_t(QK_WARPS) * 2 * s->head_dim * 4, stream, a);
  }
  if (e != cudaSuccess || a.parts == nullptr) return e;
  const dim3 grid((2 * s->head_dim + 31) / 32), block(1024);
  return s->grad_dtype == GRS_DTYPE_FP32
             ? launch_pdl(qk_weights_kernel<float>, grid, block, 0, stream, static_cast<const float*>(a.parts), blocks, s->head_dim,
                          static_cast<float*>(dwq), static_cast<float*>(dwk))
             : launch_pdl(qk_weights_kernel<uint16_t>, grid, block, 0, stream, static_cast<const float*>(a.parts), blocks, s->head_dim,
                          static_cast<uint16_t*>(dwq), static_cast<uint16_t*>(dwk));
}

}  // namespace

cudaError_t qk_norm_flags(int** at) { return cudaGetSymbolAddress(reinterpret_cast<void**>(at), qk_flags); }

}  // namespace grs

using namespace grs;

extern "C" {

grs_status grs_rope_turns(const double* inv_freq, int32_t n, uint64_t* turns) {
  static const char who[] = "grs_rope_turns";
  if (n < 0 || (n > 0 && (inv_freq == nullptr || turns == nullptr))) return api_fail(GRS_ERR_INVALID_ARG, who, "NULL argument or n < 0");
  for (int32_t i = 0; i < n; ++i) {
    if (!std::isfinite(inv_freq[i])) return api_fail(GRS_ERR_INVALID_ARG, who, "a frequency that is not finite");
    // 1 / (2 pi) in two doubles, so that the product in two doubles is good to 2^-107 of the frequency.
    const double f = inv_freq[i], inv_hi = 0.15915494309189535, inv_lo = -9.839338337591243e-18;
    const double p = f * inv_hi, rest = std::fma(f, inv_lo, std::fma(f, inv_hi, -p));
    turns[i] = fraction64(p) + fraction64(rest);
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
#define GRS_QK_CALL(T, P) qk_forward<T, P>(s, ld, qk_args<T, P>(s, ld, nullptr, nullptr, q, k, wq, wk, positions, turns, qo, ko, nullptr), stream)
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
  qk_backward<T, P>(s, ld, qk_args<T, P>(s, ld, dqo, dko, q, k, wq, wk, positions, turns, dq, dk, parts), dwq, dwk, stream)
  e = f ? (pf ? GRS_QK_CALL(float, float) : GRS_QK_CALL(float, uint16_t))
        : (pf ? GRS_QK_CALL(uint16_t, float) : GRS_QK_CALL(uint16_t, uint16_t));
#undef GRS_QK_CALL
  return e == cudaSuccess ? GRS_OK : api_cuda_fail(e, who);
}

}  // extern "C"
