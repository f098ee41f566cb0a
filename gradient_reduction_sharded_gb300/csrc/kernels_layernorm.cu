// Layer norm over rows, forward and backward.
//
//   mean = sum x / C,  var = sum (x - mean)^2 / C,  r = 1 / sqrt(var + eps)
//   h = (x - mean) r,  y = h w + b
//   dh = dy w,  dx = r (dh - mean_C(dh) - h mean_C(dh h))
//   dw = sum over rows of dy h,  db = sum over rows of dy
//
// All arithmetic and every sum in fp32; one rounding to the output's type.
// The variance is the mean square of the differences from the mean, from
// registers: no cancellation, at the price of a second sum over the row.
//
// Both passes are bound by memory, x (and dy) read once.  What it takes to
// get there on a GB300 (copy rate 6.78 TB/s):
//   * rows in registers, 16 or 32 elements a thread, so that a row's sums
//     meet across few warps;
//   * blocks that stay (152 SMs x 1 or 2), the parameters and the parameters'
//     gradients in registers, and the rows to come in flight in shared memory:
//     without them each row waits for its loads (bf16 32768 x 2048: 43.2 us,
//     6.2 TB/s, against 59 us);
//   * fp32 pairs, half the instructions (packed.cuh).
// Backward, 8192 x 2048 bf16: 25 us (4.0 TB/s; 65536 rows 6.1), of which about
// 5 are launch and first loads and 5 the parameters' gradients (parts of 152
// blocks, summed by a second kernel); 65536 x 128 in rows 384 apart: 15 us.
// One row of 2048: 2.2 us forward, 5.3 us backward, launch latency.
// Loose rows cost two to four times as much (8192 x 1027 bf16: 30 and 37 us):
// more instructions an element, and threads of whole warps without one.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "api_util.h"
#include "device.cuh"
#include "internal.h"
#include "launch.cuh"
#include "packed.cuh"

namespace grs {
namespace {

constexpr int LN_THREADS = 256;
constexpr int LN_RING_THREADS = 512; // a block of the forward ring at most
constexpr int LN_RING_GROUPS = 256;  // and its rows at a time (a loose row takes 32 bytes more)
constexpr int LN_BWD_THREADS = 512;  // a block of the backward pass at most
constexpr int LN_RED_BYTES = 256;    // two float2 a warp of a block, twice
constexpr int LN_PEERS = 8;          // blocks of a cluster at most (the portable size)
constexpr int LN_WIDE_RED = LN_PEERS * LN_RED_BYTES + 16;  // the warps' sums of a cluster, twice, and their barriers
// Slots of its ring: the row that is finished, the one that is summed, and
// those in flight.  Few, so that more blocks fit an SM where their registers
// allow it: fp32 (62 registers) 7812 x 8192 126 us with 3, 150 with 4, 152 with
// 6; bf16 (122) 7812 x 16384 159, 150 and 151.
template <typename T>
constexpr int ln_wide_slots = sizeof(T) == 4 ? 3 : 4;
constexpr uint64_t LN_LINGER_NS = 50000;
constexpr int LN_PARTS = 304;        // partial rows of dw and db at most: two blocks an SM

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

// --------------------------------------------- rows held in registers
// A group of `tpr` threads (a power of two up to a warp, or whole warps) has
// a row: thread t holds the chunks t, t + tpr, ... of VEC elements, E
// elements in all, read once.  VEC is 16 bytes where every row starts at a
// multiple of 16 bytes and has whole chunks, else a pair of elements, of
// which the row's last may be half (a "loose" row).
template <typename T, int VEC, int E>
struct Row {
  static constexpr int NV = E / VEC;
  static constexpr int WORDS = VEC * static_cast<int>(sizeof(T)) / 4;  // 32-bit words of a chunk
  uint32_t r[NV * WORDS];

  // Elements 2 i and 2 i + 1 of the thread's E.
  __device__ __forceinline__ float2 pair(int i) const {
    if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
    return bf16_pair(r[i]);
  }
  // Straight from memory; zeros beyond the row.
  __device__ __forceinline__ void load(const T* p, int t, int tpr, int cols, bool on) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (t + j * tpr) * VEC;
      if constexpr (VEC == 2) {
        const float lo = on && c < cols ? ln_load(p + c) : 0.0f, hi = on && c + 1 < cols ? ln_load(p + c + 1) : 0.0f;
        if constexpr (sizeof(T) == 4) {
          r[2 * j] = __float_as_uint(lo);
          r[2 * j + 1] = __float_as_uint(hi);
        } else {
          r[j] = __float_as_uint(lo) >> 16 | __float_as_uint(hi);
        }
      } else {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (on && c < cols) v = *reinterpret_cast<const uint4*>(p + c);
        r[4 * j] = v.x;
        r[4 * j + 1] = v.y;
        r[4 * j + 2] = v.z;
        r[4 * j + 3] = v.w;
      }
    }
  }
};

// The rows to come, in flight in shared memory (cp.async, 16 bytes each), so
// that the bytes in flight do not cost registers.  A slot is refilled one row
// after it was read.  `slot` is the slot's first byte.
//
// Whole rows: a thread copies the chunks that it will read itself, so nobody
// waits for anybody; a thread's chunks lie blockDim.x chunks apart.
// Loose rows: the group copies the aligned 16-byte pieces that cover the row,
// which keeps its place modulo 16 bytes, and waits for one another before
// reading pairs.  A piece that reaches outside the matrix is copied by its
// elements.
struct Matrix {
  const uint8_t *first, *last;  // the first byte and the one after the last
};

template <typename T, int VEC, int E>
struct Ring {
  static constexpr int NV = E / VEC;
  static constexpr int BYTES = E * static_cast<int>(sizeof(T));  // a thread and row
  static constexpr int EXTRA = VEC == 2 ? 32 : 0;                // a group's row may start and end inside a piece

  static __device__ __forceinline__ void copy16(void* dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(bytes) : "memory");
  }

  static __device__ __forceinline__ void issue(uint8_t* slot, const T* p, const Matrix& m, int g, int t, int tpr, int cols,
                                               bool on) {
    if constexpr (VEC > 2) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (t + j * tpr) * VEC;
        const bool in = on && c < cols;
        copy16(slot + (j * blockDim.x + threadIdx.x) * 16, in ? p + c : p, in ? 16 : 0);
      }
    } else if (on) {
      uint8_t* row = slot + g * (tpr * BYTES + EXTRA);
      const uint8_t* end = reinterpret_cast<const uint8_t*>(p + cols);
      const uint8_t* src = reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15)) + t * 16;
      for (int at = t * 16; src < end; at += tpr * 16, src += tpr * 16) {
        if (src >= m.first && src + 16 <= m.last) {
          copy16(row + at, src, 16);
        } else {
          for (int k = 0; k < 16; k += sizeof(T))
            if (src + k >= reinterpret_cast<const uint8_t*>(p) && src + k < end)
              *reinterpret_cast<T*>(row + at + k) = *reinterpret_cast<const T*>(src + k);
        }
      }
    }
  }

  // p: the row that was copied to the slot.
  static __device__ __forceinline__ void read(const uint8_t* slot, const T* p, int g, int t, int tpr, int cols, bool on,
                                              Row<T, VEC, E>& x) {
    if constexpr (VEC > 2) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const uint4 v = *reinterpret_cast<const uint4*>(slot + (j * blockDim.x + threadIdx.x) * 16);
        x.r[4 * j] = v.x;
        x.r[4 * j + 1] = v.y;
        x.r[4 * j + 2] = v.z;
        x.r[4 * j + 3] = v.w;
      }
    } else {
      const uint8_t* row = slot + g * (tpr * BYTES + EXTRA) + (reinterpret_cast<uintptr_t>(p) & 15);
      const bool odd = sizeof(T) == 2 && (reinterpret_cast<uintptr_t>(p) & 2) != 0;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = 2 * (t + j * tpr);
        const bool lo = on && c < cols, hi = on && c + 1 < cols;
        if constexpr (sizeof(T) == 4) {
          const float* f = reinterpret_cast<const float*>(row) + c;
          x.r[2 * j] = lo ? __float_as_uint(f[0]) : 0u;
          x.r[2 * j + 1] = hi ? __float_as_uint(f[1]) : 0u;
        } else {
          // the pair is one word, or the high half of one and the low half of the next
          const uint32_t* w = reinterpret_cast<const uint32_t*>(row + 2 * c - (odd ? 2 : 0));
          uint32_t v = lo ? w[0] : 0u;
          if (odd) v = __funnelshift_r(v, lo ? w[1] : 0u, 16);
          x.r[j] = hi ? v : lo ? v & 0xffffu : 0u;
        }
      }
    }
  }
};

__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void ring_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Slots of a ring whose rows take `bytes` a thread: two blocks of 256 threads an SM.
__host__ __device__ constexpr int ring_slots(int bytes) { return bytes <= 16 ? 8 : bytes <= 32 ? 6 : bytes <= 64 ? 5 : 3; }

// The thread's E elements to a row, rounded to T.
template <typename T, int VEC, int E>
__device__ __forceinline__ void store_row(T* p, int t, int tpr, int cols, const float2 (&o)[E / 2]) {
  if constexpr (VEC == 2) {
    const bool whole = (reinterpret_cast<uintptr_t>(p) & (2 * sizeof(T) - 1)) == 0;
#pragma unroll
    for (int j = 0; j < E / 2; ++j) {
      const int c = 2 * (t + j * tpr);
      if (whole && c + 1 < cols) {
        if constexpr (sizeof(T) == 4)
          *reinterpret_cast<float2*>(p + c) = o[j];
        else
          *reinterpret_cast<uint32_t*>(p + c) = to_bf16_pair(o[j]);
      } else {
        if (c < cols) ln_store(p + c, o[j].x);
        if (c + 1 < cols) ln_store(p + c + 1, o[j].y);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < E / VEC; ++j) {
      const int c = (t + j * tpr) * VEC;
      if (c >= cols) continue;
      if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float4*>(p + c) = make_float4(o[2 * j].x, o[2 * j].y, o[2 * j + 1].x, o[2 * j + 1].y);
      else
        *reinterpret_cast<uint4*>(p + c) = make_uint4(to_bf16_pair(o[4 * j]), to_bf16_pair(o[4 * j + 1]),
                                                      to_bf16_pair(o[4 * j + 2]), to_bf16_pair(o[4 * j + 3]));
    }
  }
}

// A thread's place: its group of tpr threads in the block, and where the
// group's warps leave their sums ([2 phases][warps] float2 in shared memory).
struct Place {
  int tpr, t, g, warps, bar;
  float2 *red, *mine;
};

__device__ __forceinline__ Place ln_place(int tpr, float2* red) {
  Place p;
  p.tpr = tpr;
  p.g = threadIdx.x / tpr;
  p.t = threadIdx.x - p.g * tpr;
  p.warps = tpr >> 5;
  p.bar = 1 + p.g;  // barrier 0 is the block's
  p.red = red + p.g * 2 * p.warps;
  p.mine = p.red + (p.t >> 5);
  return p;
}

// Sums over the group, the same bits for each of its threads.  Successive
// calls alternate `phase`, so one barrier a call is enough: who writes a
// phase again has passed the barrier of the other, after all of its reads.
__device__ __forceinline__ void group_sum2(float& a, float& b, const Place& p, int phase) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float x = __shfl_xor_sync(0xffffffffu, a, o), y = __shfl_xor_sync(0xffffffffu, b, o);
    if (o < p.tpr) {
      a = __fadd_rn(a, x);
      b = __fadd_rn(b, y);
    }
  }
  if (p.tpr <= 32) return;
  const int at = phase ? p.warps : 0;
  if ((threadIdx.x & 31) == 0) p.mine[at] = make_float2(a, b);
  asm volatile("bar.sync %0, %1;" ::"r"(p.bar), "r"(p.tpr) : "memory");
  a = b = 0.0f;
#pragma unroll 4
  for (int k = 0; k < p.warps; ++k) {
    const float2 v = p.red[at + k];
    a = __fadd_rn(a, v.x);
    b = __fadd_rn(b, v.y);
  }
}

__device__ __forceinline__ float group_sum(float a, const Place& p, int phase) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float x = __shfl_xor_sync(0xffffffffu, a, o);
    if (o < p.tpr) a = __fadd_rn(a, x);
  }
  if (p.tpr <= 32) return a;
  const int at = phase ? p.warps : 0;
  if ((threadIdx.x & 31) == 0) p.mine[at].x = a;
  asm volatile("bar.sync %0, %1;" ::"r"(p.bar), "r"(p.tpr) : "memory");
  a = 0.0f;
#pragma unroll 4
  for (int k = 0; k < p.warps; ++k) a = __fadd_rn(a, p.red[at + k].x);
  return a;
}

// The same over the blocks of a cluster (each with one group): every warp
// sends its sums to each block's shared memory, whose barrier of the phase
// counts their bytes, and every thread adds up the same numbers in the same
// order.  Who sends to a phase again has taken the sums of the other, so every
// warp has sent those, after it took what this phase held.  Hence a warp that
// gave up a wait sends nothing more: its peers find the next row's sums
// incomplete and give up in turn, where another row's would complete them.
__device__ __forceinline__ unsigned cluster_size() {
  unsigned n;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_meet() {
  __syncwarp();
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\t"
      "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_sum2_send(float a, float b, const Place& p, uint64_t* bar, unsigned peer, unsigned peers,
                                                  int phase) {
  const unsigned lane = threadIdx.x & 31;
  if (threadIdx.x == 0) mbar_arrive_expect_tx(bar + phase, peers * p.warps * 8);
  if (lane < peers) {  // lane k to block k
    uint32_t to, to_bar;
    const float2* at = p.red + (phase * LN_PEERS + peer) * p.warps + (p.t >> 5);
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_addr(at)), "r"(lane));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to_bar) : "r"(smem_addr(bar + phase)), "r"(lane));
    const uint64_t v = uint64_t(__float_as_uint(b)) << 32 | __float_as_uint(a);
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(to), "l"(v), "r"(to_bar)
                 : "memory");
  }
}

// False, for the whole warp, if the sums did not come in time.
__device__ __forceinline__ bool cluster_sum2_take(float& a, float& b, const Place& p, uint64_t* bar, unsigned peers, int phase,
                                                  uint32_t parity, uint64_t limit_ns) {
  bool in = mbar_try_wait(bar + phase, parity);
  if (!in) {
    const uint64_t t0 = global_ns();
    while (!in && global_ns() - t0 <= limit_ns) in = mbar_try_wait(bar + phase, parity);
  }
  if (!__all_sync(0xffffffffu, in)) return false;
  a = b = 0.0f;
  const float2* red = p.red + phase * LN_PEERS * p.warps;
  for (unsigned k = threadIdx.x & 31; k < peers * p.warps; k += 32) {
    const float2 v = red[k];
    a = __fadd_rn(a, v.x);
    b = __fadd_rn(b, v.y);
  }
  a = warp_sum(a);
  b = warp_sum(b);
  return true;
}

// The thread's E parameters of p, `none` without any and beyond the row.
template <typename W, int VEC, int E>
__device__ __forceinline__ void row_params(const W* p, float none, int t, int tpr, int cols, float2 (&o)[E / 2]) {
#pragma unroll
  for (int i = 0; i < E / 2; ++i) o[i] = both(none);
  if (p == nullptr) return;
#pragma unroll
  for (int j = 0; j < E / VEC; ++j) {
    const int c = (t + j * tpr) * VEC;
    if (c >= cols) continue;
    float2* v = o + j * VEC / 2;
    if constexpr (VEC == 2) {
      v[0].x = ln_load(p + c);
      if (c + 1 < cols) v[0].y = ln_load(p + c + 1);
    } else if constexpr (sizeof(W) == 4) {
#pragma unroll
      for (int i = 0; i < VEC / 4; ++i) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(p + c) + i);
        v[2 * i] = make_float2(f.x, f.y);
        v[2 * i + 1] = make_float2(f.z, f.w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC / 4; ++i) {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(p + c) + i);
        v[2 * i] = bf16_pair(u.x);
        v[2 * i + 1] = bf16_pair(u.y);
      }
    }
  }
}

template <typename T, typename W>
struct LnFwd {
  const T* x;
  const W *w, *b;
  T* y;
  float *mean, *rstd;
  int64_t ld_x, ld_y, rows;
  int32_t cols, tpr;
  float eps;
};

// The row in d (this thread's E elements, zeros beyond the row) to y.
template <typename T, typename W, int VEC, int E>
__device__ __forceinline__ void ln_fwd_row(const LnFwd<T, W>& a, float2 (&d)[E / 2], const float2 (&w)[E / 2],
                                           const float2 (&b)[E / 2], int64_t row, T* y, const Place& p, float inv_c) {
  float2 s = both(0.0f);
#pragma unroll
  for (int i = 0; i < E / 2; ++i) s = add2(s, d[i]);
  const float mean = group_sum(s.x + s.y, p, 0) * inv_c;
  s = both(0.0f);
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    d[i] = add2(d[i], both(-mean));
    const int c = (p.t + (2 * i / VEC) * p.tpr) * VEC;
    if constexpr (VEC == 2) {
      if (c < a.cols) s.x = fmaf(d[i].x, d[i].x, s.x);
      if (c + 1 < a.cols) s.y = fmaf(d[i].y, d[i].y, s.y);
    } else if (c < a.cols) {
      s = fma2(d[i], d[i], s);
    }
  }
  const float rstd = 1.0f / sqrtf(group_sum(s.x + s.y, p, 1) * inv_c + a.eps);
  if (row >= a.rows) return;
#pragma unroll
  for (int i = 0; i < E / 2; ++i) d[i] = fma2(mul2(d[i], both(rstd)), w[i], b[i]);
  store_row<T, VEC, E>(y, p.t, p.tpr, a.cols, d);
  if (p.t == 0) {
    if (a.mean != nullptr) a.mean[row] = mean;
    if (a.rstd != nullptr) a.rstd[row] = rstd;
  }
}

// Few rows: a group a row, as many threads as its loads can use.
template <typename T, typename W, int VEC, int E>
__global__ void __launch_bounds__(1024) ln_fwd_kernel(const __grid_constant__ LnFwd<T, W> a) {
  __shared__ float2 red[2 * 32];
  pdl_wait();
  pdl_trigger();
  const Place p = ln_place(a.tpr, red);
  const int64_t row = int64_t(blockIdx.x) * (blockDim.x / a.tpr) + p.g;
  const bool on = row < a.rows;
  float2 d[E / 2], w[E / 2], b[E / 2];
  Row<T, VEC, E> x;
  x.load(a.x + (on ? row : 0) * a.ld_x, p.t, p.tpr, a.cols, on);
  row_params<W, VEC, E>(a.w, 1.0f, p.t, p.tpr, a.cols, w);
  row_params<W, VEC, E>(a.b, 0.0f, p.t, p.tpr, a.cols, b);
#pragma unroll
  for (int i = 0; i < E / 2; ++i) d[i] = x.pair(i);
  ln_fwd_row<T, W, VEC, E>(a, d, w, b, row, a.y + row * a.ld_y, p, 1.0f / static_cast<float>(a.cols));
}

// The group's threads have each other's copies (loose rows only).
template <int VEC>
__device__ __forceinline__ void group_meet(const Place& p) {
  if constexpr (VEC == 2) {
    if (p.tpr <= 32)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(p.bar), "r"(p.tpr) : "memory");
  }
}

template <typename T>
__device__ __forceinline__ Matrix matrix_of(const T* p, int64_t ld, int64_t rows, int32_t cols) {
  return {reinterpret_cast<const uint8_t*>(p), reinterpret_cast<const uint8_t*>(p + (rows - 1) * ld + cols)};
}

// Many rows: blocks that stay, each group walking the rows with the stride
// of the whole grid, the parameters in registers and the rows to come in
// flight in shared memory.
template <typename T, typename W, int VEC, int E>
__global__ void __launch_bounds__(LN_RING_THREADS) ln_fwd_ring_kernel(const __grid_constant__ LnFwd<T, W> a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float2 red[2 * (LN_RING_THREADS / 32)];
  pdl_wait();
  pdl_trigger();
  using R = Ring<T, VEC, E>;
  constexpr int SLOTS = ring_slots(R::BYTES);
  const Place p = ln_place(a.tpr, red);
  const int groups = blockDim.x / a.tpr, slot_bytes = R::BYTES * blockDim.x + R::EXTRA * groups;
  const Matrix m = matrix_of(a.x, a.ld_x, a.rows, a.cols);
  const int64_t step = int64_t(gridDim.x) * groups, x_step = step * a.ld_x, y_step = step * a.ld_y;
  int64_t row = int64_t(blockIdx.x) * groups + p.g, ahead = row;
  const T *x_ahead = a.x + ahead * a.ld_x, *x_now = x_ahead;
  T* y = a.y + row * a.ld_y;
  const auto issue = [&](int slot) {  // the next row to come
    const bool on = ahead < a.rows;
    R::issue(ring + slot * slot_bytes, on ? x_ahead : a.x, m, p.g, p.t, p.tpr, a.cols, on);
    ring_commit();
    ahead += step;
    x_ahead += x_step;
  };
#pragma unroll 1
  for (int s = 0; s < SLOTS - 1; ++s) issue(s);
  float2 w[E / 2], b[E / 2];
  row_params<W, VEC, E>(a.w, 1.0f, p.t, p.tpr, a.cols, w);
  row_params<W, VEC, E>(a.b, 0.0f, p.t, p.tpr, a.cols, b);
  const float inv_c = 1.0f / static_cast<float>(a.cols);
  int slot = 0;
  for (int64_t base = row - p.g; base < a.rows; base += step, row += step, y += y_step, x_now += x_step) {
    ring_wait<SLOTS - 2>();
    group_meet<VEC>(p);
    float2 d[E / 2];
    {
      Row<T, VEC, E> x;
      R::read(ring + slot * slot_bytes, x_now, p.g, p.t, p.tpr, a.cols, row < a.rows, x);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) d[i] = x.pair(i);
    }
    issue(slot == 0 ? SLOTS - 1 : slot - 1);
    slot = slot == SLOTS - 1 ? 0 : slot + 1;
    ln_fwd_row<T, W, VEC, E>(a, d, w, b, row, y, p, inv_c);
  }
  ring_wait<0>();  // no copy outlives the slots
}

// Set by a warp that gave up a wait; the calls have no handle to keep it in.
__device__ int ln_gave_up;

// How long a block of a cluster waits for the others' sums.  The self-test
// has block `quitter` of every cluster give up at its `quit_row`th row.
struct LnWait {
  uint64_t limit_ns = WAIT_LIMIT_NS;
  int32_t quitter = -1, quit_row = 0;
};

template <typename T, typename W>
struct LnBwd {
  const T *dy, *x;
  const W* w;
  const float *mean, *rstd;
  T* dx;         // may be null
  float* parts;  // [gridDim.x][2][cols], or null
  int64_t ld_dy, ld_x, ld_dx, rows;
  int32_t cols, tpr, span;  // span: columns of a block, where a cluster shares the rows
  LnWait wait;
};

// A block's groups walk the rows with the stride of the whole grid; each
// thread keeps its columns' dw and db in registers over all its rows, and the
// block adds its groups' sums in shared memory into one part.  The next row
// is in flight while a row is worked on.
// Without kParams the sums over the rows are left out.
template <typename T, typename W, int VEC, int E, bool kParams>
__global__ void __launch_bounds__(LN_BWD_THREADS) ln_bwd_kernel(const __grid_constant__ LnBwd<T, W> a) {
  extern __shared__ __align__(16) float sums[];  // the groups' warp sums and the ring; the parts' sums after it
  pdl_wait();
  pdl_trigger();
  const Place p = ln_place(a.tpr, reinterpret_cast<float2*>(sums));
  const int tpr = a.tpr, t = p.t, g = p.g, groups = blockDim.x / tpr;
  const float inv_c = 1.0f / static_cast<float>(a.cols);
  const int64_t step = int64_t(gridDim.x) * groups;
  int64_t row = int64_t(blockIdx.x) * groups + g, ahead = row;
  const int64_t x_step = step * a.ld_x, dy_step = step * a.ld_dy, dx_step = step * a.ld_dx;
  const T *x_ahead = a.x + row * a.ld_x, *dy_ahead = a.dy + row * a.ld_dy, *x_now = x_ahead, *dy_now = dy_ahead;
  T* dx = a.dx != nullptr ? a.dx + row * a.ld_dx : nullptr;
  const Matrix mx = matrix_of(a.x, a.ld_x, a.rows, a.cols), my = matrix_of(a.dy, a.ld_dy, a.rows, a.cols);
  Row<T, VEC, E> x, dy;
  // Statistics two rows ahead (their loads are as far away as the rows').
  float mean, rstd, mean_1, rstd_1, mean_2, rstd_2;
  const auto stats = [&](int64_t r, float& m, float& s) {
    m = r < a.rows ? __ldg(a.mean + r) : 0.0f;
    s = r < a.rows ? __ldg(a.rstd + r) : 0.0f;
  };
  using R = Ring<T, VEC, E>;
  constexpr int SLOTS = ring_slots(2 * R::BYTES);
  uint8_t* ring = reinterpret_cast<uint8_t*>(sums) + LN_RED_BYTES;
  const int half_slot = R::BYTES * blockDim.x + R::EXTRA * groups;
  const auto fetch = [&](int slot) {  // the next rows to come
    const bool on = ahead < a.rows;
    uint8_t* at = ring + slot * (2 * half_slot);
    R::issue(at, on ? x_ahead : a.x, mx, g, t, tpr, a.cols, on);
    R::issue(at + half_slot, on ? dy_ahead : a.dy, my, g, t, tpr, a.cols, on);
    ring_commit();
    ahead += step;
    x_ahead += x_step;
    dy_ahead += dy_step;
  };
  int slot = 0, phase = 0;
  if (a.rows > 0) {
#pragma unroll 1
    for (int s = 0; s < SLOTS - 1; ++s) fetch(s);
  }
  stats(row, mean, rstd);
  stats(row + step, mean_1, rstd_1);
  float2 w[E / 2], dw[E / 2], db[E / 2];
  row_params<W, VEC, E>(a.w, 1.0f, t, tpr, a.cols, w);
#pragma unroll
  for (int i = 0; i < E / 2; ++i) dw[i] = db[i] = both(0.0f);
  for (int64_t base = row - g; base < a.rows; base += step) {
    stats(row + 2 * step, mean_2, rstd_2);
    ring_wait<SLOTS - 2>();
    group_meet<VEC>(p);
    const uint8_t* at = ring + slot * (2 * half_slot);
    R::read(at, x_now, g, t, tpr, a.cols, row < a.rows, x);
    R::read(at + half_slot, dy_now, g, t, tpr, a.cols, row < a.rows, dy);
    fetch(slot == 0 ? SLOTS - 1 : slot - 1);
    slot = slot == SLOTS - 1 ? 0 : slot + 1;
    x_now += x_step;
    dy_now += dy_step;
    float2 h[E / 2], dh[E / 2], s1 = both(0.0f), s2 = both(0.0f);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const float2 d = dy.pair(i);
      h[i] = mul2(add2(x.pair(i), both(-mean)), both(rstd));
      dh[i] = mul2(d, w[i]);
      s1 = add2(s1, dh[i]);
      s2 = fma2(dh[i], h[i], s2);
      if constexpr (kParams) {
        dw[i] = fma2(d, h[i], dw[i]);
        db[i] = add2(db[i], d);
      }
    }
    if (dx != nullptr) {
      float c1 = s1.x + s1.y, c2 = s2.x + s2.y;
      group_sum2(c1, c2, p, phase);
      phase ^= 1;
      // dx = r dh - r c1 - h r c2
      c1 *= -inv_c * rstd;
      c2 *= -inv_c * rstd;
#pragma unroll
      for (int i = 0; i < E / 2; ++i) dh[i] = fma2(h[i], both(c2), fma2(dh[i], both(rstd), both(c1)));
      if (row < a.rows) store_row<T, VEC, E>(dx, t, tpr, a.cols, dh);
      dx += dx_step;
    }
    row += step;
    mean = mean_1;
    rstd = rstd_1;
    mean_1 = mean_2;
    rstd_1 = rstd_2;
  }
  ring_wait<0>();  // no copy outlives the slots
  if constexpr (!kParams) return;
  // The groups' sums meet in the ring's place: [dw or db][group][tpr * E].
  const int wide = tpr * E, half = groups * wide;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float* mine = sums + k * half + g * wide;
#pragma unroll
    for (int i = 0; i < E / 2; i += VEC == 2 ? 1 : 2) {
      const float2* v = (k == 0 ? dw : db) + i;
      float* at = mine + (2 * i / VEC * tpr + t) * VEC + 2 * i % VEC;
      if constexpr (VEC == 2)
        *reinterpret_cast<float2*>(at) = v[0];
      else
        *reinterpret_cast<float4*>(at) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    }
  }
  __syncthreads();
  float* part = a.parts + int64_t(blockIdx.x) * 2 * a.cols;
  for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
    float s = sums[c], u = sums[half + c];
    for (int k = 1; k < groups; ++k) {
      s += sums[c + k * wide];
      u += sums[half + c + k * wide];
    }
    part[c] = s;
    part[a.cols + c] = u;
  }
}

// Whole rows wider than a block's registers: a cluster shares them, each of its
// blocks `span` columns.  A row's two sums need the whole cluster, 1 us from
// one block to the next, so they travel while the block does other work:
//   sums of row i (and its dw, db)  ->  take the cluster's sums of row i - 1,
//   send row i's  ->  dx of row i - 1, its elements read from the ring again.
// (With a barrier of the cluster in place of the counted sends, its release
// waits for dx: 2.3 us a row instead of 1.3.)  256 MB in rows of 16384: bf16
// 150 us (5.1 TB/s), fp32 131 to 151; with a pass for dx and another over x and dy
// for dw and db 280 and 308.  The ring is read by who filled it, so a slot
// may be filled again two rows on without a barrier.
template <typename T, typename W, int E>
__global__ void __launch_bounds__(LN_BWD_THREADS) ln_bwd_wide_kernel(const __grid_constant__ LnBwd<T, W> a) {
  extern __shared__ __align__(16) float sums[];  // the cluster's warp sums, and the ring
  constexpr int VEC = 16 / sizeof(T);
  pdl_wait();
  pdl_trigger();
  const Place p = ln_place(a.tpr, reinterpret_cast<float2*>(sums));
  const int tpr = a.tpr, t = p.t;
  const unsigned peers = cluster_size(), peer = cluster_rank();
  const int first = peer * a.span, cols = min(a.span, a.cols - first);
  const int64_t block = blockIdx.x / peers, step = gridDim.x / peers;
  const float inv_c = 1.0f / static_cast<float>(a.cols);
  const int64_t x_step = step * a.ld_x, dy_step = step * a.ld_dy, dx_step = step * a.ld_dx;
  uint64_t* bar = reinterpret_cast<uint64_t*>(sums) + LN_PEERS * LN_RED_BYTES / 8;
  if (threadIdx.x == 0) {
    mbar_init(bar, 1);
    mbar_init(bar + 1, 1);
    fence_mbar_init();
  }
  const T *x_ahead = a.x + block * a.ld_x + first, *dy_ahead = a.dy + block * a.ld_dy + first;
  const T *x_now = x_ahead, *dy_now = dy_ahead;
  const Matrix mx = matrix_of(a.x, a.ld_x, a.rows, a.cols), my = matrix_of(a.dy, a.ld_dy, a.rows, a.cols);
  using R = Ring<T, VEC, E>;
  constexpr int SLOTS = ln_wide_slots<T>;
  uint8_t* ring = reinterpret_cast<uint8_t*>(sums) + LN_WIDE_RED;
  const int half_slot = R::BYTES * tpr;
  int64_t ahead = block;
  const auto fetch = [&](int slot) {  // the next row to come
    const bool on = ahead < a.rows;
    uint8_t* at = ring + slot * (2 * half_slot);
    R::issue(at, on ? x_ahead : a.x, mx, 0, t, tpr, cols, on);
    R::issue(at + half_slot, on ? dy_ahead : a.dy, my, 0, t, tpr, cols, on);
    ring_commit();
    ahead += step;
    x_ahead += x_step;
    dy_ahead += dy_step;
  };
  const auto stats = [&](int64_t r, float& m, float& s) {
    m = r < a.rows ? __ldg(a.mean + r) : 0.0f;
    s = r < a.rows ? __ldg(a.rstd + r) : 0.0f;
  };
#pragma unroll 1
  for (int s = 0; s < SLOTS - 2; ++s) fetch(s);
  float mean_last = 0.0f, rstd_last = 0.0f, mean, rstd, mean_1, rstd_1;
  stats(block, mean, rstd);
  stats(block + step, mean_1, rstd_1);
  float2 w[E / 2], dw[E / 2], db[E / 2];
  row_params<W, VEC, E>(a.w != nullptr ? a.w + first : nullptr, 1.0f, t, tpr, cols, w);
#pragma unroll
  for (int i = 0; i < E / 2; ++i) dw[i] = db[i] = both(0.0f);
  T* dx = a.dx != nullptr ? a.dx + block * a.ld_dx + first : nullptr;
  int slot = 0;
  // dx of the last row: its sums are in, its elements still in the slot before.
  const auto finish = [&](float c1, float c2) {
    const uint8_t* at = ring + (slot == 0 ? SLOTS - 1 : slot - 1) * (2 * half_slot);
    Row<T, VEC, E> x, dy;
    R::read(at, x_now - x_step, 0, t, tpr, cols, true, x);
    R::read(at + half_slot, dy_now - dy_step, 0, t, tpr, cols, true, dy);
    c1 *= -inv_c * rstd_last;
    c2 *= -inv_c * rstd_last;
    float2 o[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const float2 h = mul2(add2(x.pair(i), both(-mean_last)), both(rstd_last));
      o[i] = fma2(h, both(c2), fma2(mul2(dy.pair(i), w[i]), both(rstd_last), both(c1)));
    }
    store_row<T, VEC, E>(dx, t, tpr, cols, o);
    dx += dx_step;
  };
  cluster_meet();  // every peer has started: its shared memory may be written
  bool lost = false;  // the warp gave up a wait (never, unless a peer is gone): no number stands for sums from there on
  const auto take = [&](float& c1, float& c2, int row_no) {
    if (!lost)
      lost = (static_cast<int>(peer) == a.wait.quitter && row_no == a.wait.quit_row) ||
             !cluster_sum2_take(c1, c2, p, bar, peers, row_no & 1, (row_no >> 1) & 1, a.wait.limit_ns);
    if (lost) c1 = c2 = __int_as_float(0x7fc00000);
  };
  int n = 0;  // this cluster's rows so far
  for (int64_t row = block; row < a.rows; row += step) {
    ring_wait<SLOTS - 3>();
    fetch(slot < 2 ? slot + SLOTS - 2 : slot - 2);
    float mean_2, rstd_2;
    stats(row + 2 * step, mean_2, rstd_2);
    float2 s1 = both(0.0f), s2 = both(0.0f);
    {
      const uint8_t* at = ring + slot * (2 * half_slot);
      Row<T, VEC, E> x, dy;
      R::read(at, x_now, 0, t, tpr, cols, true, x);
      R::read(at + half_slot, dy_now, 0, t, tpr, cols, true, dy);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        const float2 d = dy.pair(i), h = mul2(add2(x.pair(i), both(-mean)), both(rstd)), dh = mul2(d, w[i]);
        s1 = add2(s1, dh);
        s2 = fma2(dh, h, s2);
        dw[i] = fma2(d, h, dw[i]);
        db[i] = add2(db[i], d);
      }
    }
    if (dx != nullptr) {
      const float c1 = warp_sum(s1.x + s1.y), c2 = warp_sum(s2.x + s2.y);
      float l1 = 0.0f, l2 = 0.0f;
      if (n > 0) take(l1, l2, n - 1);
      if (!lost) cluster_sum2_send(c1, c2, p, bar, peer, peers, n & 1);
      if (n > 0) finish(l1, l2);
    }
    ++n;
    slot = slot == SLOTS - 1 ? 0 : slot + 1;
    x_now += x_step;
    dy_now += dy_step;
    mean_last = mean;
    rstd_last = rstd;
    mean = mean_1;
    rstd = rstd_1;
    mean_1 = mean_2;
    rstd_1 = rstd_2;
  }
  if (dx != nullptr && block < a.rows) {
    float l1, l2;
    take(l1, l2, n - 1);
    finish(l1, l2);
  }
  ring_wait<0>();  // no copy outlives the slots
  cluster_meet();  // nor a peer's sums, which have been taken
  if (lost) {      // or else were sent before the meeting: far more than their way from a peer (1 us)
    if ((threadIdx.x & 31) == 0) atomicExch(&ln_gave_up, 1);
    for (const uint64_t t0 = global_ns(); global_ns() - t0 < LN_LINGER_NS;) {
    }
  }
  if (a.parts == nullptr) return;
  float* part = a.parts + block * 2 * a.cols + first;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float2(&v)[E / 2] = k == 0 ? dw : db;
#pragma unroll
    for (int i = 0; i < E / 2; i += 2) {
      const int c = (t + 2 * i / VEC * tpr) * VEC + 2 * i % VEC;
      if (c < cols)
        *reinterpret_cast<float4*>(part + k * int64_t(a.cols) + c) = make_float4(v[i].x, v[i].y, v[i + 1].x, v[i + 1].y);
    }
  }
}

// ------------------------------------------------ any width, any alignment
template <typename T>
constexpr int ln_dparam_cols = 16 / static_cast<int>(sizeof(T));

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

// Parts of dw and db alone.  A block has a strip of 32 N columns, a lane N of
// them: N next to each other (kWhole, one 16-byte chunk of each row) or 32
// apart.  Part blockIdx.y and its warps share the rows, some of a warp's in
// flight at once; the warps' sums meet in shared memory.
template <typename T, bool kWhole>
__global__ void __launch_bounds__(LN_THREADS) ln_dparam_kernel(const T* __restrict__ dy, int64_t ld_dy, const T* __restrict__ x,
                                                               int64_t ld_x, const float* __restrict__ mean_in,
                                                               const float* __restrict__ rstd_in, float* __restrict__ parts,
                                                               int64_t rows, int32_t cols) {
  constexpr int WARPS = LN_THREADS / 32, N = ln_dparam_cols<T>, ROWS = kWhole ? 4 : 2;
  __shared__ float red[2][WARPS][32 * N];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * (32 * N) + (kWhole ? lane * N : lane);
  float dw[N], db[N];
#pragma unroll
  for (int q = 0; q < N; ++q) dw[q] = db[q] = 0.0f;
  const int64_t step = int64_t(gridDim.y) * WARPS;
  for (int64_t row = int64_t(blockIdx.y) * WARPS + w; row < rows; row += ROWS * step) {
    float g[ROWS][N], v[ROWS][N], mean[ROWS], rstd[ROWS];
    uint4 gw[ROWS], vw[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const int64_t r = row + k * step;
      const bool on = r < rows;
      mean[k] = on ? __ldg(mean_in + r) : 0.0f;
      rstd[k] = on ? __ldg(rstd_in + r) : 0.0f;
      const T *gr = dy + (on ? r : 0) * ld_dy + c, *xr = x + (on ? r : 0) * ld_x + c;
      if constexpr (kWhole) {
        gw[k] = vw[k] = make_uint4(0, 0, 0, 0);
        if (on && c < cols) {
          gw[k] = *reinterpret_cast<const uint4*>(gr);
          vw[k] = *reinterpret_cast<const uint4*>(xr);
        }
      } else {
#pragma unroll
        for (int q = 0; q < N; ++q) {
          const bool in = on && c + 32 * q < cols;
          g[k][q] = in ? ln_load(gr + 32 * q) : 0.0f;
          v[k][q] = in ? ln_load(xr + 32 * q) : 0.0f;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      if constexpr (kWhole) {
        const uint32_t a[4] = {gw[k].x, gw[k].y, gw[k].z, gw[k].w}, b[4] = {vw[k].x, vw[k].y, vw[k].z, vw[k].w};
#pragma unroll
        for (int q = 0; q < N; ++q) {
          g[k][q] = sizeof(T) == 4 ? __uint_as_float(a[q & 3]) : (q & 1 ? bf16_hi(a[q / 2]) : bf16_lo(a[q / 2]));
          v[k][q] = sizeof(T) == 4 ? __uint_as_float(b[q & 3]) : (q & 1 ? bf16_hi(b[q / 2]) : bf16_lo(b[q / 2]));
        }
      }
#pragma unroll
      for (int q = 0; q < N; ++q) {
        dw[q] = fmaf(g[k][q], (v[k][q] - mean[k]) * rstd[k], dw[q]);
        db[q] += g[k][q];
      }
    }
  }
#pragma unroll
  for (int q = 0; q < N; ++q) {
    red[0][w][lane + 32 * q] = dw[q];
    red[1][w][lane + 32 * q] = db[q];
  }
  __syncthreads();
  float* p = parts + int64_t(blockIdx.y) * 2 * cols;
  for (int i = threadIdx.x; i < 2 * 32 * N; i += LN_THREADS) {
    const int k = i / (32 * N), at = i - k * (32 * N);
    const int64_t col = int64_t(blockIdx.x) * (32 * N) + (kWhole ? (at & 31) * N + at / 32 : at);
    if (col >= cols) continue;
    float s = red[k][0][at];
    for (int j = 1; j < WARPS; ++j) s += red[k][j][at];
    p[k * int64_t(cols) + col] = s;
  }
}

// dw and db from the parts, in a fixed order.  A block of n warps takes 32 of
// the 2 C sums, warp k of it the parts k, k + n, ..., all in flight at once.
constexpr int LN_SUM_LOADS = 10;  // a thread's, of LN_PARTS at most

template <typename D>
__global__ void __launch_bounds__(1024) ln_dparam_sum_kernel(const float* __restrict__ parts, int32_t n_parts, int32_t cols,
                                                             D* __restrict__ dw, D* __restrict__ db) {
  __shared__ float red[32][33];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, k = threadIdx.x >> 5, n = blockDim.x >> 5;
  const int64_t c = int64_t(blockIdx.x) * 32 + lane, width = 2 * int64_t(cols);
  float s = 0.0f;
  if (c < width) {
    float x[LN_SUM_LOADS];
    const float* p = parts + k * width + c;
#pragma unroll
    for (int i = 0; i < LN_SUM_LOADS; ++i) x[i] = k + n * i < n_parts ? p[n * i * width] : 0.0f;
#pragma unroll
    for (int i = 0; i < LN_SUM_LOADS; ++i) s += x[i];
  }
  red[k][lane] = s;
  __syncthreads();
  int64_t col = c;
  if (n == 32) {  // warp k adds up column k
    s = warp_sum(red[lane][k]);
    col += k - lane;
    if (lane != 0) return;
  } else {  // few terms, other blocks beside this one: a lane of warp 0 a column
    if (k != 0) return;
#pragma unroll 8
    for (int i = 1; i < n; ++i) s += red[i][lane];
  }
  if (col >= width) return;
  D* out = col < cols ? dw : db;
  if (out != nullptr) ln_store(out + (col < cols ? col : col - cols), s);
}

// Its threads: 32 warps where a block has an SM to itself; where there are
// more blocks, as few as have all the parts in flight (2 x 16384 sums of 76
// parts: 6 us, and 10 with 32 warps).
dim3 ln_sum_block(int64_t blocks, int32_t parts) {
  static_assert(32 * LN_SUM_LOADS >= LN_PARTS, "a thread takes its parts at once");
  return dim3(blocks <= 152 || parts > 16 * LN_SUM_LOADS ? 1024 : parts > 8 * LN_SUM_LOADS ? 512 : 256);
}

int32_t ln_parts(int64_t rows) { return static_cast<int32_t>(rows < LN_PARTS ? (rows > 0 ? rows : 1) : LN_PARTS); }

struct LnLd {
  int64_t x, y, dy, dx;
};

grs_status check_norm(const grs_norm* s, const char* who, LnLd* ld) {
  if (s == nullptr) return api_fail(GRS_ERR_INVALID_ARG, who, "shape is NULL");
  if (s->rows < 0 || s->cols < 1 || s->cols > GRS_MAX_WIDTH)
    return api_fail(GRS_ERR_SHAPE, who, "rows must be >= 0 and cols in [1, GRS_MAX_WIDTH]");
  if (!dtype_ok(s->dtype) || !dtype_ok(s->param_dtype) || !dtype_ok(s->grad_dtype))
    return api_fail(GRS_ERR_INVALID_ARG, who, "unknown element type");
  if (!(s->eps >= 0.0f) || std::isinf(s->eps)) return api_fail(GRS_ERR_INVALID_ARG, who, "eps must be finite and >= 0");
  *ld = {s->ld_x ? s->ld_x : s->cols, s->ld_y ? s->ld_y : s->cols, s->ld_dy ? s->ld_dy : s->cols,
         s->ld_dx ? s->ld_dx : s->cols};
  if (ld->x < s->cols || ld->y < s->cols || ld->dy < s->cols || ld->dx < s->cols)
    return api_fail(GRS_ERR_SHAPE, who, "a leading dimension is less than cols");
  return GRS_OK;
}

// Whether every row of a matrix starts at a multiple of 16 bytes.
bool rows16(const void* p, int64_t ld, int esize) { return api_aligned(p, 16) && ld * esize % 16 == 0; }

// Threads of a row of `cols` elements with e elements a thread: a power of two up to a warp, then whole warps.
int32_t ln_tpr(int32_t cols, int e) {
  const int64_t need = (int64_t(cols) + e - 1) / e;
  if (need > 32) return static_cast<int32_t>((need + 31) / 32 * 32);
  int32_t t = 1;
  while (t < need) t *= 2;
  return t;
}

// Rows at a time in a block of the forward ring, and blocks an SM.
//
// Up to 64 MB of x two blocks of about 256 threads an SM (8192 x 1024 fp32:
// 13.0 us, and 14.1 with one block); beyond, where x and y no longer share L2,
// one block:
//  fp32  as many rows as keep 96 KB of copies in flight on an SM (256 MB in
//        rows of 1024: 6.3 TB/s, and 5.6 with twice that, 5.5 with two thirds
//        of it; in rows of 2560 6.0, and 3.6 with one row at a time); where
//        the block's threads are enough for one row of less than that, two
//        blocks (rows of 5120: 5.9 and 4.9);
//  bf16  as many rows as it has threads for (256 MB in rows of 2048 and 4096:
//        5.9 and 6.0 TB/s, 5.8 and 5.8 with two blocks); two blocks for fewer
//        than three rows (rows of 8192: 6.4 and 6.3).
// In bf16 one block also where two have threads for fewer rows (rows of 5120,
// 48 MB: 5.0 and 3.8).
struct RingShape {
  int groups, blocks;
};

template <typename T>
RingShape ln_ring_shape(int64_t rows, int32_t cols, int32_t tpr) {
  const int64_t row_bytes = int64_t(cols) * sizeof(T);
  const bool beyond = rows * row_bytes > int64_t(64) << 20;
  const int most = LN_RING_THREADS / tpr < LN_RING_GROUPS ? LN_RING_THREADS / tpr : LN_RING_GROUPS;
  RingShape r;
  if (sizeof(T) == 4) {
    const int64_t in_flight = 24 << 10;  // four rows ahead of each group
    const int64_t want = beyond ? (in_flight + row_bytes - 1) / row_bytes : (256 + tpr / 2) / tpr;
    r.groups = want > most ? most : want < 1 ? 1 : static_cast<int>(want);
    r.blocks = !beyond || (most == 1 && row_bytes < in_flight) ? 2 : 1;
  } else {
    const int half = 256 / tpr;
    const bool one = most >= 3 && (beyond || 2 * half < most);
    r.groups = one ? most : half < 1 ? 1 : half;
    r.blocks = one ? 1 : 2;
  }
  return r;
}

template <typename T, typename W, int VEC, int E, bool kRing>
cudaError_t ln_forward_e(const LnFwd<T, W>& args, void* stream) {
  LnFwd<T, W> a = args;
  a.tpr = ln_tpr(a.cols, E);
  if constexpr (kRing) {
    const RingShape shape = ln_ring_shape<T>(a.rows, a.cols, a.tpr);
    const int groups = shape.groups, threads = groups * a.tpr;
    int64_t grid = (a.rows + groups - 1) / groups;
    if (grid > 152 * shape.blocks) grid = 152 * shape.blocks;
    using R = Ring<T, VEC, E>;
    constexpr int SLOTS = ring_slots(R::BYTES);
    constexpr int ring_most = SLOTS * (LN_RING_THREADS * R::BYTES + LN_RING_GROUPS * R::EXTRA);
    static_assert(ring_most <= 226 * 1024, "shared memory of a block");
    const cudaError_t e = allow_smem<ln_fwd_ring_kernel<T, W, VEC, E>>(ring_most);
    if (e != cudaSuccess) return e;
    return launch_pdl(ln_fwd_ring_kernel<T, W, VEC, E>, dim3(static_cast<unsigned>(grid)), dim3(threads),
                    size_t(SLOTS) * (threads * R::BYTES + groups * R::EXTRA), stream, a);
  } else {
    const int threads = a.tpr > 128 ? a.tpr : 128 / a.tpr * a.tpr;
    const int64_t per = threads / a.tpr;
    return launch_pdl(ln_fwd_kernel<T, W, VEC, E>, dim3(static_cast<unsigned>((a.rows + per - 1) / per)), dim3(threads), 0, stream, a);
  }
}

// Measured on bf16 rows of 2048: 32 elements a thread (64 threads a row)
// take 43.6 us for 32768 rows against 50.6 with 16 and 94 with 8, whose sums
// meet across more warps; up to 4096 rows 16 fill the SMs better, and a few
// rows are done soonest with 8 (one row: 2.2 us).
template <typename T, typename W, int VEC>
cudaError_t ln_forward_vec(const LnFwd<T, W>& a, void* stream, bool* done) {
  const int t8 = ln_tpr(a.cols, 8), t16 = ln_tpr(a.cols, 16);
  const int t32 = ln_tpr(a.cols, 32);
  *done = true;
  if (a.rows > 1216 || t16 > 1024) {
    const bool wide = sizeof(T) == 2 ? a.rows >= 4096 || t16 > LN_RING_THREADS : t16 > LN_RING_THREADS;
    if (!wide) return ln_forward_e<T, W, VEC, 16, true>(a, stream);
    if (t32 <= LN_RING_THREADS) return ln_forward_e<T, W, VEC, 32, true>(a, stream);
  }
  if (a.rows <= INT32_MAX && t8 <= 1024) return ln_forward_e<T, W, VEC, 8, false>(a, stream);
  if (a.rows <= INT32_MAX && t16 <= 1024) return ln_forward_e<T, W, VEC, 16, false>(a, stream);
  *done = false;
  return cudaSuccess;
}

template <typename T, typename W>
cudaError_t ln_forward(const grs_norm* s, const LnLd& ld, const void* x, const void* w, const void* b, void* y, float* mean,
                       float* rstd, void* stream) {
  const LnFwd<T, W> a{static_cast<const T*>(x), static_cast<const W*>(w), static_cast<const W*>(b), static_cast<T*>(y), mean,
                      rstd, ld.x, ld.y, s->rows, s->cols, 0, s->eps};
  constexpr int VEC = 16 / sizeof(T);
  bool done = false;
  const bool vec = s->cols % VEC == 0 && rows16(x, ld.x, sizeof(T)) && rows16(y, ld.y, sizeof(T)) && api_aligned(w, 16) && api_aligned(b, 16);
  const cudaError_t e = vec ? ln_forward_vec<T, W, VEC>(a, stream, &done) : ln_forward_vec<T, W, 2>(a, stream, &done);
  if (done || e != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>(s->rows < 1 << 20 ? s->rows : 1 << 20);
  return launch_pdl(ln_fwd_any_kernel<T, W>, dim3(grid), dim3(LN_THREADS), 0, stream, a.x, ld.x, a.w, a.b, a.y, ld.y, mean, rstd,
                  s->rows, s->cols, s->eps);
}

template <typename T, typename W, int VEC, int E, bool kParams>
cudaError_t ln_backward_e(const LnBwd<T, W>& args, int32_t* parts, void* stream) {
  LnBwd<T, W> a = args;
  a.tpr = ln_tpr(a.cols, E);
  // Wide rows: one block of 512 threads an SM, half as many parts (8192 x 2048
  // bf16: 24.6 us, and 25.7 with two of 256); narrow ones the other way round
  // (65536 x 128: 15.0 and 15.5).
  const int want = a.tpr >= 64 ? LN_BWD_THREADS : LN_BWD_THREADS / 2;
  const int groups = want / a.tpr, threads = groups * a.tpr;
  const int64_t most_parts = a.tpr >= 64 ? LN_PARTS / 2 : LN_PARTS;
  int64_t grid = (a.rows + groups - 1) / groups;
  if (grid > most_parts) grid = most_parts;
  if (grid < 1) grid = 1;
  *parts = static_cast<int32_t>(grid);
  using R = Ring<T, VEC, E>;
  constexpr int SLOTS = ring_slots(2 * R::BYTES);
  const size_t sums = size_t(threads) * E * 8;  // the groups' sums at the end, in the ring's place
  const size_t ring = LN_RED_BYTES + size_t(SLOTS) * 2 * (threads * R::BYTES + groups * R::EXTRA);
  constexpr int most = LN_RED_BYTES + SLOTS * 2 * LN_BWD_THREADS * (R::BYTES + R::EXTRA / 4);
  static_assert(most <= 227 * 1024, "shared memory of a block");
  const cudaError_t e = allow_smem<ln_bwd_kernel<T, W, VEC, E, kParams>>(most);
  if (e != cudaSuccess) return e;
  return launch_pdl(ln_bwd_kernel<T, W, VEC, E, kParams>, dim3(static_cast<unsigned>(grid)), dim3(threads), ring > sums ? ring : sums, stream, a);
}

// Clusters of `peers` blocks: as many as a GB300 holds at once, 152 SMs in GPCs
// that are no multiple of 4 or 8.  Fixed numbers, not what a device says of
// itself: each cluster leaves one part of dw and db, so their order of
// addition would go with the device.  One that holds fewer takes them in turn.
// Blocks an SM by registers: bf16 one (128 a thread), fp32 three of up to 320
// threads, else two (64).
template <typename T>
int32_t ln_wide_clusters(int peers, int threads) {
  const int blocks = sizeof(T) == 2 ? 1 : threads <= 320 ? 3 : 2;
  constexpr int32_t held[3][3] = {{76, 152, 228}, {36, 74, 110}, {15, 36, 51}};
  return held[peers == 2 ? 0 : peers == 4 ? 1 : 2][blocks - 1];
}

// Rows over the blocks of a cluster: 2, 4 or 8 of them, as few as hold a row
// (256 MB of bf16: rows of 20000 225 us in four blocks, half as much again in
// three; rows of 11968 186 us in two blocks of 384 threads, no less in four).
template <typename T, typename W, int E>
cudaError_t ln_backward_wide(const LnBwd<T, W>& args, int32_t* parts, void* stream) {
  LnBwd<T, W> a = args;
  int peers = 2;
  while (int64_t(peers) * LN_BWD_THREADS * E < a.cols) peers *= 2;
  const int32_t eights = (a.cols + 7) / 8;
  a.span = (eights + peers - 1) / peers * 8;
  a.tpr = ln_tpr(a.span, E);
  constexpr int slots = ln_wide_slots<T> * 2 * E * static_cast<int>(sizeof(T));  // a thread's
  static_assert(LN_WIDE_RED + slots * LN_BWD_THREADS <= 227 * 1024, "shared memory of a block");
  constexpr auto* kernel = ln_bwd_wide_kernel<T, W, E>;
  const cudaError_t e = allow_smem<kernel>(LN_WIDE_RED + slots * LN_BWD_THREADS);
  if (e != cudaSuccess) return e;
  const unsigned smem = LN_WIDE_RED + slots * a.tpr;
  int64_t clusters = ln_wide_clusters<T>(peers, a.tpr);
  if (clusters > a.rows) clusters = a.rows;
  *parts = static_cast<int32_t>(clusters);
  return launch_pdl_cluster(kernel, static_cast<unsigned>(peers), dim3(static_cast<unsigned>(clusters * peers)), dim3(a.tpr), smem,
                            stream, a);
}

// Whether whole rows are shared by a cluster: rows wider than a block's
// registers; fp32 also from 4096, where there are rows enough to pay for the
// sums' way (12500 x 5120 127 us, 172 in one block; 1562 rows 24.5 and 26.7,
// 390 rows 12.9 and 10.9).
template <typename T>
constexpr int ln_wide_elements = sizeof(T) == 4 ? 8 : 16;  // a thread's

template <typename T>
bool ln_shares_rows(int64_t rows, int32_t cols) {
  const bool wide = ln_tpr(cols, 16) > LN_BWD_THREADS || (sizeof(T) == 4 && ln_tpr(cols, 8) > LN_BWD_THREADS && rows >= 4 * 152);
  return rows > 0 && wide && cols <= LN_PEERS * LN_BWD_THREADS * ln_wide_elements<T>;
}

// dx, and the parts of dw and db (their number in *parts; 0: not done).
template <typename T, typename W, int VEC>
cudaError_t ln_backward_vec(const LnBwd<T, W>& a, int32_t* parts, bool* dx_done, void* stream) {
  const int t8 = ln_tpr(a.cols, 8), t16 = ln_tpr(a.cols, 16);
  *dx_done = true;
  // Fewer elements a thread where registers are short (fp32) or rows few.
  const bool eight = (a.rows <= LN_PARTS || sizeof(T) == 4) && t8 <= LN_BWD_THREADS;
  int32_t unused = 0;
  if constexpr (VEC > 2)
    if (ln_shares_rows<T>(a.rows, a.cols))
      return ln_backward_wide<T, W, ln_wide_elements<T>>(a, a.parts != nullptr ? parts : &unused, stream);
  if (a.parts != nullptr) {
    if (eight) return ln_backward_e<T, W, VEC, 8, true>(a, parts, stream);
    if (t16 <= LN_BWD_THREADS) return ln_backward_e<T, W, VEC, 16, true>(a, parts, stream);
  }
  if (a.dx != nullptr && a.rows > 0) {
    if (eight) return ln_backward_e<T, W, VEC, 8, false>(a, &unused, stream);
    if (t16 <= LN_BWD_THREADS) return ln_backward_e<T, W, VEC, 16, false>(a, &unused, stream);
  }
  *dx_done = false;
  return cudaSuccess;
}

// Every row of x, dy and dx and the parameters at multiples of 16 bytes, in whole chunks.
bool ln_whole_rows(const grs_norm* s, const LnLd& ld, const void* dy, const void* x, const void* w, const void* dx) {
  const int esize = dtype_size(s->dtype);
  return s->cols % (16 / esize) == 0 && rows16(x, ld.x, esize) && rows16(dy, ld.dy, esize) && (dx == nullptr || rows16(dx, ld.dx, esize)) &&
         api_aligned(w, 16);
}

template <typename T, typename W>
cudaError_t ln_backward(const grs_norm* s, const LnLd& ld, const void* dy, const void* x, const void* w, const float* mean,
                        const float* rstd, void* dx, void* dw, void* db, float* ws, const LnWait& wait, void* stream) {
  const bool params = dw != nullptr || db != nullptr;
  const LnBwd<T, W> a{static_cast<const T*>(dy), static_cast<const T*>(x), static_cast<const W*>(w), mean, rstd,
                      static_cast<T*>(dx), params ? ws : nullptr, ld.dy, ld.x, ld.dx, s->rows, s->cols, 0, s->cols, wait};
  if (dx == nullptr && !params) return cudaSuccess;
  constexpr int VEC = 16 / sizeof(T);
  const bool vec = ln_whole_rows(s, ld, dy, x, w, dx);
  int32_t parts = 0;
  bool dx_done = false;
  cudaError_t e = vec ? ln_backward_vec<T, W, VEC>(a, &parts, &dx_done, stream) : ln_backward_vec<T, W, 2>(a, &parts, &dx_done, stream);
  if (e != cudaSuccess) return e;
  if (!dx_done && dx != nullptr && s->rows > 0) {
    // Loose rows of more than 8192 elements, and rows beyond a cluster's registers: a block a row, the second
    // reading from L2 (14220 x 9001 bf16 with dw and db: 446 us, 637 with the rows in a block's registers).
    const unsigned grid = static_cast<unsigned>(s->rows < 1 << 20 ? s->rows : 1 << 20);
    e = launch_pdl(ln_dx_any_kernel<T, W>, dim3(grid), dim3(LN_THREADS), 0, stream, a.dy, ld.dy, a.x, ld.x, a.w, mean, rstd, a.dx,
                   ld.dx, s->rows, s->cols);
    if (e != cudaSuccess) return e;
  }
  if (params && parts == 0) {  // wide loose rows, or wider than a cluster's registers
    // A second pass over x and dy: enough strips of columns and parts of rows for eight blocks an SM.
    constexpr int64_t strip = 32 * ln_dparam_cols<T>;
    const int64_t strips = (s->cols + strip - 1) / strip;
    int64_t most = (8 * 152 + strips - 1) / strips, have = (s->rows + LN_THREADS / 32 - 1) / (LN_THREADS / 32);
    if (most > LN_PARTS) most = LN_PARTS;
    if (have > most) have = most;
    const int64_t limit = ln_parts(s->rows);
    parts = static_cast<int32_t>(have < 1 ? 1 : have > limit ? limit : have);
    const dim3 grid(static_cast<unsigned>(strips), static_cast<unsigned>(parts));
    e = vec ? launch_pdl(ln_dparam_kernel<T, true>, grid, dim3(LN_THREADS), 0, stream, a.dy, ld.dy, a.x, ld.x, mean, rstd, ws, s->rows, s->cols)
            : launch_pdl(ln_dparam_kernel<T, false>, grid, dim3(LN_THREADS), 0, stream, a.dy, ld.dy, a.x, ld.x, mean, rstd, ws, s->rows, s->cols);
    if (e != cudaSuccess) return e;
  }
  if (!params) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>((2 * int64_t(s->cols) + 31) / 32));
  const float* parts_in = ws;
  return s->grad_dtype == GRS_DTYPE_FP32
             ? launch_pdl(ln_dparam_sum_kernel<float>, grid, ln_sum_block(grid.x, parts), 0, stream, parts_in, parts, s->cols,
                        static_cast<float*>(dw), static_cast<float*>(db))
             : launch_pdl(ln_dparam_sum_kernel<uint16_t>, grid, ln_sum_block(grid.x, parts), 0, stream, parts_in, parts, s->cols,
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

static grs_status backward(const grs_norm* s, const void* dy, const void* x, const void* w, const float* mean, const float* rstd,
                           void* dx, void* dw, void* db, void* workspace, const LnWait& wait, void* stream, const char* who) {
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
  if (wait.quitter >= 0 && (dx == nullptr || !ln_whole_rows(s, ld, dy, x, w, dx) ||
                            !(s->dtype == GRS_DTYPE_FP32 ? ln_shares_rows<float>(s->rows, s->cols) : ln_shares_rows<uint16_t>(s->rows, s->cols))))
    return api_fail(GRS_ERR_SHAPE, who, "no rows that blocks share");
  const bool f = s->dtype == GRS_DTYPE_FP32, pf = s->param_dtype == GRS_DTYPE_FP32;
  float* ws = static_cast<float*>(workspace);
  const cudaError_t e = f ? (pf ? ln_backward<float, float>(s, ld, dy, x, w, mean, rstd, dx, dw, db, ws, wait, stream)
                                : ln_backward<float, uint16_t>(s, ld, dy, x, w, mean, rstd, dx, dw, db, ws, wait, stream))
                          : (pf ? ln_backward<uint16_t, float>(s, ld, dy, x, w, mean, rstd, dx, dw, db, ws, wait, stream)
                                : ln_backward<uint16_t, uint16_t>(s, ld, dy, x, w, mean, rstd, dx, dw, db, ws, wait, stream));
  return e == cudaSuccess ? GRS_OK : api_cuda_fail(e, who);
}

grs_status grs_layernorm_backward(const grs_norm* s, const void* dy, const void* x, const void* w, const float* mean,
                                  const float* rstd, void* dx, void* dw, void* db, void* workspace, void* stream) {
  return backward(s, dy, x, w, mean, rstd, dx, dw, db, workspace, LnWait{}, stream, "grs_layernorm_backward");
}

grs_status grs_selftest_layernorm_wait(const grs_norm* s, const void* dy, const void* x, const void* w, const float* mean,
                                       const float* rstd, void* dx, void* dw, void* db, void* workspace, int64_t limit_ns,
                                       int32_t quitter, int32_t quit_row, void* stream) {
  static const char who[] = "grs_selftest_layernorm_wait";
  if (limit_ns < 1000 || limit_ns > 2000000000LL) return api_fail(GRS_ERR_INVALID_ARG, who, "limit_ns must be in [1 us, 2 s]");
  if (quitter < 0 || quit_row < 0) return api_fail(GRS_ERR_INVALID_ARG, who, "quitter and quit_row must be >= 0");
  const LnWait wait{static_cast<uint64_t>(limit_ns), quitter, quit_row};
  return backward(s, dy, x, w, mean, rstd, dx, dw, db, workspace, wait, stream, who);
}

grs_status grs_layernorm_check_device_errors(void* stream) {
  static const char who[] = "grs_layernorm_check_device_errors";
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  void* flag = nullptr;
  int gave_up = 0;
  cudaError_t e = cudaStreamSynchronize(st);
  if (e == cudaSuccess) e = cudaGetSymbolAddress(&flag, ln_gave_up);
  if (e == cudaSuccess) e = cudaMemcpy(&gave_up, flag, sizeof(gave_up), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaMemsetAsync(flag, 0, sizeof(gave_up), st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return api_cuda_fail(e, who);
  return gave_up != 0 ? api_fail(GRS_ERR_TIMEOUT, who, "a bounded device wait timed out") : GRS_OK;
}

}  // extern "C"
