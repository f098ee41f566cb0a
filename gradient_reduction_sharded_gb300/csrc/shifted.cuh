// A warp's 256 consecutive elements at any alignment, in 16-byte chunks.
#pragma once

#include <cstdint>

#include "device.cuh"
#include "packed.cuh"

namespace grs {

// A warp's 256 consecutive elements of an array that starts at any multiple
// of its element: 8 to a lane.
//
// Aligned runs go as 16-byte chunks.  For the others every lane moves the
// aligned chunk (or two, in fp32) that holds its first element, and the
// elements that lie in the next lane's chunk cross by a shuffle: K words and
// perhaps half a word.  Only the run's two ends go by element, or all of a
// run that the tensor's own ends cut short (`inner` false): a chunk that
// reaches outside the tensor is not touched.
struct Run {
  int mis;     // bytes that the run starts after a 16-byte boundary
  bool inner;  // 8 elements of the tensor before the run and 8 after it
};

template <typename G>
__device__ __forceinline__ Run run_of(const G* p, int64_t before, int64_t rest) {
  return {static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15), before >= 8 && rest >= 264};
}

// The N words that start BYTES (even, below 16) after the first of (own, next).
template <int BYTES, int N>
__device__ __forceinline__ void shift_words(const uint32_t (&own)[N], const uint32_t (&next)[4], uint32_t (&o)[N]) {
  constexpr int K = BYTES / 4;
  uint32_t w[N + 4];
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = own[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[N + i] = next[i];
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] = (BYTES & 2) != 0 ? __funnelshift_r(w[i + K], w[i + K + 1], 16) : w[i + K];
}

// Of chunk i of a lane whose 8 elements start `off` elements after its first
// aligned chunk (of el elements) the elements [lo, hi) may be read: elements
// [-before, n) of the lane.  May reach beyond the chunk.
struct Span {
  int lo, hi;
};
__host__ __device__ constexpr Span chunk_span(int el, int i, int off, int before, int n) {
  return {off - before - i * el, off + n - i * el};
}

// The chunk of 16 bytes at p: all of it, or its elements [lo, hi) and zeros.
__device__ __forceinline__ uint4 load_chunk(const uint16_t* p, int lo, int hi) {
  if (lo <= 0 && hi >= 8) return __ldcs(reinterpret_cast<const uint4*>(p));
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    w[q] = (2 * q >= lo && 2 * q < hi ? uint32_t(p[2 * q]) : 0u) | (2 * q + 1 >= lo && 2 * q + 1 < hi ? uint32_t(p[2 * q + 1]) << 16 : 0u);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 load_chunk(const float* p, int lo, int hi) {
  if (lo <= 0 && hi >= 4) return __ldcs(reinterpret_cast<const uint4*>(p));
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) w[q] = q >= lo && q < hi ? __float_as_uint(p[q]) : 0u;
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename G>
__device__ __forceinline__ uint4 load_chunk(const G* p, Span s) {
  return load_chunk(p, s.lo, s.hi);
}

// What a lane has of its 8 elements while they are on their way: its own
// aligned words (the last lane the chunk behind them too), shifted into place
// by finish().  Several can be in flight: start() only loads.
template <typename G>
struct Moving {
  static constexpr int N = static_cast<int>(sizeof(G)) * 2;  // words of 8 elements
  uint32_t own[N];
  uint4 last;

  // The lane's 8 elements at p, 16-byte aligned.
  __device__ __forceinline__ void start(const G* p) {
    const uint4* c = reinterpret_cast<const uint4*>(p);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = __ldcs(c + i);
      own[4 * i] = v.x;
      own[4 * i + 1] = v.y;
      own[4 * i + 2] = v.z;
      own[4 * i + 3] = v.w;
    }
  }

  // Elements [0, n) of the lane's 8 at p, zeros beyond, where nothing may be
  // read behind them or more than `before` elements before them.  Aligned
  // chunks that lie in there come whole, others by their elements.  mis:
  // bytes that the run starts after a 16-byte boundary; whole warp.
  __device__ __forceinline__ void start_within(const G* p, int mis, int before, int n) {
    constexpr int EL = 16 / static_cast<int>(sizeof(G));
    const int off = mis / static_cast<int>(sizeof(G));
    const G* c = p - off;
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = load_chunk(c + i * EL, chunk_span(EL, i, off, before, n));
      own[4 * i] = v.x;
      own[4 * i + 1] = v.y;
      own[4 * i + 2] = v.z;
      own[4 * i + 3] = v.w;
    }
    if (mis != 0 && (threadIdx.x & 31) == 31) last = load_chunk(c + N / 4 * EL, chunk_span(EL, N / 4, off, before, n));
  }

  template <int MIS>
  __device__ __forceinline__ void shift() {
    const bool end = (threadIdx.x & 31) == 31;
    uint32_t next[4] = {__shfl_down_sync(0xffffffffu, own[0], 1), __shfl_down_sync(0xffffffffu, own[1], 1),
                        __shfl_down_sync(0xffffffffu, own[2], 1), __shfl_down_sync(0xffffffffu, own[3], 1)};
    if (end) {
      next[0] = last.x;
      next[1] = last.y;
      next[2] = last.z;
      next[3] = last.w;
    }
    uint32_t w[N];
    shift_words<MIS>(own, next, w);
#pragma unroll
    for (int i = 0; i < N; ++i) own[i] = w[i];
  }

  // The same run as start's; whole warp.
  __device__ __forceinline__ void finish(int mis) {
    if (mis == 0) return;
    if constexpr (sizeof(G) == 2) {
      switch (mis) {
        case 2: shift<2>(); break;
        case 4: shift<4>(); break;
        case 6: shift<6>(); break;
        case 8: shift<8>(); break;
        case 10: shift<10>(); break;
        case 12: shift<12>(); break;
        default: shift<14>(); break;
      }
    } else {
      switch (mis) {
        case 4: shift<4>(); break;
        case 8: shift<8>(); break;
        default: shift<12>(); break;
      }
    }
  }

  __device__ __forceinline__ float2 pair(int q) const {
    if constexpr (sizeof(G) == 2) return bf16_pair(own[q]);
    return make_float2(__uint_as_float(own[2 * q]), __uint_as_float(own[2 * q + 1]));
  }
};

// The lane's N words to p, MIS bytes after a 16-byte boundary; whole warp.
// The last aligned chunk that starts in a lane's words ends in the next lane's.
template <int MIS, int N>
__device__ __forceinline__ void store_shifted(uint8_t* p, const uint32_t (&w)[N]) {
  constexpr int SKIP = 16 - MIS, HALF = MIS & 2;
  const int lane = threadIdx.x & 31;
  uint32_t next[4], c[N];
#pragma unroll
  for (int i = 0; i < 4; ++i) next[i] = __shfl_down_sync(0xffffffffu, w[i], 1);
  shift_words<SKIP>(w, next, c);
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    if (i < N / 4 - 1 || lane < 31)
      __stcs(reinterpret_cast<uint4*>(p + SKIP) + i, make_uint4(c[4 * i], c[4 * i + 1], c[4 * i + 2], c[4 * i + 3]));
  if (lane == 0) {  // the run's first SKIP bytes
    if (HALF) *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
#pragma unroll
    for (int j = 0; j < SKIP / 4; ++j)
      *reinterpret_cast<uint32_t*>(p + HALF + 4 * j) = HALF ? __funnelshift_r(w[j], w[j + 1 < 4 ? j + 1 : 3], 16) : w[j];
  }
  if (lane == 31) {  // and its last MIS bytes
    constexpr int L = N - 4;
#pragma unroll
    for (int j = 0; j < MIS / 4; ++j) *reinterpret_cast<uint32_t*>(p + 4 * L + SKIP + 4 * j) = c[L + j];
    if (HALF) *reinterpret_cast<uint16_t*>(p + 4 * L + 14) = static_cast<uint16_t>(w[N - 1] >> 16);
  }
}

// The lane's N words from p, MIS bytes after a 16-byte boundary; whole warp.
template <int MIS, int N>
__device__ __forceinline__ void load_shifted(const uint8_t* p, uint32_t (&o)[N]) {
  const uint4* c = reinterpret_cast<const uint4*>(p - MIS);
  uint32_t own[N];
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const uint4 v = __ldcs(c + i);
    own[4 * i] = v.x;
    own[4 * i + 1] = v.y;
    own[4 * i + 2] = v.z;
    own[4 * i + 3] = v.w;
  }
  const bool end = (threadIdx.x & 31) == 31;
  uint4 last;
  if (end) last = __ldcs(c + N / 4);
  uint32_t next[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) next[i] = __shfl_down_sync(0xffffffffu, own[i], 1);
  if (end) {
    next[0] = last.x;
    next[1] = last.y;
    next[2] = last.z;
    next[3] = last.w;
  }
  shift_words<MIS>(own, next, o);
}

// Elements [0, n) of the lane's 8 at p, zeros beyond, at once; whole warp.
// Beside Moving for its registers: of the list step's 48 it spills 0 to 32
// bytes, a Moving 24 to 112.
__device__ __forceinline__ void load8(const uint16_t* p, Run r, int n, float2 (&o)[4]) {
  uint32_t w[4];
  if (r.mis == 0 && n >= 8) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else if (r.inner) {
    const uint8_t* b = reinterpret_cast<const uint8_t*>(p);
    switch (r.mis) {
      case 2: load_shifted<2>(b, w); break;
      case 4: load_shifted<4>(b, w); break;
      case 6: load_shifted<6>(b, w); break;
      case 8: load_shifted<8>(b, w); break;
      case 10: load_shifted<10>(b, w); break;
      case 12: load_shifted<12>(b, w); break;
      default: load_shifted<14>(b, w); break;
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      w[q] = (2 * q < n ? uint32_t(p[2 * q]) : 0u) | (2 * q + 1 < n ? uint32_t(p[2 * q + 1]) << 16 : 0u);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) o[q] = bf16_pair(w[q]);
}

__device__ __forceinline__ void load8(const float* p, Run r, int n, float2 (&o)[4]) {
  uint32_t w[8];
  if (r.mis == 0 && n >= 8) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p)), b = __ldcs(reinterpret_cast<const uint4*>(p) + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  } else if (r.inner) {
    const uint8_t* b = reinterpret_cast<const uint8_t*>(p);
    switch (r.mis) {
      case 4: load_shifted<4>(b, w); break;
      case 8: load_shifted<8>(b, w); break;
      default: load_shifted<12>(b, w); break;
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) w[q] = q < n ? __float_as_uint(p[q]) : 0u;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) o[q] = make_float2(__uint_as_float(w[2 * q]), __uint_as_float(w[2 * q + 1]));
}

// The words of the lane's elements [0, n) to p; whole warp.
template <typename G>
__device__ __forceinline__ void store_words(G* p, Run r, int n, const uint32_t (&w)[sizeof(G) * 2]) {
  constexpr int N = static_cast<int>(sizeof(G)) * 2;
  uint8_t* b = reinterpret_cast<uint8_t*>(p);
  if (r.mis == 0 && n >= 8) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      __stcs(reinterpret_cast<uint4*>(p) + i, make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
  } else if (r.inner) {
    if constexpr (sizeof(G) == 2) {
      switch (r.mis) {
        case 2: store_shifted<2>(b, w); break;
        case 4: store_shifted<4>(b, w); break;
        case 6: store_shifted<6>(b, w); break;
        case 8: store_shifted<8>(b, w); break;
        case 10: store_shifted<10>(b, w); break;
        case 12: store_shifted<12>(b, w); break;
        default: store_shifted<14>(b, w); break;
      }
    } else {
      switch (r.mis) {
        case 4: store_shifted<4>(b, w); break;
        case 8: store_shifted<8>(b, w); break;
        default: store_shifted<12>(b, w); break;
      }
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < n) {
        if constexpr (sizeof(G) == 2)
          p[q] = static_cast<uint16_t>(w[q >> 1] >> (16 * (q & 1)));
        else
          p[q] = __uint_as_float(w[q]);
      }
  }
}

// The lane's elements [0, n) to p, rounded to the type; whole warp.
template <typename G>
__device__ __forceinline__ void store8(G* p, Run r, int n, const float2 (&o)[4]) {
  uint32_t w[sizeof(G) * 2];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (sizeof(G) == 2) {
      w[q] = to_bf16_pair(o[q]);
    } else {
      w[2 * q] = __float_as_uint(o[q].x);
      w[2 * q + 1] = __float_as_uint(o[q].y);
    }
  }
  store_words(p, r, n, w);
}

}  // namespace grs
