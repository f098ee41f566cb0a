// Two fp32 numbers in one instruction: sm_103a adds, multiplies and fuses
// pairs of neighbouring registers (add/mul/fma.rn.f32x2).  The streaming kernels that are bound
// by instruction issue, not by memory, work on pairs.
#pragma once

#include <cstdint>

namespace grs {

__device__ __forceinline__ uint64_t pair_bits(float2 a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}

__device__ __forceinline__ float2 pair_floats(uint64_t r) {
  float2 a;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(r));
  return a;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair_bits(a)), "l"(pair_bits(b)));
  return pair_floats(r);
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair_bits(a)), "l"(pair_bits(b)));
  return pair_floats(r);
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pair_bits(a)), "l"(pair_bits(b)), "l"(pair_bits(c)));
  return pair_floats(r);
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// The product rounded by itself, whatever is added to it.  The assembler
// fuses mul.rn.f32x2 and an addition of its result into one rounding (which
// it does not do with the scalar mul.rn.f32), also where the product is
// written as a fused one with a -0 that it knows; with a -0 that comes in at
// run time the product stays, and has a product's value and sign.
__device__ __forceinline__ float2 mul2_rounded(float2 a, float2 b, float minus_zero) { return fma2(a, b, both(minus_zero)); }

// bf16 pair in one word <-> two floats.
__device__ __forceinline__ float2 bf16_pair(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t to_bf16_pair(float2 a) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(a.y), "f"(a.x));
  return r;
}

}  // namespace grs
