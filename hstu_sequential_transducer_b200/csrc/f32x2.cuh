// Arithmetic on pairs of fp32 values: one instruction for both (f32x2).
#pragma once

#include "common.cuh"

namespace hstu {

using F2 = float2;
__device__ __forceinline__ uint64_t bits(F2 a) { return *reinterpret_cast<const uint64_t*>(&a); }
__device__ __forceinline__ F2 pair(uint64_t a) { return *reinterpret_cast<const F2*>(&a); }
__device__ __forceinline__ F2 both(float a) { return make_float2(a, a); }
__device__ __forceinline__ F2 add(F2 a, F2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return pair(r);
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return pair(r);
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return pair(r);
}

// 1 / (1 + exp(-x)) by the hardware's 2^x and reciprocal (2 ulp each; exp
// flushes below 2^-126 to 0, and the reciprocal of an infinity is 0).
__device__ __forceinline__ F2 sigmoid2(F2 x) {
  F2 e = mul(x, both(-1.4426950408889634f));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.x));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.y));
  e = add(e, both(1.f));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.x));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.y));
  return e;
}

}  // namespace hstu
