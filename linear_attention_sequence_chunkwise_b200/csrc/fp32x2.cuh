// fp32x2.cuh -- packed fp32: two lanes an instruction (sm_100), for kernels whose issue slots, not
// their FMA units, are what runs out.
#pragma once

#include <stdint.h>

namespace retnet {

using Two = uint64_t;
__device__ __forceinline__ Two two(float a, float b) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ Two two(float a) { return two(a, a); }
__device__ __forceinline__ float2 parts(Two x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Two mul2(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// (by the FMA units: two sign flips would be two instructions of the integer pipe)
__device__ __forceinline__ Two neg2(Two a) { return mul2(a, 0xbf800000bf800000ull); }
__device__ __forceinline__ float sum_of(Two a) {
  const float2 p = parts(a);
  return p.x + p.y;
}

}  // namespace retnet
