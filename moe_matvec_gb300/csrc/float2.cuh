// Packed fp32 arithmetic: two floats an instruction.
#pragma once
#include "common.cuh"

namespace qmv {

// Two floats at once (packed fp32 arithmetic).
struct F2 {
  unsigned long long u;
  __device__ __forceinline__ static F2 of(float x, float y) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.u) : "f"(x), "f"(y));
    return r;
  }
  __device__ __forceinline__ float x() const { return __uint_as_float((uint32_t)u); }
  __device__ __forceinline__ float y() const { return __uint_as_float((uint32_t)(u >> 32)); }
};
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(a.u), "l"(b.u));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(a.u), "l"(b.u));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.u) : "l"(a.u), "l"(b.u), "l"(c.u));
  return r;
}

}  // namespace qmv
