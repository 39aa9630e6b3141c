// Loads and stores of values held as fp32, binary16 or bfloat16 (QMV_DT_*),
// computed with in fp32.
#pragma once
#include <cuda_bf16.h>

#include <type_traits>

#include "common.cuh"

namespace qmv {

template <int DT>
struct Elem;
template <>
struct Elem<QMV_DT_F32> {
  using type = float;
};
template <>
struct Elem<QMV_DT_F16> {
  using type = __half;
};
template <>
struct Elem<QMV_DT_BF16> {
  using type = __nv_bfloat16;
};

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_float(float v, float& o) { o = v; }
__device__ __forceinline__ void from_float(float v, __half& o) { o = __float2half_rn(v); }
__device__ __forceinline__ void from_float(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }

// N consecutive values (N * sizeof(T) a multiple of 8 bytes, p aligned to
// it up to 16) as wide loads / stores.
template <int N, class T>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[N]) {
  constexpr int BYTES = N * (int)sizeof(T);
  static_assert(BYTES % 8 == 0, "whole 8-byte words");
  alignas(16) T t[N];
  if constexpr (BYTES % 16 == 0) {
#pragma unroll
    for (int i = 0; i < BYTES / 16; i++) reinterpret_cast<uint4*>(t)[i] = reinterpret_cast<const uint4*>(p)[i];
  } else {
#pragma unroll
    for (int i = 0; i < BYTES / 8; i++) reinterpret_cast<uint2*>(t)[i] = reinterpret_cast<const uint2*>(p)[i];
  }
#pragma unroll
  for (int i = 0; i < N; i++) v[i] = to_float(t[i]);
}
template <int N, class T>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[N]) {
  constexpr int BYTES = N * (int)sizeof(T);
  static_assert(BYTES % 8 == 0, "whole 8-byte words");
  alignas(16) T t[N];
#pragma unroll
  for (int i = 0; i < N; i++) from_float(v[i], t[i]);
  if constexpr (BYTES % 16 == 0) {
#pragma unroll
    for (int i = 0; i < BYTES / 16; i++) reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<uint4*>(t)[i];
  } else {
#pragma unroll
    for (int i = 0; i < BYTES / 8; i++) reinterpret_cast<uint2*>(p)[i] = reinterpret_cast<uint2*>(t)[i];
  }
}

// N consecutive values of type T on their way from or to memory, in whole
// registers (arrays of 16-bit values that are loaded under a condition become
// a register and a merge per value).  N * sizeof(T) is 4, 8, 16 or 32 bytes, and
// memory is aligned to it up to 16; a single 16-bit value takes a register.
template <class T, int N>
struct Packed {
  static constexpr int BYTES = N * (int)sizeof(T), WORDS = BYTES < 4 ? 1 : BYTES / 4;
  static_assert(BYTES == 2 || BYTES == 4 || BYTES == 8 || BYTES % 16 == 0, "whole loads");
  uint32_t w[WORDS];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < WORDS; i++) w[i] = 0;
  }
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (BYTES == 2) {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else if constexpr (BYTES == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (BYTES == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < WORDS / 4; i++) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (BYTES == 2) {
      *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
    } else if constexpr (BYTES == 4) {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    } else if constexpr (BYTES == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < WORDS / 4; i++)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
  }
  __device__ __forceinline__ void to(float (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < N; i++) {
      if constexpr (sizeof(T) == 4) {
        v[i] = __uint_as_float(w[i]);
      } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
      } else if (!(i & 1)) {
        const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i / 2]));
        v[i] = t.x;
        if constexpr (N > 1) v[i + 1] = t.y;
      }
    }
  }
  __device__ __forceinline__ void from(const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i++) {
      if constexpr (sizeof(T) == 4) {
        w[i] = __float_as_uint(v[i]);
      } else if (!(i & 1)) {
        const float next = N > 1 ? v[(i + 1) % N] : 0.f;
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
          const __nv_bfloat162 t = __floats2bfloat162_rn(v[i], next);
          w[i / 2] = *reinterpret_cast<const uint32_t*>(&t);
        } else {
          const __half2 t = __floats2half2_rn(v[i], next);
          w[i / 2] = *reinterpret_cast<const uint32_t*>(&t);
        }
      }
    }
  }
};

}  // namespace qmv
