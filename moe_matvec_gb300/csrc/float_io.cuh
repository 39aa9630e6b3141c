// Loads and stores of values held as fp32, binary16 or bfloat16 (QMV_DT_*),
// computed with in fp32.
#pragma once
#include <cuda_bf16.h>

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

}  // namespace qmv
