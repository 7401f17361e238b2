// Element types of the entry points that take a tm_dtype: conversion to and
// from fp32 (one rounding to nearest even on the way out).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace tmoe {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// N consecutive elements as fp32. `vec`: p is aligned to 16 bytes and N
// elements are whole 16-byte words; else one element at a time.
template <int N, typename T>
__device__ __forceinline__ void load_f32(const T* __restrict__ p, bool vec, float (&v)[N]) {
  constexpr int PER = 16 / (int)sizeof(T);
  static_assert(N % PER == 0, "whole 16-byte words");
  if (vec) {
#pragma unroll
    for (int c = 0; c < N / PER; ++c) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + c);
      const T* t = reinterpret_cast<const T*>(&q);
#pragma unroll
      for (int i = 0; i < PER; ++i) v[c * PER + i] = to_f32(t[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = to_f32(p[i]);
  }
}

template <int N, typename T>
__device__ __forceinline__ void store_f32(T* __restrict__ p, bool vec, const float (&v)[N]) {
  constexpr int PER = 16 / (int)sizeof(T);
  static_assert(N % PER == 0, "whole 16-byte words");
  if (vec) {
#pragma unroll
    for (int c = 0; c < N / PER; ++c) {
      uint4 q;
      T* t = reinterpret_cast<T*>(&q);
#pragma unroll
      for (int i = 0; i < PER; ++i) t[i] = from_f32<T>(v[c * PER + i]);
      reinterpret_cast<uint4*>(p)[c] = q;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = from_f32<T>(v[i]);
  }
}

}  // namespace tmoe

// Calls F with a value of the element type of tm_dtype `d`.
#define TM_BY_DTYPE(d, F)                     \
  ((d) == TM_F32    ? F(float())              \
   : (d) == TM_BF16 ? F(__nv_bfloat16())      \
                    : F(__half()))
