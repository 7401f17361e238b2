// Element types of the entry points that take a tm_dtype: conversion to and
// from fp32 (one rounding to nearest even on the way out).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <type_traits>

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

// Eight consecutive elements, of which the first n (0..8) exist. VEC: the
// elements are whole 16-byte words at an aligned address and n is 0 or 8; the
// words are then loaded without a branch, and converted where they are used,
// so that a thread's loads can all be in flight at once.
template <typename T, bool VEC>
struct Eight {
  static constexpr int kWords = 8 * (int)sizeof(T) / 16;
  uint4 q[kWords];

  __device__ __forceinline__ void load(const T* __restrict__ p, int n) {
    if (VEC) {
#pragma unroll
      for (int w = 0; w < kWords; ++w)
        q[w] = n == 8 ? __ldg(reinterpret_cast<const uint4*>(p) + w) : make_uint4(0, 0, 0, 0);
    } else {
      T* t = reinterpret_cast<T*>(q);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = i < n ? p[i] : from_f32<T>(0.0f);
    }
  }
  __device__ __forceinline__ void to(float (&v)[8]) const {
    const T* t = reinterpret_cast<const T*>(q);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(t[i]);
  }
  // The largest |v| of the eight and of the three neighbouring lanes' (four
  // lanes from a multiple of four), as the bits of an fp32: these compare like
  // the values, with infinities and then NaN above all numbers. 16-bit types
  // compare two at a time. All 32 lanes take part.
  __device__ __forceinline__ uint32_t block_amax_bits() const {
    if (sizeof(T) == 2) {
      const uint32_t a = 0x7FFF7FFFu;
      uint32_t m = __vmaxu2(__vmaxu2(q[0].x & a, q[0].y & a), __vmaxu2(q[0].z & a, q[0].w & a));
      m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      const uint16_t h = (uint16_t)max(m >> 16, m & 0xFFFFu);
      return __float_as_uint(to_f32(*reinterpret_cast<const T*>(&h)));
    }
    uint32_t m = 0;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      const uint32_t a = 0x7FFFFFFFu;
      m = max(max(m, max(q[w].x & a, q[w].y & a)), max(q[w].z & a, q[w].w & a));
    }
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    return max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  }
  __device__ __forceinline__ void from(const float (&v)[8]) {
    T* t = reinterpret_cast<T*>(q);
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = from_f32<T>(v[i]);
  }
  __device__ __forceinline__ void store(T* __restrict__ p, int n) const {
    if (VEC) {
      if (n == 8) {
#pragma unroll
        for (int w = 0; w < kWords; ++w) reinterpret_cast<uint4*>(p)[w] = q[w];
      }
    } else {
      const T* t = reinterpret_cast<const T*>(q);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = t[i];
    }
  }
};

// Whether rows of `cols` elements of `es` bytes, `ld` elements apart, can be
// read as Eight<T, true>.
inline bool eights(const void* p, int64_t ld, int64_t cols, int es) {
  return ((uintptr_t)p) % 16 == 0 && (ld * es) % 16 == 0 && cols % 8 == 0;
}

// n / d for 0 <= n < 2^31 by one multiplication: m = floor(2^(31+L) / d) + 1
// with L = ceil(log2 d) is at most 2^(31+L)/d + 1, and the excess times n stays
// below 2^(31+L), so the quotient is exact.
struct FastDiv {
  uint32_t d, m, shift;
  explicit FastDiv(uint32_t div) : d(div) {
    uint32_t l = 0;
    while ((1ull << l) < div) ++l;
    shift = 31 + l;
    m = (uint32_t)((1ull << shift) / div + 1);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (uint32_t)(((uint64_t)n * m) >> shift); }
};

}  // namespace tmoe

// Calls F with a value of the element type of tm_dtype `d` (and with whether
// its rows are whole eights).
#define TM_BY_DTYPE(d, F)                     \
  ((d) == TM_F32    ? F(float())              \
   : (d) == TM_BF16 ? F(__nv_bfloat16())      \
                    : F(__half()))
#define TM_BY_DTYPE_VEC(d, vec, F)                                                                              \
  ((d) == TM_F32 ? ((vec) ? F(float(), std::true_type()) : F(float(), std::false_type()))                       \
   : (d) == TM_BF16 ? ((vec) ? F(__nv_bfloat16(), std::true_type()) : F(__nv_bfloat16(), std::false_type()))    \
                    : ((vec) ? F(__half(), std::true_type()) : F(__half(), std::false_type())))
