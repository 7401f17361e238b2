// MXFP4 blocks: 32 values along a row share one power of two 2^(byte - 127)
// (E8M0, 255 = NaN); each value is an E2M1 code s|ee|m of magnitude 0, .5, 1,
// 1.5, 2, 3, 4 or 6.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace tmoe {

// Scale byte of a block from its max |v| (as bits of the fp32 maximum): the
// layer's UE8M0 rule with E2M1's largest value, e = ceil(log2(fp32(amax / 6)))
// clamped to [-127, 127], so that nothing saturates; amax = 0 gives -127. A
// block that holds an infinity or a NaN has no finite scale: 255 (NaN).
// Without the division: amax = m 2^k, 1 <= m < 2, and amax / 6 = (m / 1.5)
// 2^(k - 2), whose exponent rounds up to k - 2 while m <= 1.5 and to k - 1
// above, where m / 1.5 lies at least 2/3 of an ulp above 1 and so rounds above
// 1, except at k = -125: there the quotient is subnormal with half the
// precision, and one ulp above 1.5 still rounds to 1. (Checked against the
// division at every exponent.)
__device__ __forceinline__ uint32_t mxfp4_scale_byte(uint32_t amax_bits) {
  const uint32_t f = amax_bits >> 23, man = amax_bits & 0x7FFFFFu;
  const uint32_t byte = (uint32_t)max((int)f - 2 + (man > 0x400000u + (f == 2u ? 1u : 0u) ? 1 : 0), 0);
  return f == 255u ? 255u : byte;
}

// 2^-(e) for the scale byte e + 127 of a finite block.
__device__ __forceinline__ float mxfp4_inverse(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0u : (254u - byte) << 23);  // (byte <= 253 from fp32 data)
}

// 2^(byte - 127) in fp32, NaN for 255.
__device__ __forceinline__ float mxfp4_power(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7FC00000u : byte == 0u ? 0x00400000u : byte << 23);
}

// Eight scaled values -> eight codes, value 0 in the low nibble (round to
// nearest even, saturating at 6).
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n.reg .b8 a, b, c, d;\n"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      "mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Eight values of a block whose largest |v| has the bits amax_bits: returns
// their codes, `byte` the block's scale.
__device__ __forceinline__ uint32_t mxfp4_codes(float (&v)[8], uint32_t amax_bits, uint32_t& byte) {
  byte = mxfp4_scale_byte(amax_bits);
  const float inv = mxfp4_inverse(byte);
#pragma unroll
  for (int c = 0; c < 8; ++c) v[c] *= inv;
  return byte == 255u ? 0u : e2m1x8(v);
}

// Eight codes -> four fp16 pairs (exact).
__device__ __forceinline__ void e2m1x8_to_half(uint32_t c, uint32_t (&h)[4]) {
  asm("{\n.reg .b8 a, b, c, d;\n"
      "mov.b32 {a, b, c, d}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(c));
}

__device__ __forceinline__ void e2m1x8_to_f32(uint32_t c, float (&v)[8]) {
  uint32_t h[4];
  e2m1x8_to_half(c, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

}  // namespace tmoe
