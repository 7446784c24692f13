// Device helpers of the 4-bit cache: e2m1 codes, their group scales, and both
// conversions.
//
// An element of a 4-bit pool stands for e2m1 x s x g: e2m1 in {0, .5, 1, 1.5, 2,
// 3, 4, 6} with a sign, s the e4m3 scale of the 16 elements of a row that it is
// one of, g the fp32 scale of its KV head (a power of two, 2^-60 .. 2^60).
//   - e2m1 x s has 6 significand bits and lies between 2^-10 and 2,688: an f16
//     number, so a tile becomes an operand of f16 products exactly.
//   - A group belongs to one token, so tokens are written independently of each
//     other: nothing that the cache holds is read or moved by a write.
//   - g is one for the whole cache, so it leaves the products: it multiplies a
//     score, or an output row.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "device.cuh"

namespace pkv {
namespace fp4 {

constexpr int kGroup = 16;  // elements that share an e4m3 scale

// ------------------------------------------------------------- to values

// The eight codes of a word as f16 pairs: r[i] holds elements 2 i (low) and 2 i + 1.
__device__ __forceinline__ void codes_to_f16x2(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&x);
}

__device__ __forceinline__ float2 f16x2_to_float2(uint32_t u) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// ------------------------------------------------------------- to codes

// The larger of two magnitudes; NaN if one of them is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// a / d, where a is the exact sum of the returned value and a remainder: rounded
// to nearest, but odd where it is not exact, so that a later rounding to fewer
// bits decides as on the quotient itself (a border between two codes has an even
// last bit).  inv: 1 / d.
__device__ __forceinline__ float div_odd(float a, float d, float inv) {
  float q = a * inv;
  q = fmaf(fmaf(-q, d, a), inv, q);  // the nearest
  const float r = fmaf(-q, d, a);    // its remainder, exact
  const uint32_t bits = __float_as_uint(q);
  if (r != 0.f && (bits & 1u) == 0u) q = __uint_as_float(bits + (r > 0.f ? 1u : ~0u));
  return q;
}

// e4m3 code of the scale for magnitudes up to a (>= 0): the value nearest to
// a / 6, 448 at most; NaN for NaN.
__device__ __forceinline__ uint32_t scale_code(float a) {
  const float q = a > 0.f && a < 3.0e38f ? div_odd(a, 6.f, 1.f / 6.f) : a;
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(q));
  return r;
}

__device__ __forceinline__ float scale_value(uint32_t code) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(code)));
  return f16x2_to_float2(r).x;
}

// The codes of eight values, element 0 in the lowest four bits: the nearest e2m1,
// ties to the even code, 6 at most.
__device__ __forceinline__ uint32_t pack_codes(const float (&y)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return r;
}

// One group: its 16 values times 1 / g (exact) as codes and the scale's code.
// The decisions are those of exact arithmetic.  EXACT: values of 24 bits (fp32),
// whose quotient by the scale may be so near to a border that it is rounded onto
// it; a bf16 value lies on the border or 2^-9 away.
template <bool EXACT>
__device__ __forceinline__ void quantise(const float (&x)[16], float inv_g, uint2& codes,
                                         uint32_t& scale) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) a = max_nan(a, fabsf(x[i]));
  a *= inv_g;
  scale = scale_code(a);
  const float s = scale_value(scale);
  const float inv = s > 0.f ? 1.f / s : s;  // (0 and NaN stay)
  // past the largest code whatever its size: as far as that goes without infinities
  const bool large = !(a <= 1.0e30f);
  float y[2][8];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float v = fabsf(x[i] * inv_g);
    if (large) v = fminf(v, 1.0e30f);
    float q;
    if constexpr (EXACT) {
      q = s > 0.f ? div_odd(v, s, inv) : 0.f;
    } else {
      q = v * inv;
      q = fmaf(fmaf(-q, s, v), inv, q);  // exact on a border
    }
    // (the sign of a zero stays too)
    y[i >> 3][i & 7] = __uint_as_float((__float_as_uint(q) & 0x7fffffffu) |
                                       (__float_as_uint(x[i]) & 0x80000000u));
  }
  codes = make_uint2(pack_codes(y[0]), pack_codes(y[1]));
}

}  // namespace fp4
}  // namespace pkv
