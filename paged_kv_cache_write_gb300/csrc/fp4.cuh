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

// The larger of two magnitudes, as their bits; NaN if one of them is.
__device__ __forceinline__ float max_mag(float a, float b) {
  return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
}

// 1 / g for a power of two (normal range).
__device__ __forceinline__ float pow2_inverse(float g) {
  return __uint_as_float(0x7f000000u - __float_as_uint(g));
}

// Whether g is a head's scale that codes can be made for: a power of two, 2^-60 .. 2^60.
__device__ __forceinline__ bool is_head_scale(float g) {
  const uint32_t u = __float_as_uint(g);
  return (u & 0x007fffffu) == 0u && u - (67u << 23) <= (120u << 23);
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

// Two vectors of eight elements as codes, and their groups' scales' codes.
struct Codes {
  uint32_t a, b, scale_a, scale_b;
};

// Codes of eight values under a scale (its code; g: the head's) for magnitudes whose
// largest is amax, over g.  The decisions are those of exact arithmetic.
//   A bf16 value lies on a border between two codes or 2^-9 away from it, so its
//   quotient has to be exact on a border and good to some bits elsewhere: 1 / (s g) is
//   taken as two terms, hi (rounded down) and lo, and x hi + x lo rounded once.  (With
//   one term, quotients by scales of 13 .. 15 eighths miss their borders.)  Both terms
//   are >= 0, so a zero keeps its sign.
//   EXACT, for fp32: a quotient may be so near to a border that it is rounded onto it.
template <bool EXACT>
__device__ __forceinline__ uint32_t codes_under(const float2* x, float amax, uint32_t scale,
                                                float g) {
  const float s = scale_value(scale);
  float y[8];
  if constexpr (EXACT) {
    const float inv_g = pow2_inverse(g), inv = s > 0.f ? 1.f / s : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = i & 1 ? x[i / 2].y : x[i / 2].x;
      const float q = s > 0.f ? div_odd(fminf(fabsf(v * inv_g), 1.0e30f), s, inv) : 0.f;
      y[i] = __uint_as_float(__float_as_uint(q) | (__float_as_uint(v) & 0x80000000u));
    }
  } else {
    const float sg = s * g;
    const float hi = s > 0.f ? __frcp_rz(sg) : 0.f;
    const float lo = fmaf(-sg, hi, 1.f) * hi;  // (0 where s is)
    const float2 hi2 = make_float2(hi, hi), lo2 = make_float2(lo, lo);
    const bool large = !(amax <= 1.0e30f);  // no infinities and NaN below
    const float most = 1.0e30f * g;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 v = x[i];
      if (large) v = make_float2(fminf(fmaxf(v.x, -most), most), fminf(fmaxf(v.y, -most), most));
      const float2 q = __ffma2_rn(v, hi2, __fmul2_rn(v, lo2));
      y[2 * i] = q.x;
      y[2 * i + 1] = q.y;
    }
  }
  return pack_codes(y);
}

// The largest magnitude of eight fp32 values, or of eight bf16 values in four words; NaN if
// one is (its bits are the larger).
__device__ __forceinline__ float amax8(float4 a, float4 b) {
  const uint32_t u[8] = {__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(a.z),
                         __float_as_uint(a.w), __float_as_uint(b.x), __float_as_uint(b.y),
                         __float_as_uint(b.z), __float_as_uint(b.w)};
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, u[i] & 0x7fffffffu);
  return __uint_as_float(m);
}
__device__ __forceinline__ float amax8(uint4 w) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  __nv_bfloat162 m = __float2bfloat162_rn(0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&u[i])));
  return max_mag(__low2float(m), __high2float(m));
}

// One group of 16 values.
// (amax_a, amax_b: the largest magnitudes of its halves)
template <bool EXACT>
__device__ __forceinline__ Codes quantise(const float2 (&x)[8], float amax_a, float amax_b, float g) {
  const float a = max_mag(amax_a, amax_b) * pow2_inverse(g);
  Codes r;
  r.scale_a = r.scale_b = scale_code(a);
  r.a = codes_under<EXACT>(x, a, r.scale_a, g);
  r.b = codes_under<EXACT>(x + 4, a, r.scale_b, g);
  return r;
}

// Halves of two groups, whose largest magnitudes are ma and mb; other(j, ma, mb) is the largest magnitude
// in the other half of half j's group (both by every lane of the warp).
template <bool EXACT, typename Other>
__device__ __forceinline__ Codes quantise_apart(const float2 (&x)[8], float ma, float mb, float g,
                                                Other other) {
  const float oa = other(0, ma, mb), ob = other(1, ma, mb);
  const float a = max_mag(ma, oa) * pow2_inverse(g), b = max_mag(mb, ob) * pow2_inverse(g);
  Codes r;
  r.scale_a = scale_code(a);
  r.scale_b = scale_code(b);
  r.a = codes_under<EXACT>(x, a, r.scale_a, g);
  r.b = codes_under<EXACT>(x + 4, b, r.scale_b, g);
  return r;
}

}  // namespace fp4
}  // namespace pkv
