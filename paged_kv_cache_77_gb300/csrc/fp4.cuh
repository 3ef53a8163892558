// The 4-bit cache's format on the device.
//
// A row of 128 values is 64 bytes of E2M1 codes (element 2i in the low half of byte i, 2i + 1
// in the high half; sign, two bits of exponent, one of fraction: 0, 0.5, 1, 1.5, 2, 3, 4, 6)
// and 8 scale bytes, one per 16 consecutive values. A scale byte is the upper 8 of the 15
// magnitude bits of an fp16 (5 of exponent, 3 of fraction; no sign): it widens by a shift,
// spans 2^-17 to 10240 without a second scale or a calibration, and code times scale has 6
// significant bits and at most 61440: exact in fp16, so the tensor cores take the values as
// they stand. 0xFF (an fp16 NaN) marks 16 values among which one is infinite or NaN.
#pragma once

#include <stdint.h>

#include "ieee_math.cuh"

namespace pkv {
namespace fp4 {

constexpr int kCodeBytes = 64;    // of a row of 128 values
constexpr int kScaleBytes = 8;
constexpr int kMaxScale = 0xE2;   // 10240: 6 of it are the last that fit fp16
constexpr int kNanScale = 0xFF;

// The eight values of four code bytes as pairs of fp16: r[i] holds byte i, its low code first.
__device__ __forceinline__ void widen(uint32_t codes, uint32_t (&r)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n"
      " cvt.rn.f16x2.e2m1x2 %1, b;\n cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(codes));
}

// Product of two pairs of fp16, subnormals kept.
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Scale bytes lo and hi (whole words below 256) as a pair of fp16.
__device__ __forceinline__ uint32_t scale_pair(uint32_t lo, uint32_t hi) {
  return __byte_perm(lo, hi, 0x4707) >> 1;
}
// Byte 0 or byte 1 of w, in both halves of a pair.
__device__ __forceinline__ uint32_t scale_dup0(uint32_t w) { return __byte_perm(w, 0, 0x0404) >> 1; }
__device__ __forceinline__ uint32_t scale_dup1(uint32_t w) { return __byte_perm(w, 0, 0x1414) >> 1; }

// Eight fp32 quotients as four code bytes: q[2i] goes to the low half of byte i.
__device__ __forceinline__ uint32_t codes(const float* q) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(r)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return r;
}

// fp32 value of a scale byte.
__device__ __forceinline__ float scale_value(uint32_t u) {
  float r;
  asm("{\n .reg .b16 h;\n cvt.u16.u32 h, %1;\n cvt.f32.f16 %0, h;\n}\n" : "=f"(r) : "r"(u << 7));
  return r;
}

// x / d, given -d, for a quotient that decides between codes or scales: exact where the exact quotient is an
// fp32 number, else within 2^-22 of itself (the remainder of a product with an approximate
// reciprocal, added back).
__device__ __forceinline__ float quotient(float x, float minus_d, float reciprocal) {
  const float q = mul_ieee(x, reciprocal);
  return fma_ieee(fma_ieee(q, minus_d, x), reciprocal, q);
}

// Scale byte of 16 bf16 values with largest magnitude `amax` (finite, not negative): the
// scale nearest to amax / 6, ties to the even byte. amax has 8 significant bits and 6 times
// a border between two scales 7: a quotient that does not equal a border is 2^-8 of itself away
// from it or more, one that does is exact.
__device__ __forceinline__ uint32_t scale_byte(float amax) {
  const float want = quotient(amax, -6.f, 1.f / 6.f);
  uint32_t u;
  if (want >= 0x1p-14f) {
    const uint32_t w = __float_as_uint(want);
    u = ((w + 0x7ffffu + (w >> 20 & 1u)) >> 20) - ((127 - 15) << 3);
  } else {
    u = (uint32_t)__float2int_rn(mul_ieee(want, 0x1p17f));
  }
  return u < (uint32_t)kMaxScale ? u : (uint32_t)kMaxScale;
}

// Codes of 16 bf16 values, in pairs, under a scale byte (not 0xFF): x / scale rounded to the nearest
// code, ties to the even one, magnitudes past 6 to 6. A border between two codes times the scale
// has 7 bits, x has 8: the quotient decides as above.
__device__ __forceinline__ uint2 quantise(const uint32_t (&x)[8], uint32_t scale) {
  if (scale == 0) return make_uint2(0, 0);
  const float s = scale_value(scale), minus = -s;
  float inv, q[16];
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(inv) : "f"(s));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    q[2 * i] = quotient(__uint_as_float(x[i] << 16), minus, inv);
    q[2 * i + 1] = quotient(__uint_as_float(x[i] & 0xffff0000u), minus, inv);
  }
  return make_uint2(codes(q), codes(q + 8));
}

}  // namespace fp4
}  // namespace pkv
