// Queries as fp16 operands.
#pragma once

#include "device_common.cuh"
#include "ieee_math.cuh"
#include "mma_f16.cuh"

namespace pkv {

// A query row of 128 bf16 values, spread over the four lanes of a quad (32 each, in w): turns
// them into fp16, scaled by a power of two that brings the row's largest finite magnitude to
// [2^8, 2^9), and returns the power's inverse. All 8 bits stay but for elements 2^22 times
// smaller than the largest; infinities and NaN pass through.
__device__ __forceinline__ float query_to_f16(uint4 (&w)[4]) {
  uint32_t u[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    u[4 * i] = w[i].x;
    u[4 * i + 1] = w[i].y;
    u[4 * i + 2] = w[i].z;
    u[4 * i + 3] = w[i].w;
  }
  uint32_t top = 0;  // as bits
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t lo = u[i] << 16 & 0x7fffffffu, hi = u[i] & 0x7fff0000u;
    if (lo < 0x7f800000u && lo > top) top = lo;
    if (hi < 0x7f800000u && hi > top) top = hi;
  }
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  // Exponents of the factor and of its inverse, both normal numbers.
  const int e = min(262 - (int)(top >> 23), 253);
  const float up = __uint_as_float((uint32_t)e << 23);
#pragma unroll
  for (int i = 0; i < 16; ++i) u[i] = pack_f16(mul_ieee(bf16lo(u[i]), up), mul_ieee(bf16hi(u[i]), up));
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
  return __uint_as_float((uint32_t)(254 - e) << 23);
}

}  // namespace pkv
