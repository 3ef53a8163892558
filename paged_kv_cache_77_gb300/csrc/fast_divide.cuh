// Division of 32-bit numbers by one that is fixed for a launch: a product and a shift.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pkv {

// n / d for 0 <= n < 2^31 and 1 <= d < 2^31. With s = ceil(log2 d) and m = ceil(2^(31 + s) / d),
// m d = 2^(31 + s) + e with 0 <= e < d <= 2^s, so n m / 2^(31 + s) = n / d + n e / (d 2^(31 + s)), and the
// error is below 1 / d: the floor is n / d's. m < 2^32 since d > 2^(s - 1).
struct FastDivide {
  uint32_t m = 0, s = 0;
  FastDivide() = default;
  explicit FastDivide(int d) {
    while ((1ll << s) < d) ++s;
    m = (uint32_t)(((1ull << (31 + s)) + (uint64_t)d - 1) / (uint64_t)d);
  }
  __device__ __forceinline__ uint32_t divide(uint32_t n) const {
    return (uint32_t)(((uint64_t)n * m) >> 31 >> s);
  }
};

}  // namespace pkv
