// A warp's product of bf16 matrices with fp32 sums.
#pragma once

#include <stdint.h>

namespace pkv {

// d = A B with A of 16 rows and 16 columns, B of 8 columns. Lane 4 i + c holds of A the columns
// 2c, 2c + 1 of rows i and i + 8, then 2c + 8, 2c + 9 of both; of B those rows of column i; of d
// columns 2c, 2c + 1 of row i, then of row i + 8.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

}  // namespace pkv
