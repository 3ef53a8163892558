// fp32 arithmetic whose results do not depend on the build's floating-point flags.
#pragma once

#include <cuda_runtime.h>

namespace pkv {

// Arithmetic that keeps subnormals whatever the build's flags: each result is the IEEE one.
__device__ __forceinline__ float mul_ieee(float a, float b) {
  float r;
  asm("mul.rn.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float add_ieee(float a, float b) {
  float r;
  asm("add.rn.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float sub_ieee(float a, float b) {
  float r;
  asm("sub.rn.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float fma_ieee(float a, float b, float c) {
  float r;
  asm("fma.rn.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float div_ieee(float a, float b) {
  float r;
  asm("div.rn.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float neg_ieee(float a) {
  float r;
  asm("neg.f32 %0, %1;\n" : "=f"(r) : "f"(a));
  return r;
}
__device__ __forceinline__ float abs_ieee(float a) {
  float r;
  asm("abs.f32 %0, %1;\n" : "=f"(r) : "f"(a));
  return r;
}
// Maximum and minimum; NaN if either operand is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ double widen_ieee(float a) {
  double r;
  asm("cvt.f64.f32 %0, %1;\n" : "=d"(r) : "f"(a));
  return r;
}

}  // namespace pkv
