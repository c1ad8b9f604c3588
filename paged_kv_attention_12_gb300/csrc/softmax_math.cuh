// Softmax arithmetic of the tensor-core attention kernels: packed fp32 pairs,
// three-input extrema and the forms of tanh for the logit cap.
#pragma once

#include "common.cuh"

namespace pka {

namespace {

// Packed fp32 pairs (sm_100 family): one instruction computes both lanes of
// a float2, each rounded exactly as the scalar fmaf / a * b / a + b is.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// Three-input maximum and minimum (sm_100 family): fmaxf / fminf of three.
__device__ __forceinline__ float max3f(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float min3f(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// exp2-based tanh: tanh(y) = 1 - 2 / (exp(2y) + 1); absolute error ~1e-7;
// NaN stays NaN.
__device__ __forceinline__ float tanh_via_exp2(float y) {
  const float e = fast_exp2(min_nan(2.f * kLog2e * y, 126.f));
  return 1.f - __fdividef(2.f, e + 1.f);
}

// tanh(y) for |y| < 1/8 from y - y^3/3 + 2 y^5/15 (the first omitted term,
// 17 y^7 / 315, is below 2.6e-8 there): four FMA-pipe operations.
__device__ __forceinline__ float tanh_taylor_short(float y) {
  const float y2 = y * y;
  const float q = fmaf(y2, 2.f / 15.f, -1.f / 3.f);
  return fmaf(y * y2, q, y);
}

// tanh(y) for |y| < 0.5 from its odd Taylor series through y^11 (the first
// omitted term, 21844 y^13 / 6081075, is below 4.5e-7 there): FMA-pipe work
// only, where the exp2 form needs two MUFU operations.
__device__ __forceinline__ float tanh_taylor(float y) {
  const float y2 = y * y;
  float q = fmaf(y2, -1382.f / 155925.f, 62.f / 2835.f);
  q = fmaf(y2, q, -17.f / 315.f);
  q = fmaf(y2, q, 2.f / 15.f);
  q = fmaf(y2, q, -1.f / 3.f);
  return fmaf(y * y2, q, y);
}

}  // namespace

}  // namespace pka
