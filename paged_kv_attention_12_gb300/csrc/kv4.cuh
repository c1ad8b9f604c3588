// The 4-bit cache format (sm_103a): e2m1 codes with an e4m3 scale for every
// 16 channels of a token and KV head, and one fp32 scale per pool:
//   value = pool scale * e4m3 * e2m1.
//
// A pool is uint8 [num_blocks][Hkv][D / 128][1152]: units of 16 tokens x 128
// channels.  The layouts inside a unit are those the decode kernel's MMA
// fragments want, so that a lane's 16-byte shared-memory loads are whole
// fragments and free of bank conflicts:
//  * K: 1024 bytes of codes [16 tokens][64], channel 2i in the low nibble of
//    byte i, then the scales [16 tokens][8 groups];
//  * V: 1024 bytes of codes [8 groups of 16 channels][16 tokens][8], tokens
//    8..15 before tokens 0..7 in the odd groups, then the scales
//    [8 groups][16 tokens].
// 4.5 bits per value; 1152 is a multiple of 128, so every unit starts on a
// 128-byte line.
//
// Quantisation of a group of 16 values x (all fp32 arithmetic, each operation
// rounded once): r = max|x| / (6 * pool scale); s = e4m3 nearest to
// min(r, 448), ties to even; code = e2m1 nearest to x / (s * pool scale), ties
// to even, saturating; s = 0 gives zeros that keep their sign.  A group that
// holds an infinity or a NaN gets the scale NaN and zero codes: every reader
// sees NaN, never a finite number that stands for something else.
#pragma once

#include "common.cuh"

namespace pka {

constexpr int kUnitChannels = 128;
constexpr int kUnitCodes = 1024;
constexpr int kUnitBytes = 1152;

// Offset in a unit of the 8 code bytes of (token, group of 16 channels).
__host__ __device__ __forceinline__ int k_code_offset(int tok, int grp) {
  return tok * 64 + grp * 8;
}
__host__ __device__ __forceinline__ int v_code_offset(int tok, int grp) {
  return grp * 128 + ((tok * 8) ^ ((grp & 1) * 64));
}
// Offset in a unit of the scale of (token, group).
__host__ __device__ __forceinline__ int k_scale_offset(int tok, int grp) {
  return kUnitCodes + tok * 8 + grp;
}
__host__ __device__ __forceinline__ int v_scale_offset(int tok, int grp) {
  return kUnitCodes + grp * 16 + tok;
}

// Two e2m1 codes (the low nibble first) -> two f16, exact.
template <int BYTE>
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t w) {
  uint32_t r;
  if constexpr (BYTE == 0)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}"
        : "=r"(r)
        : "r"(w));
  else if constexpr (BYTE == 1)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}"
        : "=r"(r)
        : "r"(w));
  else if constexpr (BYTE == 2)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}"
        : "=r"(r)
        : "r"(w));
  else
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}"
        : "=r"(r)
        : "r"(w));
  return r;
}

// Two e4m3 values (the low byte first) -> two f16, exact (NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}

__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ void f16x2_to_f32(uint32_t v, float& lo, float& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(v));
}

// fp32 -> e4m3 (nearest, ties to even, saturating) as a byte.
__device__ __forceinline__ uint32_t f32_to_e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xffu;
}

// Eight fp32 -> eight e2m1 codes (nearest, ties to even, saturating), the
// first in the lowest nibble.
__device__ __forceinline__ uint32_t f32x8_to_e2m1x8(const float (&q)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return r;
}

// v0 / step and v1 / step from the reciprocal y of step: q = v y, then
// q + (v - q step) y, two lanes an instruction.
__device__ __forceinline__ void markstein_x2(float v0, float v1, float y, float step, float& q0,
                                             float& q1) {
  asm("{\n\t.reg .b64 v, y, s, q, r;\n\t"
      "mov.b64 v, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\tmov.b64 s, {%5, %5};\n\t"
      "mul.rn.f32x2 q, v, y;\n\tfma.rn.f32x2 r, q, s, v;\n\tfma.rn.f32x2 q, r, y, q;\n\t"
      "mov.b64 {%0, %1}, q;\n\t}"
      : "=f"(q0), "=f"(q1)
      : "f"(v0), "f"(v1), "f"(y), "f"(-step));
}

// A group of 16 bf16 values -> 8 code bytes and the scale byte.  s6 = 6 * pool
// scale, rounded to fp32.
__device__ __forceinline__ uint2 quantise_group(const uint4& in0, const uint4& in1,
                                                float pool_scale, float s6,
                                                uint32_t& scale_byte) {
  const uint32_t in[8] = {in0.x, in0.y, in0.z, in0.w, in1.x, in1.y, in1.z, in1.w};
  // the largest magnitude, as bf16 bits (from 0x7f80 on: infinity or NaN)
  uint32_t top2 = in[0] & 0x7fff7fffu;
#pragma unroll
  for (int i = 1; i < 8; ++i) top2 = __vmaxu2(top2, in[i] & 0x7fff7fffu);
  const uint32_t top = max(top2 & 0xffffu, top2 >> 16);
  if (top >= 0x7f80u) {
    scale_byte = 0x7fu;
    return make_uint2(0u, 0u);
  }
  const float ftop = __uint_as_float(top << 16);
  scale_byte = f32_to_e4m3(fminf(__fdiv_rn(ftop, s6), 448.f));
  float s, unused;
  f16x2_to_f32(e4m3x2_to_f16x2(static_cast<uint16_t>(scale_byte)), s, unused);
  const float step = __fmul_rn(s, pool_scale);
  // x / step, rounded to nearest: with the correctly rounded reciprocal y and
  // q = x y, the remainder x - q step is exact in one fma and q + remainder * y
  // is the correctly rounded quotient (P. Markstein, "Computation of elementary
  // functions on the IBM RISC System/6000 processor", 1990), as long as nothing
  // leaves the normal range.  Steps near its ends, and groups that saturate by
  // more than their rounding, take the division itself.
  const float y = __frcp_rn(step);
  const bool plain = step > 0x1p-60f && step < 0x1p60f && __fmul_rn(ftop, y) < 16.f;
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v0, v1, q0, q1;
      bf16x2_to_f32(in[h * 4 + i], v0, v1);
      markstein_x2(v0, v1, y, step, q0, q1);
      q[2 * i] = copysignf(q0, v0);  // (-0 stays -0)
      q[2 * i + 1] = copysignf(q1, v1);
    }
    if (!plain) {
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {
        const uint32_t word = (i >> 1) == 0 ? in[h * 4] : (i >> 1) == 1 ? in[h * 4 + 1]
                              : (i >> 1) == 2 ? in[h * 4 + 2] : in[h * 4 + 3];
        const float v = __uint_as_float((i & 1) ? word & 0xffff0000u : word << 16);
        // s = 0 (or s * pool scale below the smallest fp32): signed zeros
        const float d = step > 0.f ? __fdiv_rn(v, step) : copysignf(0.f, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) q[k] = k == i ? d : q[k];
      }
    }
    w[h] = f32x8_to_e2m1x8(q);
  }
  return make_uint2(w[0], w[1]);
}

}  // namespace pka
