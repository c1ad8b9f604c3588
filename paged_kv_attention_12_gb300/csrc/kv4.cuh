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

// Two fp32 -> two e2m1 codes (nearest, ties to even, saturating) in a byte,
// `lo` in the low nibble.
__device__ __forceinline__ uint32_t f32x2_to_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
      "mov.b32 %0, {b, b, b, b};\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r & 0xffu;
}

// A group of 16 values -> 8 code bytes and the scale byte.  s6 = 6 * pool
// scale, rounded to fp32.
__device__ __forceinline__ uint2 quantise_group(const float (&x)[16], float pool_scale, float s6,
                                                uint32_t& scale_byte) {
  float top = 0.f;
  bool finite = true;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float a = fabsf(x[i]);
    finite = finite && (a <= 3.402823466e38f);
    top = fmaxf(top, a);
  }
  if (!finite) {
    scale_byte = 0x7fu;
    return make_uint2(0u, 0u);
  }
  scale_byte = f32_to_e4m3(fminf(__fdiv_rn(top, s6), 448.f));
  float s, unused;
  f16x2_to_f32(e4m3x2_to_f16x2(static_cast<uint16_t>(scale_byte)), s, unused);
  const float step = __fmul_rn(s, pool_scale);
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    w[h] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // s = 0 (or s * pool scale below the smallest fp32): zeros with a sign
      const float a = x[h * 8 + 2 * i], b = x[h * 8 + 2 * i + 1];
      const float ya = step > 0.f ? __fdiv_rn(a, step) : copysignf(0.f, a);
      const float yb = step > 0.f ? __fdiv_rn(b, step) : copysignf(0.f, b);
      w[h] |= f32x2_to_e2m1x2(ya, yb) << (8 * i);
    }
  }
  return make_uint2(w[0], w[1]);
}

}  // namespace pka
