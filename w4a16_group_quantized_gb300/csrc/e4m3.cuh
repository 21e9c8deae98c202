// Codes of 8 bits: e4m3 (4 bits of exponent, 3 of fraction, largest value 448, no infinity, 0x7F and 0xFF are NaN).
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

namespace w4 {
namespace detail {

// Two codes (the low one first) as two fp16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t codes) {
  uint32_t v;
  asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(v) : "r"(codes));
  return v;
}

// Four codes as two pairs of fp16 values.
__device__ __forceinline__ void e4m3x4_f16x4(uint32_t codes, uint32_t *lo, uint32_t *hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(*lo), "=r"(*hi)
      : "r"(codes));
}

// Two values rounded to codes, nearest even; |v| <= 448, or NaN.
__device__ __forceinline__ uint32_t f32_e4m3x2(float lo, float hi) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
  return c;
}

}  // namespace detail
}  // namespace w4
