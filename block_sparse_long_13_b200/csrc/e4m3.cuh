// e4m3 ("fn") codes: packed conversions and the block scale of the 8-bit K/V cache.
#pragma once
#include "common.cuh"

namespace msa {

constexpr float E4M3_MAX = 448.f;

// two values as e4m3 codes, nearest even, saturated to +-448 (NaN stays NaN); lo in the low byte
__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4_of(float a, float b, float c, float d) {
  return e4m3x2_of(a, b) | (e4m3x2_of(c, d) << 16);
}
// the values of two codes (every e4m3 value is an f16 value)
__device__ __forceinline__ float2 e4m3x2_value(uint32_t codes) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(codes)));
  float2 f;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h2));
  return f;
}
__device__ __forceinline__ void e4m3x4_value(uint32_t codes, float (&x)[4]) {
  const float2 a = e4m3x2_value(codes & 0xFFFFu), b = e4m3x2_value(codes >> 16);
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}

// The least power of two s with 448 s >= a (a >= 0, finite), 2^-126 at least.  A power of two costs no
// precision that a code has (codes are floating point: only the range below 2^-6 s, where their spacing
// stops shrinking, moves by less than one binade) and lets codes of an older, smaller scale be rounded
// again without a second error while they stay normal.  448 = 1.75 * 2^8.
__device__ __forceinline__ float e4m3_block_scale(float a) {
  const uint32_t u = __float_as_uint(a);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(max(e, -126) + 127) << 23);
}

}  // namespace msa
