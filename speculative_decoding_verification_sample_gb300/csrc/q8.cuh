// The 8-bit cache format: e4m3 codes and power-of-two block scales.
#pragma once
#include <cstdint>

namespace sv {

constexpr int kQ8MinExp = -100;  // smallest scale 2^-100: it and its inverse stay normal

// e with 2^e the smallest power of two (at least 2^kQ8MinExp) such that
// amax <= 448 * 2^e, 448 = 1.75 * 2^8 the largest e4m3 number. amax finite.
__device__ __forceinline__ int q8_scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  // amax = m 2^x with 1 <= m < 2; a subnormal amax is below the smallest scale
  const int e = int(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < kQ8MinExp ? kQ8MinExp : e;
}
__device__ __forceinline__ float q8_pow2(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// Four codes (lowest byte first) to fp32, exact.
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t c, float* f) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(c));
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f[0]), "=f"(f[1])
      : "r"(lo));
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f[2]), "=f"(f[3])
      : "r"(hi));
}

// Four numbers to e4m3, to nearest even, saturating; the first in the lowest byte.
__device__ __forceinline__ uint32_t f32x4_to_e4m3(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// Two fp16 numbers to two codes and back (in the lower 16 bits), to nearest even,
// saturating.
__device__ __forceinline__ uint32_t f16x2_to_e4m3(uint32_t v) {
  uint32_t r;
  asm("{\n\t.reg .b16 c;\n\tcvt.rn.satfinite.e4m3x2.f16x2 c, %1;\n\tcvt.u32.u16 %0, c;\n\t}"
      : "=r"(r)
      : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t c) {
  uint32_t r;
  asm("{\n\t.reg .b16 x;\n\tcvt.u16.u32 x, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\t}"
      : "=r"(r)
      : "r"(c));
  return r;
}

}  // namespace sv
