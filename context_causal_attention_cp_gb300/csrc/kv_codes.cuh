// Arithmetic of the quantised cache's rows: e4m3 codes with a power-of-two scale.
#pragma once
#include <cstdint>

#include <cuda_runtime.h>

namespace cpattn {
namespace {

constexpr int kMinExp = -117, kMaxExp = 119;

// ceil(log2(a / 448)) from the bits of a >= 0: a = m 2^E with m in [1, 2), 448 =
// 1.75 2^8, so it is E - 8, plus one when m > 1.75 (the carry out of the added
// 2^23 - 1 - 0.75 2^23).  A subnormal a comes out below kMinExp.
__device__ __forceinline__ int scale_exponent(float a) {
  const int e = (int)((__float_as_uint(a) + 0x1FFFFFu) >> 23) - 127 - 8;
  return min(max(e, kMinExp), kMaxExp);
}
__device__ __forceinline__ float exp2_int(int e) {  // e in [-126, 127]
  return __uint_as_float((uint32_t)(e + 127) << 23);
}
__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two codes to fp32 (exact: every e4m3 value is an f16).
__device__ __forceinline__ void e4m3x2_to_f32(uint16_t c, float& lo, float& hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
}

}  // namespace
}  // namespace cpattn
