// e4m3.cuh -- the codes of an 8-bit cache and their scales.
#pragma once

#include <cfloat>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/svw.h"

namespace svw {

// two codes, lo in the low byte: the nearest, ties to even, +-448 beyond the range, NaN for NaN
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}
// the fp16 values of the two codes in w's low half: exact
__device__ __forceinline__ uint32_t f16x2_of_e4m3(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(w)));
  return r;
}
__device__ __forceinline__ float2 f16x2_f2(uint32_t w) {
  float2 f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(w));
  return f;
}
__device__ __forceinline__ float2 e4m3x2_f2(uint32_t w) { return f16x2_f2(f16x2_of_e4m3(w)); }

// Two numbers of four bits for each of four: the code nearest to x (as fp16),
// and the one nearest to what is left; a's in the low bytes.
__device__ __forceinline__ void split_e4m3x4(float a, float b, float c, float d, uint32_t &first, uint32_t &second) {
  asm("{\n\t.reg .b32 h, r;\n\t.reg .b16 p, q, s, t;\n\t"
      "cvt.rn.f16x2.f32 h, %3, %2;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 p, h;\n\t"
      "cvt.rn.f16x2.e4m3x2 r, p;\n\t"
      "sub.rn.f16x2 h, h, r;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 s, h;\n\t"
      "cvt.rn.f16x2.f32 h, %5, %4;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 q, h;\n\t"
      "cvt.rn.f16x2.e4m3x2 r, q;\n\t"
      "sub.rn.f16x2 h, h, r;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 t, h;\n\t"
      "mov.b32 %0, {p, q};\n\tmov.b32 %1, {s, t};\n\t}"
      : "=r"(first), "=r"(second)
      : "f"(a), "f"(b), "f"(c), "f"(d));
}

// The scale of head h (1 where there are none), NaN where it is not a normal
// number > 0, which the status word is told.
__device__ __forceinline__ float head_scale(const float *scales, int h, int32_t *status) {
  if (!scales) return 1.f;
  const float s = __ldg(scales + h);
  if (s >= FLT_MIN && s <= FLT_MAX) return s;
  if (status) atomicOr(status, SVW_DEV_BAD_INPUT);
  return __int_as_float(0x7fffffff);
}

}  // namespace svw
