// fp8.cuh — e4m3 codes (sign, 4 bits of exponent with bias 7, 3 of mantissa;
// steps of 2^-9 below 2^-6, at most ±448, NaN 0x7f, no infinities) to and from
// wider types, for the kernels behind moe_kv8.h.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {

// Two values rounded to nearest even, held at ±448, lo in the lower byte. (As
// cvt has it, infinities too become ±448; NaN stays NaN.)
MOE_DEV uint16_t e4m3_of(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two codes' values; fp16 holds every one.
MOE_DEV __half2 half2_of(uint16_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
  return *reinterpret_cast<__half2*>(&r);
}

// Four values, a and b in the lower half; and four codes' values likewise.
MOE_DEV uint32_t e4m3_of(__half2 a, __half2 b) {
  uint32_t r;
  asm("{\n\t.reg .b16 x, y;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 x, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 y, %2;\n\t"
      "mov.b32 %0, {x, y};\n\t}"
      : "=r"(r)
      : "r"(*reinterpret_cast<uint32_t*>(&a)), "r"(*reinterpret_cast<uint32_t*>(&b)));
  return r;
}
MOE_DEV void halves_of(uint32_t codes, __half2* a, __half2* b) {
  uint32_t x, y;
  asm("{\n\t.reg .b16 u, v;\n\t"
      "mov.b32 {u, v}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, u;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, v;\n\t}"
      : "=r"(x), "=r"(y)
      : "r"(codes));
  *a = *reinterpret_cast<__half2*>(&x);
  *b = *reinterpret_cast<__half2*>(&y);
}

// Four codes' values.
MOE_DEV float4 floats_of(uint32_t codes) {
  const float2 a = __half22float2(half2_of((uint16_t)codes));
  const float2 b = __half22float2(half2_of((uint16_t)(codes >> 16)));
  return make_float4(a.x, a.y, b.x, b.y);
}

// 2^e for −126 ≤ e ≤ 127.
MOE_DEV float pow2(int e) { return __int_as_float((e + 127) << 23); }

}  // namespace moe
