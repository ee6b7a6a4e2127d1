// dspark_q8.cuh -- 8-bit floating point helpers shared by the 8-bit cache's kernels
// (sm_103a): conversions between e4m3, half precision and binary32.
#pragma once

#include "../../include/dspark_q8.h"
#include "dspark_common.cuh"

namespace dspark {

// two e4m3 codes (the low byte is `lo`), nearest even; NaN for NaN, 448 past 448
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}
// two half precision numbers as codes
__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(uint32_t v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(v));
  return r;
}
// two codes (of the low half of `codes`) as a pair of half precision numbers: exact
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t v) {
  float2 r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\t"
      "cvt.f32.f16 %1, hi;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(v));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t codes) {
  return f16x2_to_f32(e4m3x2_to_f16x2(codes));
}
// two 16-bit numbers of a word
template <bool F16>
__device__ __forceinline__ float2 word_to_f32(uint32_t w) {
  if constexpr (F16)
    return f16x2_to_f32(w);
  else
    return make_float2(bf16_lo(w), bf16_hi(w));
}
template <bool F16>
__device__ __forceinline__ uint32_t f32_to_word(float lo, float hi) {
  uint32_t r;
  if constexpr (F16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ bool is_scale(float s) { return s > 0.f && s < INFINITY; }

}  // namespace dspark
