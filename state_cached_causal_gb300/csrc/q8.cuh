// Rows of a cache in 8 bits: e4m3 values and a power of two a row.
#pragma once

#include "mixer.cuh"

namespace cconv {

inline int mix_check_cache_q8(const kv_cache_q8_t& c) {
  if (!c.k || !c.v || !mix_aligned16(c.k) || !mix_aligned16(c.v) || !c.k_scale || !c.v_scale)
    return CCONV_ERR_INVALID;
  if (c.num_pages <= 0 || c.page_size <= 0 || c.num_kv_heads <= 0 || c.head_dim <= 0)
    return CCONV_ERR_INVALID;
  if (c.s_page <= 0 || c.s_token <= 0 || c.s_head <= 0 || c.s_page % 16 || c.s_token % 16 ||
      c.s_head % 16 || c.c_page <= 0 || c.c_token <= 0 || c.c_head <= 0)
    return CCONV_ERR_INVALID;
  if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return CCONV_ERR_UNSUPPORTED;
  return CCONV_OK;
}

// Two values to e4m3 (nearest even; NaN stays NaN), x0 in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3x2(float x0, float x1) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(x1), "f"(x0));
  return r;
}
__device__ __forceinline__ uint32_t pack_e4m3x4(float x0, float x1, float x2, float x3) {
  return pack_e4m3x2(x0, x1) | pack_e4m3x2(x2, x3) << 16;
}
// Two e4m3 values (the low 16 bits) as fp16, which holds them all.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
  return r;
}
__device__ __forceinline__ void f16x2_to_f32(uint32_t v, float& x0, float& x1) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(x0), "=f"(x1)
      : "r"(v));
}
__device__ __forceinline__ void unpack_e4m3x4(uint32_t v, float (&f)[4]) {
  f16x2_to_f32(e4m3x2_to_f16x2(v), f[0], f[1]);
  f16x2_to_f32(e4m3x2_to_f16x2(v >> 16), f[2], f[3]);
}

// What a scale byte stands for.
__device__ __forceinline__ float q8_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// The scale byte of a row whose largest finite magnitude is m, and the factor
// 2^-e of its values: e least with m <= 448 * 2^e = 1.75 * 2^(8 + e).
__device__ __forceinline__ uint32_t q8_byte(float m) {
  const uint32_t bits = __float_as_uint(m);
  const int up = (bits & 0x7fffffu) > 0x600000u;
  return (uint32_t)max((int)(bits >> 23) - 8 + up, 1);
}
__device__ __forceinline__ float q8_factor(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}
// A value as it is rounded: infinities as NaN.
__device__ __forceinline__ float q8_in(float x) {
  return fabsf(x) == __uint_as_float(0x7f800000u) ? __uint_as_float(0x7fc00000u) : x;
}

// Rows of this byte hold values that would be rounded to 2^128: they become the largest
// one below that, 240 * 2^120.
constexpr uint32_t kQ8Top = 127 + 120;
__device__ __forceinline__ float q8_top(float x) {
  const float top = __uint_as_float(0x7f700000u);
  return x > top ? top : x < -top ? -top : x;
}

}  // namespace cconv
