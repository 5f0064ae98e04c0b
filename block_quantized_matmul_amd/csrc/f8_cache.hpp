// Codes and scales of the 8-bit paged cache (kv_append_norm.hip,
// kv_read_f8.hip, attn_f8.hip); gfx950 only.
//
// Each token's vector of one head is D e4m3 codes and one power of two, held as
// the byte exponent + 127. A block of one token, so that an append never
// touches what other tokens' codes stand for: with a scale shared by several
// tokens a later, larger token rescales the earlier ones, which two writers of
// one block cannot do at once, makes the codes depend on the history, and
// changes a page under the conversations that share it. A power of two, because
// a float code loses nothing by it and the conversions of codes to 16 bits apply
// it for nothing.
#pragma once

#include "serve_device.hpp"

namespace lqmm {

constexpr float kCodeMax = 448.0f;  // largest e4m3 value, 1.75 * 2^8
// Scales are 2^-60 .. 2^60: sums of 2^13 values stay in fp32's range. In fp16 the
// largest is 2^7, whose largest code stands for 57344; attention's 16-row kernel
// divides weights by V's scales, and those lie 2^67 apart then.
constexpr int kLeastScale = 127 - 60;
constexpr int kMostScaleF16 = 127 + 7, kMostScaleBF16 = 127 + 60;

// The scale byte of a vector whose largest magnitude is `top`: the least e with
// top <= 448 2^e. From top's bits: its fraction is over 1.75 exactly when adding
// 0x1fffff carries into the exponent.
__device__ __forceinline__ int scale_byte(float top, int most) {
  const int b = (int)((__builtin_bit_cast(uint32_t, top) + 0x1fffffu) >> 23) - 8;
  return b < kLeastScale ? kLeastScale : b > most ? most : b;
}
// 2^(byte - 127) and its inverse, for bytes 1 .. 253.
__device__ __forceinline__ float scale_of(uint32_t byte) { return __builtin_bit_cast(float, byte << 23); }
__device__ __forceinline__ float scale_inverse(uint32_t byte) {
  return __builtin_bit_cast(float, (254u - byte) << 23);
}

// Eight values times `mul` as e4m3 codes (nearest even; NaN to NaN).
__device__ __forceinline__ u32x2 codes8(const float (&x)[8], float mul) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i] * mul, x[4 * i + 1] * mul, 0, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i + 2] * mul, x[4 * i + 3] * mul, v, true);
    w[i] = (uint32_t)v;
  }
  return u32x2{w[0], w[1]};
}

// Eight codes as 16-bit values times `scale` (a power of two), each rounded
// once: exact but for fp16 values below 2^-14 (steps of 2^-24).
template <class T>
__device__ __forceinline__ typename T::vec8 values8(u32x2 c, float scale) {
  typename T::vec8 v;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (__is_same(T, TypeF16)) {
      const half2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)c[i], scale, false);
      const half2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)c[i], scale, true);
      v[4 * i] = a[0], v[4 * i + 1] = a[1], v[4 * i + 2] = b[0], v[4 * i + 3] = b[1];
    } else {
      const auto a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)c[i], scale, false);
      const auto b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)c[i], scale, true);
      v[4 * i] = a[0], v[4 * i + 1] = a[1], v[4 * i + 2] = b[0], v[4 * i + 3] = b[1];
    }
  }
  return v;
}
// Eight codes as fp16 values, each times a power of two of its own.
__device__ __forceinline__ half8_t values8_each(u32x2 c, const float (&scale)[8]) {
  half8_t v;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    half2_t a = {0, 0}, b = {0, 0};
    a = __builtin_amdgcn_cvt_scalef32_f16_fp8(a, (int)c[i], scale[4 * i], 0, false);
    a = __builtin_amdgcn_cvt_scalef32_f16_fp8(a, (int)c[i], scale[4 * i + 1], 1, true);
    b = __builtin_amdgcn_cvt_scalef32_f16_fp8(b, (int)c[i], scale[4 * i + 2], 2, false);
    b = __builtin_amdgcn_cvt_scalef32_f16_fp8(b, (int)c[i], scale[4 * i + 3], 3, true);
    v[4 * i] = a[0], v[4 * i + 1] = a[1], v[4 * i + 2] = b[0], v[4 * i + 3] = b[1];
  }
  return v;
}
// Eight codes as fp32 values.
__device__ __forceinline__ void values8(u32x2 c, float scale, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], false);
    const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], true);
    x[4 * i] = a[0] * scale, x[4 * i + 1] = a[1] * scale;
    x[4 * i + 2] = b[0] * scale, x[4 * i + 3] = b[1] * scale;
  }
}

}  // namespace lqmm
