// quant.cuh -- the 8-bit rows of a quantised cache: e4m3 codes under one power of two (e8m0).
//
// A row x is held as codes c and a scale 2^e, e the smallest integer of -15 .. 8 with
// max |x| <= 448 * 2^e, c the e4m3 number nearest to x / 2^e (ties to even), at most 448 in size, or
// 240 for e = 8. Then c * 2^e is always a finite fp16 number (a multiple of 2^-24, at most 61440),
// so every kernel that reads a row works on exactly its value in the tensor cores' fp16.
// e4m3 keeps its 4 significant bits over a range of 2^15 below a row's largest element: one scale a
// row is enough, and a power of two costs nothing in a floating format.
#pragma once

#include "device_common.cuh"
#include "internal.h"

namespace pa {

constexpr int kScaleBias = 127;  // a scale's byte is e + 127
constexpr int kMinExp = -15, kMaxExp = 8;

// Place of the scale of (page, K/V head, slot): [page][kv_head][slot] whatever the codes' layout, so
// that a head's scales of a page lie side by side.
__device__ __forceinline__ long long scale_place(int page, int kv, int slot, int kvh, int ps) {
  return (static_cast<long long>(page) * kvh + kv) * ps + slot;
}

// The exponent of a row whose largest magnitude is `top`: a mantissa above 1.75 = 448 / 2^8 carries.
__device__ __forceinline__ int row_exponent(float top) {
  const int e = static_cast<int>((__float_as_uint(top) + 0x1fffffu) >> 23) - 127 - 8;
  return min(max(e, kMinExp), kMaxExp);
}

// Two values (of rows scaled by 2^-e) as codes, the first in the low byte.
__device__ __forceinline__ uint32_t code2(float x, float y) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(y), "f"(x));
  return c;
}

__device__ __forceinline__ void pack_codes(const float (&y)[16], uint32_t (&w)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = code2(y[4 * i], y[4 * i + 1]) | code2(y[4 * i + 2], y[4 * i + 3]) << 16;
}

// 16 values of a row as codes, four to a word.
__device__ __forceinline__ void codes16(const float (&x)[16], int e, uint32_t (&w)[4]) {
  const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  float y[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = x[i] * f;
  if (e == kMaxExp) {
    // 448 * 2^8 is no fp16 number: the largest value is 240 * 2^8 (NaN stays NaN)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      asm("{\n\t.reg .f32 t;\n\tmin.NaN.f32 t, %0, %1;\n\tmax.NaN.f32 %0, t, %2;\n\t}"
          : "+f"(y[i])
          : "f"(240.f), "f"(-240.f));
  }
  pack_codes(y, w);
}

// Codes to fp16: the low and the high two of a word.
__device__ __forceinline__ uint32_t half2_of_low(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}

__device__ __forceinline__ uint32_t half2_of_high(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}

__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// 2^e of a scale byte, as an fp16 pair; anything for a byte that is no scale.
__device__ __forceinline__ uint32_t half2_of_scale(uint32_t b) {
  const float x = __uint_as_float(b << 23);
  return pack_half2(x, x);
}

// 2^e of two scale bytes, as an fp16 pair. Bytes that no row was written with (tokens that nobody
// sees) give a finite factor too.
__device__ __forceinline__ uint32_t half2_of_scales(uint32_t b0, uint32_t b1) {
  constexpr uint32_t top = kScaleBias + kMaxExp;
  const float x = __uint_as_float(min(b0, top) << 23), y = __uint_as_float(min(b1, top) << 23);
  return pack_half2(x, y);
}

}  // namespace pa
