// 8-bit activation checkpoints: 64 channels of a row share a scale 2^k, and a
// value x is held as the e4m3 value nearest x / 2^k.  The scale is a power of
// two, so dividing by it is exact and the only rounding is e4m3's own; k is
// the least integer (≥ −126, which keeps 2^k and 2^-k normal) for which the
// group's largest finite |x| is at most 448 · 2^k, e4m3's largest value.
#pragma once

#include <cuda_runtime.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "common.cuh"
#include "r2l.h"

namespace r2l {
namespace act8 {

constexpr int GROUP = R2L_ACT8_GROUP;

// |v| as bits, 0 for an infinity or a NaN: the ordering of the bits is that of
// the values, so a group's maximum is an integer maximum.
__device__ __forceinline__ uint32_t finite_abs_bits(float v) {
  const uint32_t u = __float_as_uint(v) & 0x7fffffffu;
  return u < 0x7f800000u ? u : 0u;
}

// k + 127 of a group whose largest finite magnitude has these bits: with
// max = m · 2^e, 1 ≤ m < 2, it is e − 8 when m ≤ 1.75 (448 = 1.75 · 2^8) and
// e − 7 otherwise.
__device__ __forceinline__ uint32_t scale_byte(uint32_t max_bits) {
  const int e = (int)((max_bits + 0x1fffffu) >> 23);   // the exponent, one more where m > 1.75
  return (uint32_t)max(e - 8, 1);
}

__device__ __forceinline__ float scale_up(uint32_t byte) { return __uint_as_float(byte << 23); }            // 2^k
__device__ __forceinline__ float scale_down(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }  // 2^-k

// What is held of v: NaN for an infinity or a NaN (e4m3 has no infinity, and the
// conversion below would turn one into ±448), and ±240 · 2^120 for finite values
// from 248 · 2^120 on (the bits SPECIAL), which would be rounded to 2^128 and come
// back as infinities.  Any other v as it is (its e4m3 value, that is): a group
// without these two kinds needs no call.
constexpr uint32_t SPECIAL = 0x7f780000u;
__device__ __forceinline__ float storable(float v) {
  return fminf(fmaxf(v, -240.0f * 0x1p120f), 240.0f * 0x1p120f) + (v - v);
}

// Two e4m3 bytes, `lo` in the low one, from values already divided by the scale.
__device__ __forceinline__ uint16_t to_e4m3x2(float lo, float hi) {
  uint16_t q;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(q) : "f"(hi), "f"(lo));
  return q;
}

__device__ __forceinline__ float2 from_e4m3x2(uint16_t q) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(q));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace act8
}  // namespace r2l
