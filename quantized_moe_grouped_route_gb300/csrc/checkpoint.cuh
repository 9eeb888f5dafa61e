// Activations kept in 8 bits between the passes: a block of 32 neighbouring columns of a row has
// integer codes within 127 and one scale, the least power of two for which they are:
//   x = code * 2^(byte - 127),  code = rint(x * 2^(127 - byte)),  |code| <= 127
// A power of two, so that what is kept is a value of every activation type (7 bits and a sign
// fit the 8 significant bits of bf16): it enters the backward pass's MMAs as it is.  Off by at
// most half a step, 2^-7 to 2^-8 of the block's largest value.  Byte 255: a block with an
// infinity or NaN, all of which becomes NaN.
#pragma once

#include "pack.cuh"

namespace qmoe {

constexpr int kCkBlock = 32;

// A block's scale from the bits of its largest magnitude (infinity and NaN above all numbers).
// 127 * 2^e holds a mantissa of up to 0x7e0000 of the exponent 6 above e.
__device__ __forceinline__ uint32_t ck_byte(uint32_t top) {
  const int b = (int)(top >> 23) - 6 + ((top & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return top >= 0x7f800000u ? 255u : b < 0 ? 0u : (uint32_t)b;
}
// What x is multiplied by (0 for a block that is not finite: its codes are 0).
__device__ __forceinline__ float ck_inverse(uint32_t byte) {
  return byte == 255u ? 0.f : __uint_as_float((254u - byte) << 23);
}
__device__ __forceinline__ float ck_value(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7fc00000u : byte == 0u ? 0x400000u : byte << 23);
}
// (x * inverse of an infinity or NaN is NaN, which converts to 0)
__device__ __forceinline__ int ck_code(float x, float inverse) { return __float2int_rn(x * inverse); }

template <class T>
__device__ __forceinline__ float finite_max();
template <>
__device__ __forceinline__ float finite_max<__nv_bfloat16>() {
  return __uint_as_float(0x7f7f0000u);
}
template <>
__device__ __forceinline__ float finite_max<__half>() {
  return 65504.f;
}
template <>
__device__ __forceinline__ float finite_max<float>() {
  return __uint_as_float(0x7f7fffffu);
}
// v within T's finite range; infinities and NaN stay.
template <class T>
__device__ __forceinline__ float within(float v) {
  const float most = finite_max<T>();
  return fabsf(v) < __uint_as_float(0x7f800000u) ? fminf(fmaxf(v, -most), most) : v;
}
// The value of a code within T's finite range (a block's largest can round up past it).
template <class T>
__device__ __forceinline__ float ck_restore(int code, float value) {
  const float v = (float)code * value, most = finite_max<T>();
  return v > most ? most : v < -most ? -most : v;
}

}  // namespace qmoe
