// Chunks of consecutive elements: loads, stores and the conversion to and from fp32 of
// the three element types (QMOE_DTYPE_*) the token operators take.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace qmoe {

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}

// Bytes elements of one chunk move as: the unsigned type of that width.
template <int BYTES>
struct Raw;
template <>
struct Raw<16> {
  using type = uint4;
};
template <>
struct Raw<8> {
  using type = uint2;
};
template <>
struct Raw<4> {
  using type = uint32_t;
};
template <>
struct Raw<2> {
  using type = uint16_t;
};

// 16 bytes if `there`, else zeros, without a branch: several such loads are in flight
// together (behind a branch each, the compiler waited for one before it asked for the next:
// 16384 rows of 4096 bf16 added up in 27.7 us, 24.4 so).  Read once: no place in L1.
__device__ __forceinline__ uint4 load_if(const uint4* p, bool there) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
      "@p ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"((int)there));
  return v;
}

// The same for 8 and 4 bytes; neighbouring rows' chunks share sectors, so they may stay in L1.
__device__ __forceinline__ uint2 load_if(const uint2* p, bool there) {
  uint2 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\tmov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\t"
      "@p ld.global.v2.u32 {%0, %1}, [%2];\n\t}"
      : "=&r"(v.x), "=&r"(v.y)
      : "l"(p), "r"((int)there));
  return v;
}
__device__ __forceinline__ uint32_t load_if(const uint32_t* p, bool there) {
  uint32_t v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.u32 %0, 0;\n\t"
      "@p ld.global.u32 %0, [%1];\n\t}"
      : "=&r"(v)
      : "l"(p), "r"((int)there));
  return v;
}

// N consecutive elements of type T, moved in one access.
template <class T, int N>
union Pack {
  static constexpr int kN = N;
  using raw_t = typename Raw<sizeof(T) * N>::type;
  raw_t raw;
  T v[N];
  __device__ Pack() {}
};

}  // namespace qmoe
