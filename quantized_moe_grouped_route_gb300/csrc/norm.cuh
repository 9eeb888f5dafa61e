// What the forward and backward kernels of the norms around a block share (norm.cu).
#pragma once

#include "common.cuh"
#include "launch.h"
#include "pack.cuh"

namespace qmoe {

__device__ __forceinline__ uint16_t load_if(const uint16_t* p, bool there) {
  uint16_t v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.u16 %0, 0;\n\t"
      "@p ld.global.u16 %0, [%1];\n\t}"
      : "=&h"(v)
      : "l"(p), "r"((int)there));
  return v;
}

// N elements of T that start at element `at` as fp32, from a pointer whose alignment fits N.
template <class T, int N>
__device__ __forceinline__ void load_as_f32(const void* p, long long at, float (&f)[N]) {
  constexpr int kMost = 16 / (int)sizeof(T), kStep = N < kMost ? N : kMost;
#pragma unroll
  for (int i = 0; i < N; i += kStep) {
    Pack<T, kStep> v;
    v.raw = *reinterpret_cast<const typename Pack<T, kStep>::raw_t*>(
        reinterpret_cast<const T*>(p) + at + i);
#pragma unroll
    for (int e = 0; e < kStep; ++e) f[i + e] = to_f32(v.v[e]);
  }
}
// ... of the activations' type or fp32: a weight's or a gate's elements
template <class T, int N>
__device__ __forceinline__ void load_either(const void* p, bool fp32, long long at, float (&f)[N]) {
  if (fp32)
    load_as_f32<float, N>(p, at, f);
  else
    load_as_f32<T, N>(p, at, f);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// Sums over the threads of a row: a warp, or the whole CTA through shared memory.  Two buffers
// in turn: whoever writes one again has met everybody at the other's barrier since.
struct RowSum {
  float* buf;  // [2][32]
  int warps;   // of a row
  int turn = 0;
  __device__ __forceinline__ float operator()(float v) {
    v = warp_sum(v);
    if (warps == 1) return v;
    float* s = buf + 32 * turn;
    turn ^= 1;
    const int lane = threadIdx.x & 31;
    if (lane == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(lane < warps ? s[lane] : 0.f);
  }
};

// The gate's value and its derivative in what is given.
__device__ __forceinline__ float gate_value(const NormArgs& a, float g) {
  return a.gating == QMOE_GATING_SIGMOID ? 1.f / (1.f + expf(-g)) : g;
}
__device__ __forceinline__ float gate_slope(const NormArgs& a, float value) {
  return a.gating == QMOE_GATING_SIGMOID ? value * (1.f - value) : 1.f;
}

// Threads of a row whose threads hold `elements` each, in chunks of vec elements.
__host__ __device__ constexpr int norm_threads(int H, int vec, int elements) {
  const int chunks = (H + vec - 1) / vec, per = elements / vec;
  return ((chunks + per - 1) / per + 31) / 32 * 32;
}
// Rows of a CTA: four warps with a row each, or all threads on one.
__host__ __device__ constexpr int norm_rows(int threads) { return threads == 32 ? 4 : 1; }

}  // namespace qmoe
