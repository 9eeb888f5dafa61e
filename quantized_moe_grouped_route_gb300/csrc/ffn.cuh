// What the kernels of the gated feed-forward block share: the activation and its derivative, and
// the arithmetic of the gate, the clamp and the product.
#pragma once

#include "common.cuh"
#include "launch.h"
#include "pack.cuh"

namespace qmoe {

// Both activations are g * sigmoid(k(g)): SiLU with k(g) = g, GELU in its tanh form with
// k(g) = 2 sqrt(2 / pi) (g + 0.044715 g^3), since (1 + tanh z) / 2 = sigmoid(2 z).  expf's
// approximation is documented as off by 2 + 1.173 |k| units in the last place (2^-23) and k is
// by a few of its own, so the sigmoid by some (8 + 4 |k|) 2^-23, relative: below the half step of bf16
// (2^-8) or fp16 (2^-11) by which h is rounded anyway for every |k| up to 1000, far beyond those at
// which the sigmoid is another number than 0 and 1.
constexpr float kGeluA = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

__device__ __forceinline__ float sigmoid_fast(float k) { return __fdividef(1.f, 1.f + __expf(-k)); }

// sigmoid(k(g)) and k'(g).  (Past 64 the sigmoid is 0 or 1: g^3 need not overflow.  NaN stays.)
template <bool SLOPE>
__device__ __forceinline__ void act_parts(bool gelu, float g, float* p, float* slope) {
  if (gelu) {
    const float c = g > 64.f ? 64.f : g < -64.f ? -64.f : g, c2 = c * c;
    *p = sigmoid_fast(kGeluA * c * fmaf(kGeluB, c2, 1.f));
    if (SLOPE) *slope = kGeluA * fmaf(3.f * kGeluB, c2, 1.f);
  } else {
    *p = sigmoid_fast(g);
    if (SLOPE) *slope = 1.f;
  }
}

// h = act(min(g, limit)) * clamp(u, -limit, limit); comparisons that leave NaN as it is.
__device__ __forceinline__ float gated(bool gelu, float limit, float u, float g) {
  float p, unused;
  g = g > limit ? limit : g;
  u = u > limit ? limit : u < -limit ? -limit : u;
  act_parts<false>(gelu, g, &p, &unused);
  return g * p * u;
}
// ... and its derivatives' products with dh; what the clamp holds has none.
__device__ __forceinline__ float gated_backward(bool gelu, float limit, float u, float g, float dh,
                                                float* du, float* dg) {
  float p, slope;
  const bool free_g = !(g > limit), free_u = !(fabsf(u) > limit);  // (NaN is not held)
  g = g > limit ? limit : g;
  u = u > limit ? limit : u < -limit ? -limit : u;
  act_parts<true>(gelu, g, &p, &slope);
  const float a = g * p;
  *du = free_u ? dh * a : 0.f;
  *dg = free_g ? dh * u * fmaf(a * (1.f - p), slope, p) : 0.f;
  return a * u;
}

// Tensor map of an operand [rows][cols], rows ld elements apart, in boxes of 64 columns.
inline bool map_of(CUtensorMap* map, int dtype, const void* base, long long rows, int cols,
                   long long ld, int box_rows) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows}, strides[1] = {(uint64_t)ld * 2};
  const uint32_t box[2] = {64, (uint32_t)box_rows};
  return make_tmap16(map, dtype, base, 2, dims, strides, box) == QMOE_OK;
}

}  // namespace qmoe
