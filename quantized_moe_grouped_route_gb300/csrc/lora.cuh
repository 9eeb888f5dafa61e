// What the kernels of the projection with adapters share: how t is taken up, the MMA with
// both operands in shared memory, and the tensor maps.
#pragma once

#include "common.cuh"
#include "launch.h"
#include "pack.cuh"

namespace qmoe {

constexpr int kStageA = 128 * 128;  // bytes of 128 rows x 64 elements
constexpr int kAccCols = 256;       // TMEM columns of one accumulator
constexpr int kSmemLimit = 232448;
// Tokens of a tile.  Up to 240 leave room for five stages of the GEMM's ring, 256 for four:
// taken where all units then run at once (1024 tokens, K = N = 4096, R = 16: 36.3 us, in two
// rounds of 208 38.5; 256 tokens of 64 adapters, K = 1024, N = 16384: 42.0 and 56.6).
constexpr int kMostTokens = 256, kMostInRounds = 240;
constexpr int kShrinkSegments = 8;  // of K in the tensor-core shrink, at most

// Ranks r .. r + 7 of a token's t, over the shrink's segments of K in order.
__device__ __forceinline__ void load_t8(const LoraArgs& p, int m, int r, float (&t)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) t[e] = 0.f;
  const float* src = p.t + (size_t)m * p.R + r;
#pragma unroll 4
  for (int g = 0; g < p.tsplits; ++g) {
    const float4 a = reinterpret_cast<const float4*>(src + (size_t)g * p.M * p.R)[0];
    const float4 b = reinterpret_cast<const float4*>(src + (size_t)g * p.M * p.R)[1];
    t[0] += a.x, t[1] += a.y, t[2] += a.z, t[3] += a.w;
    t[4] += b.x, t[5] += b.y, t[6] += b.z, t[7] += b.w;
  }
}
// ... as their rounding and what that leaves.
template <class T>
__device__ __forceinline__ void load_t8_split(const LoraArgs& p, int m, int r, uint4* hi,
                                              uint4* lo) {
  float t[8];
  load_t8(p, m, r, t);
  Pack<T, 8> h, l;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    h.v[e] = from_f32<T>(t[e]);
    l.v[e] = from_f32<T>(t[e] - to_f32(h.v[e]));
  }
  *hi = h.raw;
  *lo = l.raw;
}

__device__ __forceinline__ void mma_ss(uint32_t cg, uint32_t d, uint64_t a, uint64_t b,
                                       uint32_t idesc, uint32_t accumulate) {
  if (cg == 1)
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, q;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, q;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor, kind::f16: A and B both bf16 or both fp16, fp32 D.
__device__ __forceinline__ uint32_t idesc_16bit(int M, int N, int dtype) {
  return idesc_bf16_f32(M, N) & (dtype == QMOE_DTYPE_BF16 ? ~0u : ~((1u << 7) | (1u << 10)));
}

// Tensor maps: token rows in boxes of `rows`, [N][K] and [L][rows][cols] in boxes of 64
// columns.
inline cudaError_t map_rows(CUtensorMap* map, const LoraArgs& p, const void* base, int cols, int rows,
                     long long ld, int box_rows) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows}, strides[1] = {(uint64_t)ld * 2};
  const uint32_t box[2] = {64, (uint32_t)box_rows};
  return make_tmap16(map, p.dtype, base, 2, dims, strides, box) == QMOE_OK ? cudaSuccess
                                                                           : cudaErrorUnknown;
}
inline cudaError_t map_adapters(CUtensorMap* map, const LoraArgs& p, const void* base, int cols, int rows,
                         int box_rows) {
  const uint64_t dims[3] = {(uint64_t)cols, (uint64_t)rows, (uint64_t)p.L};
  const uint64_t strides[2] = {(uint64_t)cols * 2, (uint64_t)rows * cols * 2};
  const uint32_t box[3] = {64, (uint32_t)box_rows, 1};
  return make_tmap16(map, p.dtype, base, 3, dims, strides, box) == QMOE_OK ? cudaSuccess
                                                                           : cudaErrorUnknown;
}

}  // namespace qmoe
