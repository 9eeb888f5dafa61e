// What the kernels of the projection with adapters share: how t is taken up, the MMA with
// both operands in shared memory, and the tensor maps.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "launch.h"
#include "mma.cuh"
#include "pack.cuh"

namespace qmoe {

constexpr int kStageA = 128 * 128;  // bytes of 128 rows x 64 elements
constexpr int kAccCols = 256;       // TMEM columns of one accumulator
constexpr int kSmemLimit = 232448;
// Tokens of a tile.  Up to 240 leave room for five stages of the GEMM's ring, 256 for four:
// taken where all units then run at once (1024 tokens, K = N = 4096, R = 16: 36.3 us, in two
// rounds of 208 38.5; 256 tokens of 64 adapters, K = 1024, N = 16384: 42.0 and 56.6).
constexpr int kMostTokens = kLoraMostTile, kMostInRounds = 240;
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
// Eight elements times t.
template <class T>
__device__ __forceinline__ float dot8(const uint4& raw, const float4& t0, const float4& t1) {
  Pack<T, 8> v;
  v.raw = raw;
  float f = to_f32(v.v[0]) * t0.x;
  f = fmaf(to_f32(v.v[1]), t0.y, f);
  f = fmaf(to_f32(v.v[2]), t0.z, f);
  f = fmaf(to_f32(v.v[3]), t0.w, f);
  f = fmaf(to_f32(v.v[4]), t1.x, f);
  f = fmaf(to_f32(v.v[5]), t1.y, f);
  f = fmaf(to_f32(v.v[6]), t1.z, f);
  return fmaf(to_f32(v.v[7]), t1.w, f);
}

// What two values of T do not hold of a token's t is left to the GEMM's epilogue: its sums over
// the segments, and a bit per eight ranks.  The CTAs of a tile's units all leave the same.
__device__ __forceinline__ void leave_t8(const LoraArgs& p, int tile, int m, int r,
                                         const float (&t)[8]) {
  float4* dst = reinterpret_cast<float4*>(p.tleft + (size_t)m * p.R + r);
  dst[0] = make_float4(t[0], t[1], t[2], t[3]);
  dst[1] = make_float4(t[4], t[5], t[6], t[7]);
  atomicOr(&p.left[m], 1u << (r / 8));
  atomicOr(&p.any_left[tile], 1u);
  __threadfence();
}
__device__ __forceinline__ float max_abs(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}
// Ranks r .. r + 7 of t as their rounding and what that leaves: two values of T whose sum is
// within 2^-16 of the largest of the eight.  bf16 has the range of fp32, so that holds for
// every finite t (up to what rounds to infinity).  fp16 would round 65520 and more to infinity
// and leave minus infinity, and the sum is off by up to 2^-25 (half a subnormal step), so the
// largest has to be 2^-9 or more.  Eight values out of these ranges, infinities and NaN among
// them, enter the MMA as zeros and are left to the epilogue, which tell() tells.
template <class T, class F>
__device__ __forceinline__ void load_t8_split(const LoraArgs& p, int tile, int m, int r, uint4* hi,
                                              uint4* lo, F&& tell) {
  float t[8];
  load_t8(p, m, r, t);
  const float top = max_abs(max_abs(max_abs(t[0], t[1]), max_abs(t[2], t[3])),
                            max_abs(max_abs(t[4], t[5]), max_abs(t[6], t[7])));
  Pack<T, 8> h, l;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    h.v[e] = from_f32<T>(t[e]);
    l.v[e] = from_f32<T>(t[e] - to_f32(h.v[e]));
  }
  *hi = h.raw;
  *lo = l.raw;
  const bool fits = std::is_same<T, __half>::value
                        ? top < 65520.f && (top >= 0x1p-9f || top == 0.f)
                        : top < 0x1.ffp127f;
  if (__builtin_expect(!fits, 0)) {
    *hi = *lo = make_uint4(0u, 0u, 0u, 0u);
    tell();
    leave_t8(p, tile, m, r, t);
  }
}
// ... and its products in fp32 with row n of B: of one token,
template <class T>
__device__ __forceinline__ float left_products(const LoraArgs& p, int m, int n) {
  float f = 0.f;
  unsigned left = __ldcg(&p.left[m]);
  if (left == 0u || n >= p.N) return f;
  const T* b = reinterpret_cast<const T*>(p.b) + ((size_t)p.ids[m] * p.N + n) * p.R;
  const float* t = p.tleft + (size_t)m * p.R;
  for (; left; left &= left - 1) {
    const int r = 8 * (__ffs(left) - 1);
    f += dot8<T>(*reinterpret_cast<const uint4*>(b + r),
                 __ldcg(reinterpret_cast<const float4*>(t + r)),
                 __ldcg(reinterpret_cast<const float4*>(t + r) + 1));
  }
  return f;
}
// and by a warp of `tokens` tokens m0, m0 + 1, .. into v, each lane with a row of its own.  t goes
// through shared memory (buf, 32 tokens' eight values), a token's values by the lane of its
// number; the rows of four tokens' B are in flight together.  (With left_products for one token
// after the other a batch of such tokens took 2370 us where this takes 763: 8192 tokens,
// K = 7168, N = 2048, R = 64.)
template <class T>
__device__ __forceinline__ void add_left(const LoraArgs& p, int m0, int tokens, int n, float4* buf,
                                         float (&v)[32]) {
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const unsigned left = lane < tokens ? __ldcg(&p.left[m0 + lane]) : 0u;
  const int id = left ? p.ids[m0 + lane] : 0;
  // tokens with the adapter of the one before them
  const int before = __shfl_up_sync(kAll, id, 1);
  const unsigned run = __ballot_sync(kAll, lane > 0 && id == before);
  const T* b = reinterpret_cast<const T*>(p.b) + (size_t)min(n, p.N - 1) * p.R;
  for (unsigned units = __reduce_or_sync(kAll, left); units; units &= units - 1) {
    const int r = 8 * (__ffs(units) - 1);
    const unsigned who = __ballot_sync(kAll, left >> (r / 8) & 1u);
    __syncwarp();  // the values before these have been used
    if (who >> lane & 1u) {
      const float4* t = reinterpret_cast<const float4*>(p.tleft + (size_t)(m0 + lane) * p.R + r);
      buf[2 * lane] = __ldcg(t);
      buf[2 * lane + 1] = __ldcg(t + 1);
    }
    __syncwarp();
    uint4 row[4] = {};
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
      if ((run >> k & 15u) == 15u) {
        row[0] = row[1] = row[2] = row[3];
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          row[j] = *reinterpret_cast<const uint4*>(
              b + (size_t)__shfl_sync(kAll, id, k + j) * p.N * p.R + r);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (who >> (k + j) & 1u) v[k + j] += dot8<T>(row[j], buf[2 * (k + j)], buf[2 * (k + j) + 1]);
    }
  }
}

// Infinities and NaN in B.  Through the MMA a row of B meets every token of the tile, those of
// other adapters as zeros, and zero times an infinity is NaN: a row of B that holds one leaves
// every token's sum infinite or NaN there.  So sums that are not finite have the epilogue look
// at the tile's adapters, and what such a row of w spoiled is made anew from x, w and the
// token's own adapter.  Finite weights pay for one comparison a row.
//
// Whether any adapter of the tile has an infinity or NaN in row n of its B.
template <class T>
__device__ __noinline__ bool spoiled_row(const LoraArgs& p, int tile, int n) {
  constexpr uint32_t kExponent = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
  if (n >= p.N) return false;
  bool bad = false;
  const int adapters = p.count[tile];
  for (int d = 0; d < adapters; ++d) {
    const int id = p.list[(size_t)tile * p.tile_n + d];
    const uint4* b = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(p.b) +
                                                    ((size_t)id * p.N + n) * p.R);
#pragma unroll 4
    for (int u = 0; u < p.R / 8; ++u) {
      const uint4 v = b[u];
      const uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        bad |= (word[i] & kExponent) == kExponent || (word[i] >> 16 & kExponent) == kExponent;
    }
  }
  return bad;
}
// t[m] . B[n] of the token's own adapter.
template <class T>
__device__ __noinline__ float own_products(const LoraArgs& p, int m, int n) {
  const int id = p.ids[m];
  float f = 0.f;
  if (id < 0 || id >= p.L) return f;
  const T* b = reinterpret_cast<const T*>(p.b) + ((size_t)id * p.N + n) * p.R;
  for (int r = 0; r < p.R; r += 8) {
    float t[8];
    load_t8(p, m, r, t);
    f += dot8<T>(*reinterpret_cast<const uint4*>(b + r), make_float4(t[0], t[1], t[2], t[3]),
                 make_float4(t[4], t[5], t[6], t[7]));
  }
  return f;
}
// The results of the rows n0 + i, i a bit of `rows`, for the tokens m0, m0 + step, .. (`tokens` of
// them), by a warp: MMAs on fragments straight from memory, 32 rows x 32 tokens at a time.
template <class T>
__device__ __noinline__ void redo_rows(const LoraArgs& p, unsigned rows, int n0, int m0, int step,
                                       int tokens) {
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const long long ldx = step * p.ldx;
  for (int c0 = 0; c0 < tokens; c0 += 32) {
    float acc[2][4][4] = {};  // 16 rows x 8 tokens each
    if (p.w) {
      const T* w = reinterpret_cast<const T*>(p.w) + (size_t)(n0 + g) * p.K + q * 8;
      const T* x = reinterpret_cast<const T*>(p.x) + m0 * p.ldx + (c0 + g) * ldx + q * 8;
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 2
      for (int k = 0; k < p.K; k += 32) {
        const bool in = k + q * 8 < p.K;
        uint4 a[4], b[4];  // rows g, g + 8, .. and tokens g, g + 8, ..
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = b[i] = zero;
          if (in && n0 + g + 8 * i < p.N)
            a[i] = *reinterpret_cast<const uint4*>(w + (size_t)(8 * i) * p.K + k);
          if (in && c0 + g + 8 * i < tokens)
            b[i] = *reinterpret_cast<const uint4*>(x + (8 * i) * ldx + k);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            mma_m16n8k16<T>(acc[i][j], a[2 * i].x, a[2 * i + 1].x, a[2 * i].y, a[2 * i + 1].y,
                            b[j].x, b[j].y);
            mma_m16n8k16<T>(acc[i][j], a[2 * i].z, a[2 * i + 1].z, a[2 * i].w, a[2 * i + 1].w,
                            b[j].z, b[j].w);
          }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = 16 * i + g + 8 * (e >> 1), c = c0 + 8 * j + 2 * q + (e & 1);
          if (!(rows >> row & 1u) || c >= tokens) continue;
          const int m = m0 + c * step, n = n0 + row;
          float f = acc[i][j][e] + own_products<T>(p, m, n);
          if (p.base) f += to_f32(reinterpret_cast<const T*>(p.base)[m * p.ldbase + n]);
          reinterpret_cast<T*>(p.out)[(size_t)m * p.N + n] = from_f32<T>(f);
        }
  }
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
