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

// How rows come in: straight from memory; through shared memory, `depth` rows deep, so that the
// loads of the next rows run while a row waits for its sums, each thread copying the chunks that it
// will use itself (no thread waits for another's copies); or, where rows lie on odd 2-byte
// boundaries that cp.async does not take, as aligned 16-byte pieces that a row's threads share.
// (A piece may begin before its row: in the same 16 bytes, so in the same allocation.)
enum class In { kDirect, kOwn, kShared };

// Up to N matrices of which some are there; place of a row [stage][matrix][..].
template <class T, int VEC, int NCH, In HOW, int N>
struct RowsIn {
  using raw_t = typename Pack<T, VEC>::raw_t;
  static constexpr int kBytes = sizeof(T) * VEC;
  const void* source[N];  // NULL: not there
  long long apart[N];     // elements between rows
  int M, H, units, depth, mats;
  uint32_t base;  // kOwn: this thread's first place; kShared: of the threads of its row
  int stride;     // kOwn: bytes between a thread's places; kShared: bytes of a matrix' row
  int tid, threads;
  bool one_warp;
  int stage = 0;
  uint32_t place[N];         // this thread's first chunk of the row in shared memory,
  Pack<T, VEC> raw[N][NCH];  // or its chunks

  __device__ __forceinline__ const T* at(int i, int row) const {
    return reinterpret_cast<const T*>(source[i]) + row * apart[i];
  }
  // of a stage
  __device__ __forceinline__ uint32_t matrix_bytes() const {
    return HOW == In::kOwn ? NCH * stride : stride;
  }
  __device__ __forceinline__ void copy16(uint32_t to, const void* from, int bytes) const {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes)
                 : "memory");
  }
  __device__ __forceinline__ void start(int row, int to, const int (&col)[NCH],
                                        const bool (&in)[NCH]) const {
    if (row < M) {
      uint32_t into = base + to * mats * matrix_bytes();
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (!source[i]) continue;
        if constexpr (HOW == In::kOwn) {
#pragma unroll
          for (int k = 0; k < NCH; ++k) {
            const T* from = at(i, row) + (in[k] ? col[k] : 0);
            if constexpr (kBytes == 16)
              copy16(into + k * stride, from, in[k] ? 16 : 0);
            else if constexpr (kBytes >= 4)
              asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(into + k * stride),
                           "l"(from), "n"(kBytes), "r"(in[k] ? kBytes : 0)
                           : "memory");
          }
        } else {
          const uintptr_t begin = reinterpret_cast<uintptr_t>(at(i, row));
          const uintptr_t end = begin + H * sizeof(T), low = begin & ~(uintptr_t)15;
          for (uintptr_t j = low + 16 * tid; j < end; j += 16 * threads)
            copy16(into + (uint32_t)(j - low), reinterpret_cast<const void*>(j),
                   (int)min((uintptr_t)16, end - j));
        }
        into += matrix_bytes();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // All but the newest n groups of this thread's copies are there.
  __device__ __forceinline__ static void wait(int n) {
    if (n >= 3)
      asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (n == 2)
      asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (n == 1)
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
      asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  __device__ __forceinline__ void begin(int unit, const int (&col)[NCH], const bool (&in)[NCH]) {
    if constexpr (HOW != In::kDirect)
      for (int i = 0; i + 1 < depth; ++i) start(unit + i * units, i, col, in);
  }
  // Chunk k of this thread's in matrix m of the row; what is not there, and all that lies behind
  // the row's end, is 0.  (Read from shared memory each time it is used, not kept: there are few
  // registers beside the sums', and with the rows in shared memory L1 is too small for spills.)
  __device__ __forceinline__ void chunk(int m, int k, const bool (&in)[NCH], float (&f)[VEC]) const {
    Pack<T, VEC> v;
    if constexpr (HOW == In::kDirect) {
      v = raw[m][k];
    } else if constexpr (HOW == In::kOwn) {
      v.raw = raw_t{};
      if (source[m]) {
        const uint32_t from = place[m] + k * stride;
        if constexpr (kBytes == 16)
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v.raw.x), "=r"(v.raw.y), "=r"(v.raw.z), "=r"(v.raw.w)
                       : "r"(from)
                       : "memory");
        else if constexpr (kBytes == 4)
          asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v.raw) : "r"(from) : "memory");
      }
    } else {
      uint16_t r = 0;
      if (in[k] && source[m])
        asm volatile("ld.shared.u16 %0, [%1];"
                     : "=h"(r)
                     : "r"(place[m] + k * threads * (uint32_t)sizeof(T))
                     : "memory");
      if constexpr (kBytes == 2) v.raw = r;
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = to_f32(v.v[e]);
  }
  __device__ __forceinline__ void begin_zero() {
    if constexpr (HOW == In::kDirect)
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int k = 0; k < NCH; ++k) raw[i][k].raw = raw_t{};
  }
  // A row comes in; the row depth - 1 further on is asked for.
  __device__ __forceinline__ void next(int row, const int (&col)[NCH], const bool (&in)[NCH]) {
    const int free = stage == 0 ? depth - 1 : stage - 1;  // of the row before this one
    if constexpr (HOW == In::kOwn) {
      start(row + (depth - 1) * units, free, col, in);  // this thread has used its places
      wait(depth - 1);
    } else if constexpr (HOW == In::kShared) {
      wait(depth - 2);
      if (one_warp)
        __syncwarp();
      else
        __syncthreads();  // everybody's pieces are there, and the row before has been read
      start(row + (depth - 1) * units, free, col, in);
    }
    uint32_t of_stage = base + stage * mats * matrix_bytes();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      place[i] = of_stage;
      if (!source[i]) continue;
      if constexpr (HOW == In::kDirect) {
#pragma unroll
        for (int k = 0; k < NCH; ++k)
          raw[i][k].raw =
              load_if(reinterpret_cast<const raw_t*>(at(i, row) + (in[k] ? col[k] : 0)), in[k]);
      } else if constexpr (HOW == In::kShared) {
        place[i] += (uint32_t)(reinterpret_cast<uintptr_t>(at(i, row)) & 15) +
                    tid * (uint32_t)sizeof(T);
      }
      of_stage += matrix_bytes();
    }
    if (HOW != In::kDirect && ++stage == depth) stage = 0;
  }
};
// Bytes of shared memory that a stage of a CTA's rows takes.
template <class T, int VEC, In HOW>
inline int stage_bytes(int mats, int threads, int rows, int elements, int H) {
  return HOW == In::kOwn ? mats * threads * rows * elements * (int)sizeof(T)
                         : mats * rows * ((H * (int)sizeof(T) + 30) / 16 * 16);
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

// The gate's value, and its value and derivative in what is given.
__device__ __forceinline__ float gate_value(const NormArgs& a, float g) {
  return a.gating == QMOE_GATING_SIGMOID ? 1.f / (1.f + expf(-g)) : g;
}
// A sigmoid s(g)'s derivative is s(g) s(-g), and s(-g) = e^-g s(g): above 0, where 1 - s(g) loses its
// digits, by that product.
__device__ __forceinline__ float gate_parts(const NormArgs& a, float g, float* slope) {
  *slope = 1.f;
  if (a.gating != QMOE_GATING_SIGMOID) return g;
  const float e = expf(-g), s = 1.f / (1.f + e);
  *slope = s * (g > 0.f ? e * s : 1.f - s);
  return s;
}

// Vectors over a row's columns (weights, a channel's gate) that each thread keeps for its own
// columns in shared memory, as fp32: there they outlast the rows, which would push them out of L1.
// Place [vector][chunk][4 elements][thread].
template <int VEC, int NCH>
struct Vectors {
  static constexpr int kPart = VEC < 4 ? VEC : 4, kParts = VEC / kPart;
  uint8_t* base;  // this thread's first place
  int stride;     // bytes between a thread's places
  __device__ __forceinline__ float* place(int vec, int k, int part) const {
    return reinterpret_cast<float*>(base + ((vec * NCH + k) * kParts + part) * stride);
  }
  __device__ __forceinline__ void put(int vec, int k, const float (&f)[VEC]) const {
#pragma unroll
    for (int i = 0; i < VEC; ++i) place(vec, k, i / kPart)[i % kPart] = f[i];
  }
  __device__ __forceinline__ void get(int vec, int k, float (&f)[VEC]) const {
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      Pack<float, kPart> v;
      v.raw = *reinterpret_cast<const typename Pack<float, kPart>::raw_t*>(place(vec, k, i));
#pragma unroll
      for (int e = 0; e < kPart; ++e) f[i * kPart + e] = v.v[e];
    }
  }
};
// Bytes of them a thread.
__host__ __device__ constexpr int vector_bytes(int vectors, int elements) {
  return vectors * elements * 4;
}

template <class K, class... Args>
cudaError_t launch_pdl(K* kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream,
                   Args... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Threads of a row whose threads hold `elements` each, in chunks of vec elements.
__host__ __device__ constexpr int norm_threads(int H, int vec, int elements) {
  const int chunks = (H + vec - 1) / vec, per = elements / vec;
  return ((chunks + per - 1) / per + 31) / 32 * 32;
}
// Rows of a CTA: four warps with a row each, or all threads on one.
__host__ __device__ constexpr int norm_rows(int threads) { return threads == 32 ? 4 : 1; }

}  // namespace qmoe
