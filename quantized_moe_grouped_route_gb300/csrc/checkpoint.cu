// Activations to 8 bits and back (checkpoint.cuh has the format).  Both directions are bound by
// memory: 3 bytes an element of a 16-bit type.  A lane has one chunk of 16 bytes of x (of what
// the rows' alignment allows), the lanes of a block of 32 columns find its largest value by
// shuffles, and four chunks a lane are in flight.  8192 x 7168 bf16: there and back 63.5 us, 5.6
// TB/s (84 with a 64-bit division for each chunk's row).
#include <type_traits>

#include "checkpoint.cuh"
#include "common.cuh"
#include "launch.h"

namespace qmoe {
namespace {

constexpr int kThreads = 256;
constexpr int kAtOnce = 4;

template <int N>
struct Codes;
template <>
struct Codes<8> {
  using type = uint2;
};
template <>
struct Codes<4> {
  using type = uint32_t;
};
template <>
struct Codes<2> {
  using type = uint16_t;
};
template <>
struct Codes<1> {
  using type = uint8_t;
};
template <int N>
union CodePack {
  typename Codes<N>::type raw;
  int8_t v[N];
  __device__ CodePack() {}
};

// Row and place in it of unit u of `per` a row: no division where all rows are one.
__device__ __forceinline__ long long row_of(const CheckpointArgs& a, long long u, int per, int* at) {
  if (a.M == 1) {
    *at = (int)u;
    return 0;
  }
  const long long row = u < (1LL << 32) ? (uint32_t)u / (uint32_t)per : u / per;
  *at = (int)(u - row * per);
  return row;
}

// Unit u of work: LANES lanes of block u % blocks of row u / blocks.
template <class T, int VEC>
__global__ void __launch_bounds__(kThreads) pack_kernel(const CheckpointArgs a) {
  constexpr int LANES = kCkBlock / VEC;  // of a block
  const int part = threadIdx.x % LANES;
  const long long units = (long long)a.M * a.blocks;
  const long long per_cta = kThreads / LANES;
  const T* x = reinterpret_cast<const T*>(a.x);
  for (long long u0 = blockIdx.x * per_cta * kAtOnce; u0 < units;
       u0 += gridDim.x * per_cta * kAtOnce) {
    Pack<T, VEC> p[kAtOnce];
    bool in[kAtOnce];
    long long row[kAtOnce];
    int block[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const long long u = u0 + i * per_cta + threadIdx.x / LANES;
      row[i] = row_of(a, u, a.blocks, &block[i]);
      in[i] = u < units && block[i] * kCkBlock + part * VEC < a.C;
      if (in[i])
        p[i].raw = *reinterpret_cast<const typename Pack<T, VEC>::raw_t*>(
            x + row[i] * a.ldx + block[i] * kCkBlock + part * VEC);
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      uint32_t top = 0;
      float f[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        f[e] = in[i] ? to_f32(p[i].v[e]) : 0.f;
        top = max(top, __float_as_uint(f[e]) & 0x7fffffffu);
      }
#pragma unroll
      for (int d = 1; d < LANES; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
      const uint32_t byte = ck_byte(top);
      const float inverse = ck_inverse(byte);
      CodePack<VEC> c;
#pragma unroll
      for (int e = 0; e < VEC; ++e) c.v[e] = (int8_t)ck_code(f[e], inverse);
      if (!in[i]) continue;
      *reinterpret_cast<typename Codes<VEC>::type*>(a.codes + row[i] * a.C + block[i] * kCkBlock +
                                                    part * VEC) = c.raw;
      if (part == 0) a.scales[row[i] * a.blocks + block[i]] = (uint8_t)byte;
    }
  }
}

template <class T, int VEC>
__global__ void __launch_bounds__(kThreads) restore_kernel(const CheckpointArgs a) {
  const int chunks = a.C / VEC;  // VEC divides C
  const long long units = (long long)a.M * chunks;
  T* out = reinterpret_cast<T*>(a.out);
  grid_dep_wait();
  for (long long u0 = blockIdx.x * (long long)kThreads * kAtOnce; u0 < units;
       u0 += gridDim.x * (long long)kThreads * kAtOnce) {
    CodePack<VEC> c[kAtOnce];
    uint32_t byte[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const long long u = u0 + i * kThreads + threadIdx.x;
      if (u >= units) continue;
      int at;
      const long long row = row_of(a, u, chunks, &at);
      c[i].raw = *reinterpret_cast<const typename Codes<VEC>::type*>(a.codes + u * VEC);
      byte[i] = a.scales[row * a.blocks + at / (kCkBlock / VEC)];
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const long long u = u0 + i * kThreads + threadIdx.x;
      if (u >= units) continue;
      const float value = ck_value(byte[i]);
      Pack<T, VEC> p;
#pragma unroll
      for (int e = 0; e < VEC; ++e) p.v[e] = from_f32<T>(ck_restore<T>(c[i].v[e], value));
      *reinterpret_cast<typename Pack<T, VEC>::raw_t*>(out + u * VEC) = p.raw;
    }
  }
}

int grid_of(long long work, int per_cta, int sms) {
  const long long ctas = (work + per_cta - 1) / per_cta, most = (long long)sms * 8;
  return (int)(ctas < most ? ctas : most);
}

template <class T, int VEC>
cudaError_t run(const CheckpointArgs& a, bool restore, int sms, cudaStream_t stream) {
  if (restore) {
    const long long units = (long long)a.M * (a.C / VEC);
    return launch_plain(restore_kernel<T, VEC>, grid_of(units, kThreads * kAtOnce, sms), kThreads,
                        stream, a);
  }
  const long long units = (long long)a.M * a.blocks;
  return launch_plain(pack_kernel<T, VEC>, grid_of(units, kThreads / (kCkBlock / VEC) * kAtOnce, sms),
                      kThreads, stream, a);
}

template <class T>
cudaError_t of_chunk(const CheckpointArgs& a, int chunk, bool restore, int sms,
                     cudaStream_t stream) {
  if (chunk == 1) return run<T, 1>(a, restore, sms, stream);
  if (chunk == 2) return run<T, 2>(a, restore, sms, stream);
  if (std::is_same<T, float>::value || chunk == 4) return run<T, 4>(a, restore, sms, stream);
  if constexpr (sizeof(T) == 2) return run<T, 8>(a, restore, sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_checkpoint(const CheckpointArgs& args, int dtype, int chunk, bool restore, int sms,
                              cudaStream_t stream) {
  CheckpointArgs a = args;
  // rows of whole blocks one behind the other are one row
  if (a.C % kCkBlock == 0 && (restore || a.ldx == a.C) && (long long)a.M * a.C < (1LL << 31)) {
    a.C *= a.M;
    a.blocks *= a.M;
    a.M = 1;
  }
  if (dtype == QMOE_DTYPE_BF16) return of_chunk<__nv_bfloat16>(a, chunk, restore, sms, stream);
  if (dtype == QMOE_DTYPE_FP16) return of_chunk<__half>(a, chunk, restore, sms, stream);
  return of_chunk<float>(a, chunk, restore, sms, stream);
}

}  // namespace qmoe
