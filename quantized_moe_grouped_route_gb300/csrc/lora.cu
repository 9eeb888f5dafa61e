// A shared projection with a low-rank adapter per token:
//   t[m] = scales[a] * (x[m] . A[a]^T),  out[m] = base[m] + x[m] . w^T + t[m] . B[a]^T
// with a = adapter_ids[m]; sums in fp32, one rounding at the end.
#include "common.cuh"
#include "launch.h"
#include "pack.cuh"

namespace qmoe {
namespace {

// A warp per (token, rank).
template <class T>
__global__ void lora_shrink_kernel(const LoraArgs p) {
  grid_dep_wait();
  grid_dep_launch();
  if (blockIdx.x == 0 && threadIdx.x == 0) p.err[0] = 0u;
  const int lane = threadIdx.x & 31;
  const long long items = (long long)p.M * p.R;
  for (long long it = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5; it < items;
       it += ((long long)gridDim.x * blockDim.x) >> 5) {
    const int m = (int)(it / p.R), r = (int)(it % p.R);
    const int id = p.ids[m];
    float acc = 0.f;
    if (id >= 0 && id < p.L) {
      const T* x = reinterpret_cast<const T*>(p.x) + m * p.ldx;
      const T* a = reinterpret_cast<const T*>(p.a) + ((size_t)id * p.R + r) * p.K;
      for (int k = lane; k < p.K; k += 32) acc = fmaf(to_f32(x[k]), to_f32(a[k]), acc);
#pragma unroll
      for (int o = 16; o; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
      acc *= p.scales[id];
    }
    if (lane == 0) p.t[it] = acc;
  }
}

// 64 tokens x 64 outputs per block of 256 threads, 4 x 4 a thread.
template <class T>
__global__ void __launch_bounds__(256) lora_expand_kernel(const LoraArgs p) {
  __shared__ float xs[16][65], ws[16][65];
  grid_dep_wait();
  grid_dep_launch();
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
  const int tm = threadIdx.x / 16, tn = threadIdx.x % 16;
  float acc[4][4] = {};
  if (p.w) {
    for (int k0 = 0; k0 < p.K; k0 += 16) {
      for (int i = threadIdx.x; i < 64 * 16; i += 256) {
        const int r = i / 16, k = i % 16;
        const bool in = k0 + k < p.K;
        xs[k][r] = in && m0 + r < p.M
                       ? to_f32(reinterpret_cast<const T*>(p.x)[(m0 + r) * p.ldx + k0 + k])
                       : 0.f;
        ws[k][r] = in && n0 + r < p.N
                       ? to_f32(reinterpret_cast<const T*>(p.w)[(size_t)(n0 + r) * p.K + k0 + k])
                       : 0.f;
      }
      __syncthreads();
      for (int k = 0; k < 16; ++k)
        for (int i = 0; i < 4; ++i)
          for (int j = 0; j < 4; ++j)
            acc[i][j] = fmaf(xs[k][tm * 4 + i], ws[k][tn * 4 + j], acc[i][j]);
      __syncthreads();
    }
  }
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + tm * 4 + i;
    if (m >= p.M) continue;
    const int id = p.ids[m];
    if (id >= p.L && blockIdx.x == 0 && tn == 0) atomicOr(p.err, QMOE_FLAG_BAD_ID);
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tn * 4 + j;
      if (n >= p.N) continue;
      float v = acc[i][j];
      if (id >= 0 && id < p.L) {
        const T* b = reinterpret_cast<const T*>(p.b) + ((size_t)id * p.N + n) * p.R;
        for (int r = 0; r < p.R; ++r) v = fmaf(p.t[(size_t)m * p.R + r], to_f32(b[r]), v);
      }
      if (p.base) v += to_f32(reinterpret_cast<const T*>(p.base)[m * p.ldbase + n]);
      reinterpret_cast<T*>(p.out)[(size_t)m * p.N + n] = from_f32<T>(v);
    }
  }
}

template <class T>
cudaError_t run(const LoraArgs& p, int num_sms, cudaStream_t stream) {
  long long blocks = ((long long)p.M * p.R + 7) / 8;
  if (blocks > num_sms * 8LL) blocks = num_sms * 8LL;
  lora_shrink_kernel<T><<<(unsigned)blocks, 256, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if ((p.M + 63) / 64 > 65535) return cudaErrorInvalidValue;
  lora_expand_kernel<T><<<dim3((p.N + 63) / 64, (p.M + 63) / 64), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lora(const LoraArgs& p, int dtype, int num_sms, cudaStream_t stream) {
  return dtype == QMOE_DTYPE_BF16 ? run<__nv_bfloat16>(p, num_sms, stream)
                                  : run<__half>(p, num_sms, stream);
}

}  // namespace qmoe
