// Tokens in expert order and back, with their gradients.
//
//   sort            xs[pos] = x[m]                 for every routed pair (m, k), pos = pair_pos[m][k]
//   sort backward   dx[m]   = sum_k dxs[pos]
//   unsort          out[m]  = sum_k w[m][k] y[pos]
//   unsort backward dy[pos] = w[m][k] dout[m],  dw[m][k] = <dout[m], y[pos]>
//
// Skipped pairs (pair_pos < 0) take no part: their weight's gradient is 0, and the rows
// of a sorted array past the routed pairs are zeros.  All four are bound by HBM: each
// kernel walks the tokens, so a token's row is read (or written) once however many of its
// pairs are routed, and each pair row is touched once.  Sums are in fp32 in slot order,
// rounded once; no atomics, so results are deterministic.
//
// A row moves in chunks of 16 bytes where the base pointers, row strides and row length
// allow it, else in single elements (chunk_bytes in api_ops.cu).
#include "common.cuh"
#include "launch.h"
#include "pack.cuh"

namespace qmoe {
namespace {

constexpr int kTokThreads = 256;

// (token, segment of 256 chunks) items, one per warp: the segment is read once and written
// to each of the token's pairs.
template <class C>
__global__ void __launch_bounds__(kTokThreads)
    sort_copy_kernel(const C* __restrict__ x, long long ldx, const int32_t* __restrict__ pair_pos,
                     const int32_t* __restrict__ n_routed, int M, int top_k, int chunks,
                     C* __restrict__ xs) {
  grid_dep_wait();  // the route's tables
  grid_dep_launch();
  constexpr int kSeg = 256, kPer = kSeg / 32;
  const int nseg = (chunks + kSeg - 1) / kSeg;
  const int P = M * top_k;
  const long long items = (long long)M * nseg;
  const int lane = threadIdx.x & 31;
  const long long w0 = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const long long warps = ((long long)gridDim.x * blockDim.x) >> 5;
  for (long long it = w0; it < items; it += warps) {
    const int m = (int)(it / nseg);
    const int c0 = (int)(it - (long long)m * nseg) * kSeg + lane;
    const C* src = x + (size_t)m * ldx;
    C v[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (c0 + 32 * j < chunks) v[j] = src[c0 + 32 * j];
    for (int k = 0; k < top_k; ++k) {
      const int pos = pair_pos[(size_t)m * top_k + k];
      if ((unsigned)pos >= (unsigned)P) continue;
      C* dst = xs + (size_t)pos * chunks;
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (c0 + 32 * j < chunks) dst[c0 + 32 * j] = v[j];
    }
  }
  // the rows of skipped pairs, after the routed ones
  const int first = n_routed[0];
  const long long tail = (long long)(P - first) * nseg;
  for (long long it = w0; it < tail; it += warps) {
    const int r = (int)(it / nseg);
    const int c0 = (int)(it - (long long)r * nseg) * kSeg + lane;
    C* dst = xs + (size_t)(first + r) * chunks;
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (c0 + 32 * j < chunks) dst[c0 + 32 * j] = C{};
  }
}

// A thread per (token, chunk of N elements): the pairs' chunks are added in slot order.
template <class T, int N, bool WEIGHTED>
__global__ void __launch_bounds__(kTokThreads)
    unsort_kernel(const T* __restrict__ y, long long ldy, const int32_t* __restrict__ pair_pos,
                  const float* __restrict__ w, int M, int top_k, int chunks, T* __restrict__ out) {
  using P_ = Pack<T, N>;
  grid_dep_wait();
  grid_dep_launch();
  const unsigned P = (unsigned)(M * top_k);
  const long long total = (long long)M * chunks;
  const long long step = (long long)gridDim.x * blockDim.x;
  for (long long it = (long long)blockIdx.x * blockDim.x + threadIdx.x; it < total; it += step) {
    const int m = (int)(it / chunks);
    const int c = (int)(it - (long long)m * chunks);
    const int32_t* pp = pair_pos + (size_t)m * top_k;
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
    constexpr int kBatch = 8;
    for (int k0 = 0; k0 < top_k; k0 += kBatch) {
      P_ v[kBatch];
      bool has[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int pos = k0 + k < top_k ? pp[k0 + k] : -1;
        has[k] = (unsigned)pos < P;
        if (has[k])
          v[k].raw = *reinterpret_cast<const typename P_::raw_t*>(y + (size_t)pos * ldy +
                                                                  (size_t)c * N);
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (!has[k]) continue;
        const float wk = WEIGHTED ? w[(size_t)m * top_k + k0 + k] : 1.f;
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = fmaf(wk, to_f32(v[k].v[i]), acc[i]);
      }
    }
    P_ o;
#pragma unroll
    for (int i = 0; i < N; ++i) o.v[i] = from_f32<T>(acc[i]);
    *reinterpret_cast<typename P_::raw_t*>(out + (size_t)it * N) = o.raw;
  }
}

// A block per token: its gradient row is read once per eight slots (later reads hit L1),
// each slot's row of y once; the dot products are reduced over the block in a fixed order.
template <class T, int N>
__global__ void __launch_bounds__(kTokThreads)
    unsort_backward_kernel(const T* __restrict__ dout, long long ldd, const T* __restrict__ y,
                           long long ldy, const int32_t* __restrict__ sorted_pair,
                           const int32_t* __restrict__ pair_pos, const float* __restrict__ w, int M,
                           int top_k, int chunks, T* __restrict__ dy, float* __restrict__ dw) {
  using P_ = Pack<T, N>;
  using R_ = typename P_::raw_t;
  grid_dep_wait();
  grid_dep_launch();
  constexpr int kBatch = 8, kWarps = kTokThreads / 32;
  __shared__ float part[kWarps][kBatch];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned P = (unsigned)(M * top_k);
  for (int m = blockIdx.x; m < M; m += gridDim.x) {
    const T* d = dout + (size_t)m * ldd;
    for (int k0 = 0; k0 < top_k; k0 += kBatch) {
      int pos[kBatch];
      float wk[kBatch], acc[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const size_t i = (size_t)m * top_k + k0 + k;
        pos[k] = k0 + k < top_k ? pair_pos[i] : -1;
        wk[k] = k0 + k < top_k ? w[i] : 0.f;
        acc[k] = 0.f;
      }
      for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
        P_ g, v[kBatch];
        g.raw = *reinterpret_cast<const R_*>(d + (size_t)c * N);
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if ((unsigned)pos[k] < P)
            v[k].raw = *reinterpret_cast<const R_*>(y + (size_t)pos[k] * ldy + (size_t)c * N);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          if ((unsigned)pos[k] >= P) continue;
          P_ o;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float gi = to_f32(g.v[i]);
            acc[k] = fmaf(gi, to_f32(v[k].v[i]), acc[k]);
            o.v[i] = from_f32<T>(wk[k] * gi);
          }
          *reinterpret_cast<R_*>(dy + ((size_t)pos[k] * chunks + c) * N) = o.raw;
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
#pragma unroll
        for (int o = 16; o; o >>= 1) acc[k] += __shfl_xor_sync(0xffffffffu, acc[k], o);
        if (lane == 0) part[warp][k] = acc[k];
      }
      __syncthreads();
      if (threadIdx.x < kBatch && k0 + threadIdx.x < top_k) {
        float s = 0.f;
        for (int i = 0; i < (int)(blockDim.x >> 5); ++i) s += part[i][threadIdx.x];
        dw[(size_t)m * top_k + k0 + threadIdx.x] = s;
      }
      __syncthreads();
    }
    // as many positions per block as slots: those past the routed pairs are zeroed
    for (int k = 0; k < top_k; ++k) {
      const size_t pos = (size_t)m * top_k + k;
      if (sorted_pair[pos] >= 0) continue;
      P_ z;
#pragma unroll
      for (int i = 0; i < N; ++i) z.v[i] = from_f32<T>(0.f);
      for (int c = threadIdx.x; c < chunks; c += blockDim.x)
        *reinterpret_cast<R_*>(dy + (pos * chunks + c) * N) = z.raw;
    }
  }
}

cudaLaunchConfig_t config(long long blocks, int threads, cudaStream_t stream,
                          cudaLaunchAttribute* attr) {
  attr[0] = pdl_attribute();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks < 1 ? 1 : blocks));
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <class C>
cudaError_t sort_copy(const void* x, long long ldx_bytes, const int32_t* pair_pos,
                      const int32_t* n_routed, int M, int top_k, long long row_bytes, void* xs,
                      int num_sms, cudaStream_t stream) {
  const int chunks = (int)(row_bytes / (long long)sizeof(C));
  const long long warps = (long long)M * ((chunks + 255) / 256);
  long long blocks = (warps * 32 + kTokThreads - 1) / kTokThreads;
  if (blocks > num_sms * 8LL) blocks = num_sms * 8LL;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = config(blocks, kTokThreads, stream, attr);
  return cudaLaunchKernelEx(&cfg, sort_copy_kernel<C>, reinterpret_cast<const C*>(x),
                            ldx_bytes / (long long)sizeof(C), pair_pos, n_routed, M, top_k, chunks,
                            reinterpret_cast<C*>(xs));
}

template <class T, int N>
cudaError_t unsort(const TokenArgs& a, int num_sms, cudaStream_t stream) {
  const int chunks = a.H / N;
  const long long total = (long long)a.M * chunks;
  long long blocks = (total + kTokThreads - 1) / kTokThreads;
  if (blocks > num_sms * 8LL) blocks = num_sms * 8LL;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = config(blocks, kTokThreads, stream, attr);
  const T* y = reinterpret_cast<const T*>(a.y);
  T* out = reinterpret_cast<T*>(a.out);
  if (a.weights)
    return cudaLaunchKernelEx(&cfg, unsort_kernel<T, N, true>, y, a.ldy, a.pair_pos, a.weights, a.M,
                              a.top_k, chunks, out);
  return cudaLaunchKernelEx(&cfg, unsort_kernel<T, N, false>, y, a.ldy, a.pair_pos, a.weights, a.M,
                            a.top_k, chunks, out);
}

template <class T, int N>
cudaError_t unsort_backward(const TokenArgs& a, int num_sms, cudaStream_t stream) {
  const int chunks = a.H / N;
  int threads = (chunks + 31) / 32 * 32;
  if (threads > kTokThreads) threads = kTokThreads;
  long long blocks = a.M;
  if (blocks > num_sms * 64LL) blocks = num_sms * 64LL;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = config(blocks, threads, stream, attr);
  return cudaLaunchKernelEx(&cfg, unsort_backward_kernel<T, N>, reinterpret_cast<const T*>(a.dout),
                            a.ldd, reinterpret_cast<const T*>(a.y), a.ldy, a.sorted_pair,
                            a.pair_pos, a.weights, a.M, a.top_k, chunks,
                            reinterpret_cast<T*>(a.out), a.dweights);
}

}  // namespace

cudaError_t launch_sort_copy(const void* x, long long ldx_bytes, const int32_t* pair_pos,
                             const int32_t* n_routed, int M, int top_k, long long row_bytes,
                             int chunk_bytes, void* xs, int num_sms, cudaStream_t stream) {
  if (chunk_bytes == 16)
    return sort_copy<uint4>(x, ldx_bytes, pair_pos, n_routed, M, top_k, row_bytes, xs, num_sms,
                            stream);
  if (chunk_bytes == 4)
    return sort_copy<uint32_t>(x, ldx_bytes, pair_pos, n_routed, M, top_k, row_bytes, xs, num_sms,
                               stream);
  return sort_copy<uint16_t>(x, ldx_bytes, pair_pos, n_routed, M, top_k, row_bytes, xs, num_sms,
                             stream);
}

cudaError_t launch_unsort(const TokenArgs& a, int dtype, bool vec, int num_sms,
                          cudaStream_t stream) {
  if (dtype == QMOE_DTYPE_BF16)
    return vec ? unsort<__nv_bfloat16, 8>(a, num_sms, stream)
               : unsort<__nv_bfloat16, 1>(a, num_sms, stream);
  if (dtype == QMOE_DTYPE_FP16)
    return vec ? unsort<__half, 8>(a, num_sms, stream) : unsort<__half, 1>(a, num_sms, stream);
  return vec ? unsort<float, 4>(a, num_sms, stream) : unsort<float, 1>(a, num_sms, stream);
}

cudaError_t launch_unsort_backward(const TokenArgs& a, int dtype, bool vec, int num_sms,
                                   cudaStream_t stream) {
  if (dtype == QMOE_DTYPE_BF16)
    return vec ? unsort_backward<__nv_bfloat16, 8>(a, num_sms, stream)
               : unsort_backward<__nv_bfloat16, 1>(a, num_sms, stream);
  if (dtype == QMOE_DTYPE_FP16)
    return vec ? unsort_backward<__half, 8>(a, num_sms, stream)
               : unsort_backward<__half, 1>(a, num_sms, stream);
  return vec ? unsort_backward<float, 4>(a, num_sms, stream)
             : unsort_backward<float, 1>(a, num_sms, stream);
}

}  // namespace qmoe
