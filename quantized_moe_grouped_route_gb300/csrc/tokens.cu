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
// A row moves in the widest chunks, up to 16 bytes, that the base pointers, row strides and
// row length allow (Chunk in api_ops.cu); an odd width moves element by element.
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

// The whole sort of few pairs in one launch: a block per (token, segment of kTokThreads
// chunks), which finds the positions of its own token's pairs from all ids.  With a skipped
// pair standing for expert E, pair i goes to
//   #(j: e_j < e_i) + #(j < i: e_j = e_i),
// a count over all ids per pair, one warp each; the skipped pairs' positions are the rows
// past the routed ones, which their tokens' blocks zero.  The offsets (#(j: e_j < e)) are
// shared out over all warps of the grid.  Against the one-block route and the copy as two
// launches a call over 128 pairs of 7168 bf16 went from 10.8 to 6.7 us (5 of them the
// host's).  Above kSortSmallPairs the counts, P per pair, would outweigh a launch.
template <class C>
__global__ void __launch_bounds__(kTokThreads)
    sort_small_kernel(const C* __restrict__ x, long long ldx, const int32_t* __restrict__ ids,
                      int M, int top_k, int E, int chunks, C* __restrict__ xs,
                      int32_t* __restrict__ offsets, int32_t* __restrict__ sorted_pair,
                      int32_t* __restrict__ pair_pos, unsigned int* __restrict__ err) {
  __shared__ int key[kSortSmallPairs];
  __shared__ int place[64];
  grid_dep_wait();
  grid_dep_launch();
  constexpr int kWarps = kTokThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int P = M * top_k, m = blockIdx.x, c = blockIdx.y * kTokThreads + threadIdx.x;
  C v{};
  if (c < chunks) v = x[(size_t)m * ldx + c];
  bool bad = false;
  for (int i = threadIdx.x; i < P; i += kTokThreads) {
    const int e = ids[i];
    bad |= e >= E;
    key[i] = e < 0 || e > E ? E : e;
  }
  bad = __syncthreads_or(bad);
  for (int k = warp; k < top_k; k += kWarps) {
    const int i = m * top_k + k, e = key[i];
    int n = 0;
    for (int j = lane; j < P; j += 32) n += key[j] < e || (key[j] == e && j < i);
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) {
      place[k] = e < E ? n : ~n;
      if (blockIdx.y == 0) {
        sorted_pair[n] = e < E ? i : -1;
        pair_pos[i] = e < E ? n : -1;
      }
    }
  }
  const int blocks = gridDim.x * gridDim.y, block = blockIdx.y * gridDim.x + blockIdx.x;
  for (int e = block * kWarps + warp; e <= E; e += blocks * kWarps) {
    int n = 0;
    for (int j = lane; j < P; j += 32) n += key[j] < e;
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) offsets[e] = n;
  }
  if (block == 0 && threadIdx.x == 0) err[0] = bad ? QMOE_FLAG_BAD_ID : 0u;
  __syncthreads();
  if (c < chunks)
    for (int k = 0; k < top_k; ++k) {
      const int at = place[k];
      xs[(size_t)(at >= 0 ? at : ~at) * chunks + c] = at >= 0 ? v : C{};
    }
}

// (token, segment of kPer * 32 chunks of N elements) items, one per warp, so that a lane has
// kPer * (slots) loads in flight: the pairs' chunks are added in slot order.  kPer is 1 for
// 16-byte chunks; narrower ones need more of them for the same bytes in flight (fp16 rows
// of 1001 elements, 1023 tokens of 4 slots: one element a thread took 10.3 us).
template <class T, int N>
__host__ __device__ constexpr int chunks_per_lane() {
  return 16 / (int)(sizeof(T) * N) < 4 ? 16 / (int)(sizeof(T) * N) : 4;
}
template <class T, int N, bool WEIGHTED>
__global__ void __launch_bounds__(kTokThreads)
    unsort_kernel(const T* __restrict__ y, long long ldy, const int32_t* __restrict__ pair_pos,
                  const float* __restrict__ w, int M, int top_k, int chunks, T* __restrict__ out) {
  using P_ = Pack<T, N>;
  using R_ = typename P_::raw_t;
  constexpr int kPer = chunks_per_lane<T, N>(), kBatch = 8 / kPer < 4 ? 4 : 8 / kPer;
  grid_dep_wait();
  grid_dep_launch();
  const unsigned P = (unsigned)(M * top_k);
  const int lane = threadIdx.x & 31;
  const int nseg = (chunks + 32 * kPer - 1) / (32 * kPer);
  const long long items = (long long)M * nseg;
  const long long step = ((long long)gridDim.x * blockDim.x) >> 5;
  for (long long it = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5; it < items;
       it += step) {
    const int m = (int)(it / nseg);
    const int c0 = (int)(it - (long long)m * nseg) * 32 * kPer + lane;
    const size_t slot0 = (size_t)m * top_k;
    float acc[kPer][N];
#pragma unroll
    for (int j = 0; j < kPer; ++j)
#pragma unroll
      for (int i = 0; i < N; ++i) acc[j][i] = 0.f;
    for (int k0 = 0; k0 < top_k; k0 += kBatch) {
      P_ v[kBatch][kPer];
      float wk[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int pos = k0 + k < top_k ? pair_pos[slot0 + k0 + k] : -1;
        const bool has = (unsigned)pos < P;
        // a skipped pair's chunk is zeros, its row is not read
        wk[k] = !has ? 0.f : WEIGHTED ? w[slot0 + k0 + k] : 1.f;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          if constexpr (sizeof(R_) >= 4) {
            const T* at = y + (has ? (size_t)pos * ldy + (size_t)(c0 + 32 * j) * N : 0);
            v[k][j].raw = load_if(reinterpret_cast<const R_*>(at), has && c0 + 32 * j < chunks);
          } else {  // (two bytes: behind a branch 3.8 us for the 1001-wide rows, so 4.8)
            v[k][j].raw = R_{};
            if (has && c0 + 32 * j < chunks)
              v[k][j].raw = *reinterpret_cast<const R_*>(y + (size_t)pos * ldy +
                                                         (size_t)(c0 + 32 * j) * N);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
#pragma unroll
        for (int j = 0; j < kPer; ++j)
#pragma unroll
          for (int i = 0; i < N; ++i) acc[j][i] = fmaf(wk[k], to_f32(v[k][j].v[i]), acc[j][i]);
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (c0 + 32 * j >= chunks) continue;
      P_ o;
#pragma unroll
      for (int i = 0; i < N; ++i) o.v[i] = from_f32<T>(acc[j][i]);
      *reinterpret_cast<R_*>(out + ((size_t)m * chunks + c0 + 32 * j) * N) = o.raw;
    }
  }
}

template <class T, int N>
__host__ __device__ constexpr int backward_chunks() {
  return N == 1 ? 1 : chunks_per_lane<T, N>();
}

// A block per token: its gradient row is read once per batch of slots (later reads hit L1),
// each slot's row of y once; the dot products are reduced over the block in a fixed order.
// A thread takes kPer chunks of each of kBatch slots at a time: several of 4 or 8 bytes
// (4096 tokens of 1002 fp16, 8 slots: 46.8 -> 30.3 us), one of 16 bytes or of one element
// (1001: 46.4 us against 60.4).
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
  constexpr int kPer = backward_chunks<T, N>(), kBatch = kPer == 1 ? 8 : 4;
  constexpr int kWarps = kTokThreads / 32;
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
      for (int c0 = threadIdx.x; c0 < chunks; c0 += kPer * blockDim.x) {
        P_ g[kPer], v[kBatch][kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int c = c0 + j * blockDim.x;
          const bool in = c < chunks;
          g[j].raw = *reinterpret_cast<const R_*>(d + (in ? (size_t)c * N : 0));
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            if constexpr (kPer == 1) {
              if ((unsigned)pos[k] < P)
                v[k][j].raw = *reinterpret_cast<const R_*>(y + (size_t)pos[k] * ldy + (size_t)c * N);
            } else {  // an element of row 0 stands in for one that is not there
              const bool there = in && (unsigned)pos[k] < P;
              v[k][j].raw =
                  *reinterpret_cast<const R_*>(y + (there ? (size_t)pos[k] * ldy + (size_t)c * N : 0));
            }
          }
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int c = c0 + j * blockDim.x;
          if (c >= chunks) break;
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            if ((unsigned)pos[k] >= P) continue;
            P_ o;
#pragma unroll
            for (int i = 0; i < N; ++i) {
              const float gi = to_f32(g[j].v[i]);
              acc[k] = fmaf(gi, to_f32(v[k][j].v[i]), acc[k]);
              o.v[i] = from_f32<T>(wk[k] * gi);
            }
            *reinterpret_cast<R_*>(dy + ((size_t)pos[k] * chunks + c) * N) = o.raw;
          }
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
                      cudaStream_t stream) {
  const int chunks = (int)(row_bytes / (long long)sizeof(C));
  const long long warps = (long long)M * ((chunks + 255) / 256);
  long long blocks = (warps * 32 + kTokThreads - 1) / kTokThreads;
  if (blocks > (1 << 22)) blocks = 1 << 22;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = config(blocks, kTokThreads, stream, attr);
  return cudaLaunchKernelEx(&cfg, sort_copy_kernel<C>, reinterpret_cast<const C*>(x),
                            ldx_bytes / (long long)sizeof(C), pair_pos, n_routed, M, top_k, chunks,
                            reinterpret_cast<C*>(xs));
}

template <class T, int N>
cudaError_t unsort(const TokenArgs& a, cudaStream_t stream) {
  const int chunks = a.H / N;
  const int per_warp = 32 * chunks_per_lane<T, N>();
  const long long warps = (long long)a.M * ((chunks + per_warp - 1) / per_warp);
  // a block per eight items, so that the last round of blocks is a small share of them
  long long blocks = (warps * 32 + kTokThreads - 1) / kTokThreads;
  if (blocks > (1 << 22)) blocks = 1 << 22;
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
  constexpr int kPer = backward_chunks<T, N>();
  int threads = ((chunks + kPer - 1) / kPer + 31) / 32 * 32;
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
                             int chunk_bytes, void* xs, cudaStream_t stream) {
  auto go = [&](auto c) {
    return sort_copy<decltype(c)>(x, ldx_bytes, pair_pos, n_routed, M, top_k, row_bytes, xs, stream);
  };
  return chunk_bytes == 16  ? go(uint4{})
         : chunk_bytes == 8 ? go(uint2{})
         : chunk_bytes == 4 ? go(uint32_t{})
                            : go(uint16_t{});
}

cudaError_t launch_sort_small(const void* x, long long ldx_bytes, const int32_t* ids, int M,
                              int top_k, int E, long long row_bytes, int chunk_bytes, void* xs,
                              int32_t* offsets, int32_t* sorted_pair, int32_t* pair_pos,
                              unsigned int* err, cudaStream_t stream) {
  auto go = [&](auto c) {
    using C = decltype(c);
    const int chunks = (int)(row_bytes / (long long)sizeof(C));
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config(M, kTokThreads, stream, attr);
    cfg.gridDim.y = (chunks + kTokThreads - 1) / kTokThreads;
    return cudaLaunchKernelEx(&cfg, sort_small_kernel<C>, reinterpret_cast<const C*>(x),
                              ldx_bytes / (long long)sizeof(C), ids, M, top_k, E, chunks,
                              reinterpret_cast<C*>(xs), offsets, sorted_pair, pair_pos, err);
  };
  return chunk_bytes == 16  ? go(uint4{})
         : chunk_bytes == 8 ? go(uint2{})
         : chunk_bytes == 4 ? go(uint32_t{})
                            : go(uint16_t{});
}

template <class T>
static cudaError_t unsort_chunk(const TokenArgs& a, int chunk, cudaStream_t stream) {
  if constexpr (sizeof(T) == 2)
    if (chunk == 8) return unsort<T, 8>(a, stream);
  return chunk == 4 ? unsort<T, 4>(a, stream) : chunk == 2 ? unsort<T, 2>(a, stream)
                                                           : unsort<T, 1>(a, stream);
}

cudaError_t launch_unsort(const TokenArgs& a, int dtype, int chunk, cudaStream_t stream) {
  if (dtype == QMOE_DTYPE_BF16) return unsort_chunk<__nv_bfloat16>(a, chunk, stream);
  if (dtype == QMOE_DTYPE_FP16) return unsort_chunk<__half>(a, chunk, stream);
  return unsort_chunk<float>(a, chunk, stream);
}

template <class T>
static cudaError_t unsort_backward_chunk(const TokenArgs& a, int chunk, int num_sms,
                                         cudaStream_t stream) {
  if constexpr (sizeof(T) == 2)
    if (chunk == 8) return unsort_backward<T, 8>(a, num_sms, stream);
  return chunk == 4   ? unsort_backward<T, 4>(a, num_sms, stream)
         : chunk == 2 ? unsort_backward<T, 2>(a, num_sms, stream)
                      : unsort_backward<T, 1>(a, num_sms, stream);
}

cudaError_t launch_unsort_backward(const TokenArgs& a, int dtype, int chunk, int num_sms,
                                   cudaStream_t stream) {
  if (dtype == QMOE_DTYPE_BF16)
    return unsort_backward_chunk<__nv_bfloat16>(a, chunk, num_sms, stream);
  if (dtype == QMOE_DTYPE_FP16) return unsort_backward_chunk<__half>(a, chunk, num_sms, stream);
  return unsort_backward_chunk<float>(a, chunk, num_sms, stream);
}

}  // namespace qmoe
