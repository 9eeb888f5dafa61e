// The end of a product of the gated feed-forward block whose K was cut into segments (ffn_gemm.cu):
// the segments' sums, in their order, and what a tile's epilogue does with them.  A thread has eight
// neighbouring columns of a row; four threads in a row have a block of a checkpoint.  Bound by L2,
// which still holds the sums (1023 tokens, I = 1000, four segments: 8.6 us with cold caches).
#include "checkpoint.cuh"
#include "ffn.cuh"

namespace qmoe {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void add_up(const FfnGemm& p, size_t at, size_t apart, bool in,
                                       float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = 0.f;
  if (!in) return;
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s) {
    const float4* src = reinterpret_cast<const float4*>(p.part + s * apart + at);
    const float4 a = __ldcg(src), b = __ldcg(src + 1);
    f[0] += a.x, f[1] += a.y, f[2] += a.z, f[3] += a.w;
    f[4] += b.x, f[5] += b.y, f[6] += b.z, f[7] += b.w;
  }
}

template <class T>
__device__ __forceinline__ void store8(void* base, size_t at, const float (&f)[8]) {
  Pack<T, 8> o;
#pragma unroll
  for (int e = 0; e < 8; ++e) o.v[e] = from_f32<T>(f[e]);
  *reinterpret_cast<uint4*>(reinterpret_cast<T*>(base) + at) = o.raw;
}

// (all lanes of a warp; `block` of 32 columns, of a row's)
__device__ __forceinline__ void save8(const float (&f)[8], bool in, bool first, int8_t* codes,
                                      uint8_t* scale) {
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(f[e]) & 0x7fffffffu);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const uint32_t byte = ck_byte(top);
  const float inverse = ck_inverse(byte);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    w[e / 4] |= (uint32_t)(ck_code(f[e], inverse) & 255) << (8 * (e & 3));
  if (!in) return;
  *reinterpret_cast<uint2*>(codes) = make_uint2(w[0], w[1]);
  if (first) *scale = (uint8_t)byte;
}

template <class T, FfnOp OP>
__global__ void __launch_bounds__(kThreads) ffn_finish_kernel(const FfnGemm p) {
  const int blocks = (p.N + kCkBlock - 1) / kCkBlock;
  const long long units = (long long)p.M * blocks * 4;
  const size_t width = OP == FfnOp::kUp ? 2 * (size_t)p.N : (size_t)p.N, apart = p.M * width;
  const bool gelu = p.activation == QMOE_ACT_GELU;
  grid_dep_wait();
  grid_dep_launch();
  for (long long u0 = blockIdx.x * (long long)kThreads; u0 < units;
       u0 += gridDim.x * (long long)kThreads) {
    const long long u = u0 + threadIdx.x;
    const long long row = u / (4 * blocks);
    const int at = (int)(u - row * 4 * blocks), col = at * 8;
    const bool in = u < units && col < p.N;
    float f[8];
    add_up(p, row * width + col, apart, in, f);
    if constexpr (OP == FfnOp::kUp) {
      float g[8];
      add_up(p, row * width + p.N + col, apart, in, g);
      const size_t kept = (size_t)row * 2 * p.N + col, sat = (size_t)row * 2 * blocks + at / 4;
      if (p.save == 8) {
        save8(f, in, at % 4 == 0, p.codes + kept, p.scales + sat);
        save8(g, in, at % 4 == 0, p.codes + kept + p.N, p.scales + sat + blocks);
      }
      if (!in) continue;
      if (p.save == 16) {
        float a[8], b[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] = within<T>(f[e]), b[e] = within<T>(g[e]);
        store8<T>(p.ug, kept, a);
        store8<T>(p.ug, kept + p.N, b);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = gated(gelu, p.limit, f[e], g[e]);
    } else if constexpr (OP == FfnOp::kDh) {
      if (!in) continue;
      const size_t kept = (size_t)row * 2 * p.N + col, sat = (size_t)row * 2 * blocks + at / 4;
      float u8[8], g8[8], du[8], dg[8];
      if (p.kept_scales) {
        const int8_t* c = reinterpret_cast<const int8_t*>(p.kept) + kept;
        const float su = ck_value(p.kept_scales[sat]), sg = ck_value(p.kept_scales[sat + blocks]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          u8[e] = ck_restore<T>(c[e], su);
          g8[e] = ck_restore<T>(c[p.N + e], sg);
        }
      } else {
        Pack<T, 8> a, b;
        a.raw = *reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(p.kept) + kept);
        b.raw = *reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(p.kept) + kept + p.N);
#pragma unroll
        for (int e = 0; e < 8; ++e) u8[e] = to_f32(a.v[e]), g8[e] = to_f32(b.v[e]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        f[e] = gated_backward(gelu, p.limit, u8[e], g8[e], f[e], &du[e], &dg[e]);
      store8<T>(p.ug, kept, du);
      store8<T>(p.ug, kept + p.N, dg);
    }
    if (in) store8<T>(p.out, (size_t)row * p.N + col, f);
  }
}

template <class T, FfnOp OP>
cudaError_t run(const FfnGemm& p, cudaStream_t stream) {
  const long long units = (long long)p.M * ((p.N + kCkBlock - 1) / kCkBlock) * 4;
  const long long ctas = (units + kThreads - 1) / kThreads;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.gridDim = dim3((unsigned)(ctas < 1 << 16 ? ctas : 1 << 16));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, ffn_finish_kernel<T, OP>, p);
}

template <class T>
cudaError_t of_op(const FfnGemm& p, cudaStream_t stream) {
  if (p.op == FfnOp::kUp) return run<T, FfnOp::kUp>(p, stream);
  if (p.op == FfnOp::kDh) return run<T, FfnOp::kDh>(p, stream);
  return run<T, FfnOp::kNT>(p, stream);  // (plain, whatever the operands were)
}

}  // namespace

cudaError_t launch_ffn_finish(const FfnGemm& p, cudaStream_t stream) {
  return p.dtype == QMOE_DTYPE_BF16 ? of_op<__nv_bfloat16>(p, stream) : of_op<__half>(p, stream);
}

}  // namespace qmoe
