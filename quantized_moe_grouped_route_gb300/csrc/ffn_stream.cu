// The gated feed-forward block for one to eight tokens, forward: both products stream their weights
// once, bound by that stream.  A warp multiplies 16 rows of weights (m16n8k16, the tokens are the
// MMA's eight columns) straight from memory: each lane reads 16 bytes of two rows at a time, and
// since a sum over K may be taken in any order, the eight elements of such a chunk are used as the
// MMA's fragments as they come, the tokens' chunks likewise, so nothing is moved between lanes.
// The warps of a CTA take parts of K of the same rows, added up in shared memory in their order.
// The first product's 16 rows are eight of u and the same eight of g: a lane ends up with both, and
// h = act(g) u is made where they are.  1 token, H = 7168, I = 2048: 17.4 us in a graph, 5.1 TB/s
// over both launches.
#include "ffn.cuh"
#include "mma.cuh"

namespace qmoe {
namespace {

// Many warps with four chunks of two rows each in flight, in 60 registers, so that two CTAs fit an
// SM: 17.6 us a call of one token, H = 7168, I = 2048; eight warps with four chunks 20.8, with
// eight 18.3, sixteen with seven (one CTA an SM) 21.6.
constexpr int kWarps = 16;
constexpr int kAhead = 4;

// UP: rows 8 b .. 8 b + 7 of u and of g, b the CTA; else rows 16 b .. 16 b + 15.
template <class T, bool UP>
__global__ void __launch_bounds__(kWarps * 32) ffn_stream_kernel(const FfnProduct p) {
  __shared__ float4 part[kWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int row0 = blockIdx.x * (UP ? 8 : 16) + g;
  const bool in0 = row0 < p.N, in1 = UP ? in0 : row0 + 8 < p.N;
  const T* w = reinterpret_cast<const T*>(p.b);
  const T* w0 = w + (size_t)(in0 ? row0 : 0) * p.K + q * 8;
  const T* w1 = w + (size_t)(UP ? p.N + row0 : in1 ? row0 + 8 : 0) * p.K + q * 8;
  const bool token = g < p.M;
  const T* x = reinterpret_cast<const T*>(p.a) + (token ? g : 0) * p.lda + q * 8;
  const int steps = (p.K + 31) / 32;
  const int s0 = steps * warp / kWarps, s1 = steps * (warp + 1) / kWarps;
  float c[4] = {0.f, 0.f, 0.f, 0.f};
  uint4 a0[kAhead], a1[kAhead], b[kAhead];
  auto weights = [&](int s, int i) {
    const bool in = s + i < s1 && (s + i) * 32 + q * 8 < p.K;
    const int at = in ? (s + i) * 32 : 0;
    a0[i] = load_if(reinterpret_cast<const uint4*>(w0 + at), in && in0);
    a1[i] = load_if(reinterpret_cast<const uint4*>(w1 + at), in && in1);
  };
  // The second product's kernel starts while the first runs, once that has waited for what came
  // before the call: by then the weights are complete, whoever wrote them, and can be asked for.
  if (UP) grid_dep_wait();
#pragma unroll
  for (int i = 0; i < kAhead; ++i) weights(s0, i);
  if (!UP) grid_dep_wait();
  grid_dep_launch();
  if (p.clear_err && blockIdx.x == 0 && threadIdx.x == 0) *p.err = 0;
  for (int s = s0; s < s1; s += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const bool in = s + i < s1 && (s + i) * 32 + q * 8 < p.K;
      b[i] = load_if(reinterpret_cast<const uint4*>(x + (in ? (s + i) * 32 : 0)), in && token);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      mma_m16n8k16<T>(c, a0[i].x, a1[i].x, a0[i].y, a1[i].y, b[i].x, b[i].y);
      mma_m16n8k16<T>(c, a0[i].z, a1[i].z, a0[i].w, a1[i].w, b[i].z, b[i].w);
      weights(s + kAhead, i);
    }
  }
  part[warp][lane] = make_float4(c[0], c[1], c[2], c[3]);
  __syncthreads();
  if (warp != 0) return;
  float4 t = part[0][lane];
#pragma unroll
  for (int i = 1; i < kWarps; ++i) {
    const float4 v = part[i][lane];
    t.x += v.x, t.y += v.y, t.z += v.z, t.w += v.w;
  }
  // t: row0's tokens 2 q and 2 q + 1, then the other row's
  T* out = reinterpret_cast<T*>(p.out) + (size_t)(2 * q) * p.N + row0;
  if (UP) {
    const bool gelu = p.activation == QMOE_ACT_GELU;
    if (in0 && 2 * q < p.M) out[0] = from_f32<T>(gated(gelu, p.limit, t.x, t.z));
    if (in0 && 2 * q + 1 < p.M) out[p.N] = from_f32<T>(gated(gelu, p.limit, t.y, t.w));
  } else {
    if (in0 && 2 * q < p.M) out[0] = from_f32<T>(t.x);
    if (in0 && 2 * q + 1 < p.M) out[p.N] = from_f32<T>(t.y);
    if (in1 && 2 * q < p.M) out[8] = from_f32<T>(t.z);
    if (in1 && 2 * q + 1 < p.M) out[p.N + 8] = from_f32<T>(t.w);
  }
}

template <class T>
cudaError_t run(const FfnProduct& p, cudaStream_t stream) {
  const bool up = p.op == FfnOp::kUp;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.gridDim = dim3((unsigned)(up ? (p.N + 7) / 8 : (p.N + 15) / 16));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, up ? ffn_stream_kernel<T, true> : ffn_stream_kernel<T, false>, p);
}

}  // namespace

cudaError_t launch_ffn_stream(const FfnProduct& p, cudaStream_t stream) {
  return p.dtype == QMOE_DTYPE_BF16 ? run<__nv_bfloat16>(p, stream) : run<__half>(p, stream);
}

}  // namespace qmoe
