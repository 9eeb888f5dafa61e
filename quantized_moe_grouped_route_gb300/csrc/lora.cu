// A shared projection with a low-rank adapter per token:
//   t[m] = scales[a] * (x[m] . A[a]^T),  out[m] = base[m] + x[m] . w^T + t[m] . B[a]^T
// with a = adapter_ids[m].
//
// Two kernels.  The first (shrink, lora_shrink.cu: plain fp32 products for few tokens, tensor
// cores for many) forms t in fp32 and lists, for each tile of tokens, the distinct adapters
// its tokens use.  The second (lora_gemm.cu) is one GEMM whose contraction runs over K and
// then over the ranks of the tile's adapters: the MMA's M side
// is 128 rows of w (or of B[a]), its N side a tile of up to 240 tokens, and for each of
// the tile's adapters the token operand is t with the rows of other adapters zero.  So the
// adapters cost a tile (distinct adapters) * ranks more of contraction length, whatever
// the order of the tokens, and the result is rounded once.  (A zero row times an infinity
// or NaN of another token's B is NaN, so in this form an adapter's B has to be finite for
// the tokens beside it; the two forms below keep tokens apart.)
//
// t enters the tensor cores as the sum of two values of the activation type (t rounded,
// and what the rounding left): 16 (bf16) or 22 (fp16) significant bits for twice the MMAs
// of a contraction that is short, instead of a second rounding of the result's size.
//
// GEMM pipeline (a unit is 128 rows of w per CTA x one token tile; when there are fewer
// units than SMs the contraction is split into S segments, one CTA or pair each in one
// cluster):
//   warp 0      TMA producer: steps of 64 of K, [128 rows of w | token rows], then per
//               adapter and 64 ranks [128 rows of B[a]]
//   warp 1      MMA issue: 4 x tcgen05.mma kind::f16 per step, fp32 accumulator in TMEM,
//               two accumulators, so that the epilogue overlaps the next unit
//   warps 4-7   epilogue: TMEM -> registers -> base, rounding -> a transpose through shared
//               memory -> 16-byte global stores; with S > 1 each segment's sums stay in its
//               shared memory, and after a cluster barrier every CTA adds up a share of the
//               tokens over all segments, in K order
//   warps 8-15  builders: the token operand (both values of t) of the adapter steps, in
//               slots of their own; one to four warps (the more, the wider the tile) build a
//               step, so that several steps are in the making at once
//
// Few tokens of few ranks (VEC: at most 64 tokens, tokens * ranks at most 4096; a decode
// step's requests with an adapter each) do not take the adapters through the MMA: a step
// per adapter moves 128 rows of B[a] for one or two tokens, and the tensor copies took 0.24
// us a step (64-byte rows), 5.3 of the 15.9 us of 48 tokens of 43 adapters.  There warp 2
// brings in B[a]'s rows, which lie next to each other, as one bulk copy each, while w
// streams; the builder warps multiply them with t in fp32, and the epilogue adds what they
// leave in shared memory.
//
// Few tokens (one tile): one CTA per unit, w streamed once, HBM bound.  More: CTA pairs
// (cta_group::2, M = 256), each SM loading half of the token rows, since a 128 x 256 tile
// fed by one SM alone asks more of its L2 port (96 bytes a clock) than it has.
//
// One or two tokens run as plain products, warps per row of w (lora_gemv_kernel).
//
// Every wait is bounded, as in the layer's GEMMs.
#include "lora.cuh"

namespace qmoe {
namespace {

// --------------------------------------------------------------------- one or two tokens
// One, two or four warps (WPR, the more, the longer the row) per row of w: its product with
// up to MT token rows in fp32, then the row of each token's B with t.  HBM (or L2) bound, and
// there is nothing to set up: the tensor-core kernel spends 5 of its 10.3 us at M = 1,
// K = 7168, N = 2048 on barriers, TMEM, the cluster and the last sums.  What hides the loads'
// latency is warps, not loads a warp: with few registers all rows of that size are resident
// at once (two loads in flight a lane, 16 blocks an SM: 7.1 us a call; eight loads, 8
// blocks: 9.6; for two tokens three loads and 8 blocks: 9.7, six: 12.4).  On the tensor cores
// one token takes 11.4 us, two 11.9, four 12.0 (here 16.0).
constexpr int kGemvThreads = 128;

template <class T, int MT, int WPR>
__global__ void __launch_bounds__(kGemvThreads, MT == 1 ? 16 : 8) lora_gemv_kernel(const LoraArgs p) {
  using P_ = Pack<T, 8>;
  __shared__ float part[kGemvThreads / 32][MT];
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % WPR;
  const int n = blockIdx.x * (kGemvThreads / 32 / WPR) + warp / WPR;
  const bool here = n < p.N;  // the warp's row (the others only wait for the shrink kernel)
  float acc[MT];
  int id[MT];
  T bv[MT][4];  // ranks lane, lane + 32, ..
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    acc[m] = 0.f;
    id[m] = here && sub == 0 && m < p.M ? p.ids[m] : -1;
    if (id[m] >= p.L) id[m] = -1;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (id[m] >= 0 && lane + 32 * i < p.R)
        bv[m][i] = reinterpret_cast<const T*>(p.b)[((size_t)id[m] * p.N + n) * p.R + lane + 32 * i];
  }
  if (here && p.w) {
    const uint4* w = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(p.w) + (size_t)n * p.K);
    const T* x = reinterpret_cast<const T*>(p.x);
    const int chunks = p.K / 8;
    constexpr int kFlight = MT == 1 ? 2 : 3;
    for (int c0 = sub * 32 + lane; c0 < chunks; c0 += 32 * WPR * kFlight) {
      P_ wv[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        const int c = c0 + 32 * WPR * i;
        wv[i].raw = load_if(w + c, c < chunks);
      }
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        const int c = c0 + 32 * WPR * i;
        if (c >= chunks) break;
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = to_f32(wv[i].v[e]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          if (m >= p.M) break;
          P_ xv;
          xv.raw = reinterpret_cast<const uint4*>(x + m * p.ldx)[c];
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[m] = fmaf(f[e], to_f32(xv.v[e]), acc[m]);
        }
      }
    }
  }
  grid_dep_wait();  // t
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.bad[0]) atomicOr(p.err, QMOE_FLAG_BAD_ID);
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (id[m] >= 0) {
      // (so few tokens have one segment)
      const float* t = p.t + (size_t)m * p.R + lane;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < p.R) acc[m] = fmaf(to_f32(bv[m][i]), t[32 * i], acc[m]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) acc[m] += __shfl_xor_sync(0xffffffffu, acc[m], o);
    if (lane == 0) part[warp][m] = acc[m];
  }
  __syncthreads();
  if (here && sub == 0 && lane < MT && lane < p.M) {
    const int m = lane;
    float f = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) f += part[warp + w][m];
    if (p.base) f += to_f32(reinterpret_cast<const T*>(p.base)[m * p.ldbase + n]);
    reinterpret_cast<T*>(p.out)[(size_t)m * p.N + n] = from_f32<T>(f);
  }
}

template <class T, int WPR>
cudaError_t gemv(const LoraArgs& p, cudaLaunchConfig_t cfg) {
  constexpr int kRows = kGemvThreads / 32 / WPR;
  cfg.blockDim = dim3(kGemvThreads);
  cfg.gridDim = dim3((p.N + kRows - 1) / kRows);
  cfg.dynamicSmemBytes = 0;
  auto* k = p.M == 1 ? lora_gemv_kernel<T, 1, WPR> : lora_gemv_kernel<T, 2, WPR>;
  return cudaLaunchKernelEx(&cfg, k, p);
}

template <class T>
cudaError_t run_gemv(const LoraArgs& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.K <= 2048   ? gemv<T, 1>(p, cfg)
         : p.K <= 4096 ? gemv<T, 2>(p, cfg)
                       : gemv<T, 4>(p, cfg);
}

}  // namespace

// Tiles and pairs for a problem (SMs of a GB300: the workspace size must not depend on the
// device).  Up to 128 tokens are one tile and one CTA a unit; more go to CTA pairs, with the
// tile width whose last round of units leaves the least idle.
LoraPlan lora_plan(int M, int K, int N, int R, bool has_w) {
  LoraPlan L;
  const int sms = 152;
  const int ksteps = (K + 63) / 64;
  L.ksteps = has_w ? ksteps : 0;
  if (M <= 128) {
    L.cg = 1;
    L.tile_n = (M + 15) / 16 * 16;
    L.tiles = 1;
  } else {
    L.cg = 2;
    long long best = -1;
    for (int tn = kMostTokens; tn >= 128; tn -= 16) {
      const long long tiles = (M + tn - 1) / tn, units = tiles * ((N + 255) / 256);
      const long long rounds = (units + sms / 2 - 1) / (sms / 2);
      const long long cost = rounds * (tn + 16);
      if (best < 0 || cost < best) {
        best = cost;
        L.tile_n = tn;
        L.tiles = (int)tiles;
      }
    }
  }
  L.blocks = (N + 128 * L.cg - 1) / (128 * L.cg);
  // the fp32 shrink reads a token's adapter anew for each token: up to 16 MB of such reads
  // (at 33 MB, M = 256, K = N = 4096, R = 16, a call takes 19.8 us with the tensor cores
  // and 22.7 without, at 17 MB 18.3 and 17.8), and what runs as plain products throughout
  L.tensor_shrink = M > kGemvTokens && (long long)M * R * K * 2 > (16LL << 20);
  L.tsplits = 1;
  if (L.tensor_shrink) {
    const int most = ksteps / 4 < kShrinkSegments ? ksteps / 4 : kShrinkSegments;
    const int s = sms / L.tiles < most ? sms / L.tiles : most;
    L.tsplits = s < 1 ? 1 : s;
  }
  return L;
}

cudaError_t launch_lora(LoraArgs& p, int num_sms, cudaStream_t stream) {
  const cudaError_t e = launch_lora_shrink(p, num_sms, stream);
  if (e != cudaSuccess) return e;
  if (p.M > kGemvTokens) return launch_lora_gemm(p, num_sms, stream);
  return p.dtype == QMOE_DTYPE_BF16 ? run_gemv<__nv_bfloat16>(p, stream)
                                    : run_gemv<__half>(p, stream);
}

}  // namespace qmoe
