// A shared projection with a low-rank adapter per token:
//   t[m] = scales[a] * (x[m] . A[a]^T),  out[m] = base[m] + x[m] . w^T + t[m] . B[a]^T
// with a = adapter_ids[m].
//
// Two kernels.  The first (shrink, lora_shrink.cu: plain fp32 products for few tokens, tensor
// cores for many) forms t in fp32 and lists, for each tile of tokens, the distinct adapters
// its tokens use.  The second (lora_gemm.cu) is one GEMM whose contraction runs over K and
// then over the ranks of the tile's adapters: the MMA's M side
// is 128 rows of w (or of B[a]), its N side a tile of up to 256 tokens, and for each of
// the tile's adapters the token operand is t with the rows of other adapters zero.  So the
// adapters cost a tile (distinct adapters) * ranks more of contraction length, whatever
// the order of the tokens, and the result is rounded once.  A zero row times an infinity or
// NaN of another token's B is NaN; what such a B spoils is found and made anew (lora.cuh), so
// that it reaches its own tokens only: 2047 tokens, K = N = 4096, R = 16 of a few requests take
// 54 us, 370 with a NaN in one row of an adapter in use and 520 with all of it NaN.  The two
// forms below keep tokens apart.
//
// t enters the tensor cores as the sum of two values of the activation type (t rounded,
// and what the rounding left) for twice the MMAs of a contraction that is short, instead of a
// second rounding of the result's size.  That holds 16 significant bits of a bf16 t.  Of an
// fp16 t it holds 22 from 2^-3 on, fewer below, where what is left runs into the subnormals,
// and none above 65504; so eight ranks of a token whose largest is below 2^-9 or beyond fp16's
// range enter as zeros, and the epilogue adds their products in fp32 (load_t8_split).  A batch
// of such tokens only is slower (2047 tokens, K = N = 4096, R = 16: 133 us a call for 54).
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
//               slots of their own; one to four warps (the more, the longer a slot's rows)
//               build a step, so that several steps are in the making at once
//
// Few tokens of few ranks (VEC: at most 64 tokens, tokens * ranks at most 512 or, where there
// are adapters enough for one each, 1024: a decode step's requests) do not take the adapters
// through the MMA, where each is a step for one or two tokens.  There warp 2
// brings in B[a]'s rows, which lie next to each other, as one bulk copy each, while w
// streams; the builder warps multiply them with t in fp32, and the epilogue adds what they
// leave in shared memory.
//
// Few tokens (one tile): one CTA per unit, w streamed once, HBM bound.  More: CTA pairs
// (cta_group::2, M = 256), each SM loading half of the token rows, since a 128 x 256 tile
// fed by one SM alone asks more of its L2 port (96 bytes a clock) than it has.
//
// Up to eight tokens w is streamed without any staging (lora_gemv_kernel: one token, plain
// products; lora_stream_kernel: MMAs on fragments straight from memory).
//
// Every wait is bounded, as in the layer's GEMMs.
#include "lora.cuh"

namespace qmoe {
namespace {

// ------------------------------------------------------------------------------ one token
// One, two or four warps (WPR, the more, the longer the row) per row of w: its product with
// the token's row in fp32, then the row of the token's B with t.  HBM (or L2) bound, and
// there is nothing to set up.  What hides the loads' latency is warps, not loads a warp: with
// few registers all rows of w are resident at once (K = 7168, N = 2048: two loads in flight a
// lane and 16 blocks an SM 7.1 us a call, eight loads and 8 blocks 9.6; the kernel below 9.2,
// the tensor-core GEMM 11.4, of which it spends 5 on barriers, TMEM and its cluster).
constexpr int kGemvThreads = 128;

template <class T, int WPR>
__global__ void __launch_bounds__(kGemvThreads, 16) lora_gemv_kernel(const LoraArgs p) {
  using P_ = Pack<T, 8>;
  __shared__ float part[kGemvThreads / 32];
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % WPR;
  const int n = blockIdx.x * (kGemvThreads / 32 / WPR) + warp / WPR;
  const bool here = n < p.N;  // the warp's row (the others only wait for the shrink kernel)
  int id = here && sub == 0 ? p.ids[0] : -1;
  if (id >= p.L) id = -1;
  T b[4];  // ranks lane, lane + 32, ..
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (id >= 0 && lane + 32 * i < p.R)
      b[i] = reinterpret_cast<const T*>(p.b)[((size_t)id * p.N + n) * p.R + lane + 32 * i];
  float acc = 0.f;
  if (here && p.w) {
    const uint4* w = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(p.w) + (size_t)n * p.K);
    const uint4* x = reinterpret_cast<const uint4*>(p.x);
    const int chunks = p.K / 8;
    constexpr int kFlight = 2;
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
        P_ xv;
        xv.raw = x[c];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc = fmaf(to_f32(wv[i].v[e]), to_f32(xv.v[e]), acc);
      }
    }
  }
  grid_dep_wait();  // t (one token has one segment)
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.bad[0]) atomicOr(p.err, QMOE_FLAG_BAD_ID);
  if (id >= 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 32 * i < p.R) acc = fmaf(to_f32(b[i]), p.t[lane + 32 * i], acc);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (lane == 0) part[warp] = acc;
  __syncthreads();
  if (here && sub == 0 && lane == 0) {
    float f = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) f += part[warp + w];
    if (p.base) f += to_f32(reinterpret_cast<const T*>(p.base)[n]);
    reinterpret_cast<T*>(p.out)[n] = from_f32<T>(f);
  }
}

template <class T, int WPR>
cudaError_t gemv(const LoraArgs& p, cudaLaunchConfig_t cfg) {
  constexpr int kRows = kGemvThreads / 32 / WPR;
  cfg.blockDim = dim3(kGemvThreads);
  cfg.gridDim = dim3((p.N + kRows - 1) / kRows);
  return cudaLaunchKernelEx(&cfg, lora_gemv_kernel<T, WPR>, p);
}

// --------------------------------------------------------------------- two to eight tokens
// A block per 16 rows of w, its warps sharing out K: w goes straight from memory into the
// fragments of m16n8k16 (rows of w on M, the tokens on N), which here are dot-product units
// for a stream of w: nothing is staged, so nothing has to be set up.  A lane's 16 bytes (8
// of K) feed two MMAs, four elements each; the token rows are read the same way, so both
// operands see the same order of K.  Then the warps multiply the adapters' rows of B with t
// in fp32, the tokens and (with fewer tokens than warps) the ranks shared out, and all sums
// are added in order.  Whole calls at K = N = 4096, R = 16: 8.2 us at two tokens, 8.5 at
// eight (the tensor-core GEMM 11.9 and 12.5; plain products as above 10.0 at two).  Above
// eight tokens a second fragment's loads of the token rows cost more than the GEMM's set-up
// (K = 7168, N = 2048, 16 tokens: 14.0 against 11.4).
constexpr int kStreamTokens = 8, kStreamWarps = 16;

template <class T>
__global__ void __launch_bounds__(32 * kStreamWarps, 2) lora_stream_kernel(const LoraArgs p) {
  constexpr int kFlight = 4;
  __shared__ float part[kStreamWarps][kStreamTokens][17];
  __shared__ float delta[kStreamWarps][16];
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int n0 = blockIdx.x * 16;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  if (p.w) {
    const int g = lane >> 2, t = lane & 3;  // fragment rows g, g + 8, token g; 8 of K at 8 t
    const T* w = reinterpret_cast<const T*>(p.w) + (size_t)(n0 + g) * p.K + t * 8;
    const T* x = reinterpret_cast<const T*>(p.x) + (long long)g * p.ldx + t * 8;
    const bool row0 = n0 + g < p.N, row1 = n0 + g + 8 < p.N;
    const int steps = (p.K + 31) / 32;
    for (int s0 = warp; s0 < steps; s0 += warps * kFlight) {
      uint4 a[kFlight][2], xv[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        const int k = (s0 + i * warps) * 32;
        const bool in = k + t * 8 < p.K;
        a[i][0] = load_if(reinterpret_cast<const uint4*>(in && row0 ? w + k : p.w), in && row0);
        a[i][1] = load_if(
            reinterpret_cast<const uint4*>(in && row1 ? w + (size_t)8 * p.K + k : p.w), in && row1);
        xv[i] = make_uint4(0u, 0u, 0u, 0u);
        if (in && g < p.M) xv[i] = *reinterpret_cast<const uint4*>(x + k);
      }
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        mma_m16n8k16<T>(acc, a[i][0].x, a[i][1].x, a[i][0].y, a[i][1].y, xv[i].x, xv[i].y);
        mma_m16n8k16<T>(acc, a[i][0].z, a[i][1].z, a[i][0].w, a[i][1].w, xv[i].z, xv[i].w);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    part[warp][2 * (lane & 3) + (e & 1)][(lane >> 2) + 8 * (e >> 1)] = acc[e];
  // adapters: warp -> token warp % m2 (m2: a power of two from M on) and share warp / m2 of
  // its ranks; two lanes per row of B, 8 ranks at a time each.  (Fetching B before w, or
  // before t is due, costs the stream of w registers: 9.6 and 9.2 us for 8.2.)
  int m2 = 1;
  while (m2 < p.M) m2 *= 2;
  const int m = warp % m2, share = warp / m2, shares = warps / m2;
  const int row = lane >> 1, n = n0 + row, r0 = 8 * (2 * share + (lane & 1)), dr = 16 * shares;
  int id = m < p.M ? p.ids[m] : -1;
  if (id >= p.L || n >= p.N) id = -1;
  const T* b = reinterpret_cast<const T*>(p.b) + ((size_t)(id < 0 ? 0 : id) * p.N + n) * p.R;
  grid_dep_wait();  // t
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.bad[0]) atomicOr(p.err, QMOE_FLAG_BAD_ID);
  float d = 0.f;
  if (id >= 0) {
#pragma unroll 2
    for (int r = r0; r < p.R; r += dr) {
      Pack<T, 8> v;
      v.raw = *reinterpret_cast<const uint4*>(b + r);
      float f[8];
      load_t8(p, m, r, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) d = fmaf(to_f32(v.v[e]), f[e], d);
    }
  }
  d += __shfl_xor_sync(0xffffffffu, d, 1);
  if ((lane & 1) == 0) delta[warp][row] = d;
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * p.M; i += blockDim.x) {
    const int tok = i / 16, r = i % 16;
    if (n0 + r >= p.N) continue;
    float f = 0.f;
    for (int v = 0; v < warps; ++v) f += part[v][tok][r];
    for (int v = tok; v < warps; v += m2) f += delta[v][r];
    if (p.base) f += to_f32(reinterpret_cast<const T*>(p.base)[tok * p.ldbase + n0 + r]);
    reinterpret_cast<T*>(p.out)[(size_t)tok * p.N + n0 + r] = from_f32<T>(f);
  }
}

template <class T>
cudaError_t run_few(const LoraArgs& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.M == 1)
    return p.K <= 2048   ? gemv<T, 1>(p, cfg)
           : p.K <= 4096 ? gemv<T, 2>(p, cfg)
                         : gemv<T, 4>(p, cfg);
  // a warp for every 256 of K (8 steps), eight at least for the adapters' share
  const int warps = p.K < 4096 ? 8 : kStreamWarps;
  cfg.blockDim = dim3(32 * warps);
  cfg.gridDim = dim3((p.N + 15) / 16);
  return cudaLaunchKernelEx(&cfg, lora_stream_kernel<T>, p);
}

}  // namespace

// SMs of a GB300: the workspace size must not depend on the device.
constexpr int kPlanSms = 152;

// Whether x . A^T goes through the tensor cores: the fp32 shrink reads a token's adapter anew
// for each token, so up to 16 MB of such reads (at 33 MB, M = 256, K = N = 4096, R = 16, a call
// takes 19.8 us with the tensor cores and 22.7 without, at 17 MB 18.3 and 17.8) do not, nor
// does a single token.
static bool tensor_shrink(int M, int K, int R) {
  return M > 1 && (long long)M * R * K * 2 > (16LL << 20);
}
// Segments of K in that form, at most.
static int most_segments(int K) {
  const int s = (K + 63) / 64 / 4;
  return s < 1 ? 1 : s < kShrinkSegments ? s : kShrinkSegments;
}

// A plan has kPlanSms / tiles segments, or one.
size_t lora_segment_rows(int M, int K, int R) {
  if (!tensor_shrink(M, K, R)) return M;
  const size_t rows = (size_t)M * most_segments(K), full = (size_t)kPlanSms * kMostTokens;
  const size_t split = rows < full ? rows : full;
  return split > (size_t)M ? split : M;
}

// Tiles and pairs for a problem.  Up to 128 tokens are one tile and one CTA a unit; more go to CTA pairs, with the
// tile width whose last round of units leaves the least idle.
LoraPlan lora_plan(int M, int K, int N, int R, bool has_w) {
  LoraPlan L;
  const int sms = kPlanSms;
  const int ksteps = (K + 63) / 64;
  L.ksteps = has_w ? ksteps : 0;
  if (M <= 128) {
    L.cg = 1;
    L.tile_n = (M + 15) / 16 * 16;
    L.tiles = 1;
  } else {
    L.cg = 2;
    long long best = -1;
    for (int tn = kMostTokens; tn >= kLoraLeastTile; tn -= 16) {
      const long long tiles = (M + tn - 1) / tn, units = tiles * ((N + 255) / 256);
      const long long rounds = (units + sms / 2 - 1) / (sms / 2);
      if (rounds > 1 && tn > kMostInRounds) continue;
      const long long cost = rounds * (tn + 16);
      if (best < 0 || cost < best) {
        best = cost;
        L.tile_n = tn;
        L.tiles = (int)tiles;
      }
    }
  }
  L.blocks = (N + 128 * L.cg - 1) / (128 * L.cg);
  L.tensor_shrink = tensor_shrink(M, K, R);
  L.tsplits = 1;
  if (L.tensor_shrink) {
    const int most = most_segments(K), s = kPlanSms / L.tiles < most ? kPlanSms / L.tiles : most;
    L.tsplits = s < 1 ? 1 : s;
  }
  return L;
}

cudaError_t launch_lora(LoraArgs& p, int num_sms, cudaStream_t stream) {
  const cudaError_t e = launch_lora_shrink(p, num_sms, stream);
  if (e != cudaSuccess) return e;
  if (p.M > kStreamTokens) return launch_lora_gemm(p, num_sms, stream);
  return p.dtype == QMOE_DTYPE_BF16 ? run_few<__nv_bfloat16>(p, stream)
                                    : run_few<__half>(p, stream);
}

}  // namespace qmoe
