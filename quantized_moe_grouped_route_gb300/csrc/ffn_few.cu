// The gated feed-forward block for a decode batch (9 to 256 tokens), forward: the weights are the
// rows of the MMA and the tokens its columns, so a product is one pass over the weights.
//
// A unit is 128 rows of weights (64 of u and the same 64 of g in the first product) by all tokens.
// Units are fewer than SMs, so a cluster of S CTAs shares one: each takes a segment of K through a
// ring of TMA-loaded stages into an accumulator in TMEM (tcgen05, M = 128, N = tokens), puts its
// sums into shared memory, and the CTAs add up each other's by distributed shared memory, every CTA
// the tokens seg, seg + S, ..; the order of the sums is fixed.  Bound by the stream of the weights;
// up to 128 tokens two CTAs fit an SM, so that the second product's first weights are already on
// their way while the first product ends (its launch is programmatic, and only the tokens' copies
// wait).
// 48 tokens, H = 7168, I = 2048: 22.5 us in a graph (the weights' stream 13.2); 4096 x 1536: 14.8 (5.7).
#include "cluster.cuh"
#include "ffn.cuh"
#include "mma.cuh"

namespace qmoe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxStages = 8;
constexpr int kCtrl = 1024;
constexpr int kWeightBytes = 128 * 128;  // a stage's 128 rows x 64 of K
constexpr int kSmemHalf = 115712, kSmemLimit = 232448;  // two CTAs an SM, one
constexpr int kMaxSplits = 4;

struct Maps {
  CUtensorMap x, w, w2;
};

template <class T, bool UP>
__global__ void __launch_bounds__(kThreads) ffn_few_kernel(const __grid_constant__ Maps maps,
                                                           const FfnFew p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int stage_bytes = kWeightBytes + p.tile_n * 128;
  const int stages = p.stages, S = p.splits;
  uint8_t* ctrl = smem + p.ring_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(ctrl);
  uint64_t* empty = full + kMaxStages;
  uint64_t* accf = empty + kMaxStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(accf + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int seg = S > 1 ? (int)cluster_rank() : 0;
  const int row0 = (int)blockIdx.x / S * (UP ? 64 : 128);
  const int k0 = (int)((long long)p.ksteps * seg / S), k1 = (int)((long long)p.ksteps * (seg + 1) / S);
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(accf), 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.x);
    prefetch_tmap(&maps.w);
    if (UP) prefetch_tmap(&maps.w2);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), p.tmem_cols);
    tmem_relinquish();
  }
  // The second product's kernel starts while the first runs, once that has waited for what came
  // before the call: by then the weights are complete, whoever wrote them, and can be copied.
  if (UP) {
    grid_dep_wait();
    grid_dep_launch();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    const uint32_t lead = elect_one();
    const uint64_t pol_w = l2_policy_evict_first(), pol_x = l2_policy_evict_last();
    const uint32_t base = smem_u32(smem);
    auto weights = [&](int k, int s) {
      const uint32_t at = base + s * stage_bytes, bar = smem_u32(&full[s]);
      mbar_arrive_expect_tx_if(lead, bar, (uint32_t)stage_bytes);
      tma_load_2d_if(lead, at, &maps.w, k * 64, row0, bar, pol_w);
      if (UP) tma_load_2d_if(lead, at + kWeightBytes / 2, &maps.w2, k * 64, row0, bar, pol_w);
    };
    auto tokens = [&](int k, int s) {
      tma_load_2d_if(lead, base + s * stage_bytes + kWeightBytes, &maps.x, k * 64, 0,
                     smem_u32(&full[s]), pol_x);
    };
    const int first = min(stages, k1 - k0);
    for (int i = 0; i < first; ++i) weights(k0 + i, i);
    if (!UP) grid_dep_wait();
    for (int i = 0; i < first; ++i) tokens(k0 + i, i);
    bool ok = true;
    int s = 0;
    uint32_t ph = 0;
    for (int k = k0 + first; k < k1; ++k) {
      if (!warp_wait(smem_u32(&empty[s]), ph, abort_flag, p.err)) {
        ok = false;
        break;
      }
      weights(k, s);
      tokens(k, s);
      if (++s == stages) {
        s = 0;
        ph ^= 1;
      }
    }
    if (!ok) {  // the copies of the last steps may still be landing
      const unsigned long long t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 2000000ull) {
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issue
    const uint32_t lead = elect_one();
    const uint32_t idesc = idesc_16bit(128, p.tile_n, p.dtype);
    const uint64_t desc0 = sdesc_sw128(smem_u32(smem));
    int s = 0;
    uint32_t ph = 0;
    for (int k = k0; k < k1; ++k) {
      if (!warp_wait(smem_u32(&full[s]), ph, abort_flag, p.err)) break;
      tc_fence_after();
      const uint64_t a = desc0 + ((s * stage_bytes) >> 4);
      if (lead) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mma_ss(1, tmem, a + 2 * j, a + (kWeightBytes >> 4) + 2 * j, idesc, (k > k0) | (j > 0));
      }
      tc_commit_if(lead, smem_u32(&empty[s]));
      if (++s == stages) {
        s = 0;
        ph ^= 1;
      }
    }
    tc_commit_if(lead, smem_u32(accf));
  }
  // every thread: the accumulator is complete, and with it the ring is idle
  bool ok = warp_wait(smem_u32(accf), 0, abort_flag, p.err);
  tc_fence_after();
  float* sums = reinterpret_cast<float*>(smem);  // [token][128]
  if (ok) {
    const int q = warp & 3, half = warp >> 2;  // two warps a lane quarter, columns in turn
    const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16);
    for (int c = 16 * half; c < p.M; c += 32) {
      uint32_t r[16];
      tmem_ld_x16(tbase + c, r);
      tmem_wait_ld();
      tmem_ld_ready(r);
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (c + k < p.M) sums[(c + k) * 128 + q * 32 + lane] = __uint_as_float(r[k]);
    }
  }
  if (!UP) {  // what follows writes memory that earlier kernels may still read
    grid_dep_wait();
    grid_dep_launch();
  }
  if (p.clear_err && blockIdx.x == 0 && threadIdx.x == 0) *p.err = 0;
  tc_fence_before();
  __syncthreads();
  if (S > 1) cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
  const uint32_t sums0 = smem_u32(sums) + 16 * lane;
  const int n = row0 + 4 * lane;
  const bool gelu = p.activation == QMOE_ACT_GELU;
  for (int c = seg + S * warp; c < p.M; c += S * (kThreads / 32)) {
    float4 v[kMaxSplits];
#pragma unroll
    for (int i = 0; i < kMaxSplits; ++i)
      if (i < S)
        v[i] = S > 1 ? ld_cluster_f32x4(peer_addr(sums0 + c * 512, i))
                     : reinterpret_cast<const float4*>(sums + c * 128)[lane];
    float4 t = v[0];
#pragma unroll
    for (int i = 1; i < kMaxSplits; ++i)
      if (i < S) t.x += v[i].x, t.y += v[i].y, t.z += v[i].z, t.w += v[i].w;
    float f[4] = {t.x, t.y, t.z, t.w};
    if (UP) {  // lanes 0..15 have rows of u, 16..31 those of g
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float gate = __shfl_down_sync(0xffffffffu, f[e], 16);
        f[e] = gated(gelu, p.limit, f[e], gate);
      }
    }
    Pack<T, 4> o;
#pragma unroll
    for (int e = 0; e < 4; ++e) o.v[e] = from_f32<T>(f[e]);
    if (n < p.N && (!UP || lane < 16))
      *reinterpret_cast<uint2*>(reinterpret_cast<T*>(p.out) + (size_t)c * p.N + n) = o.raw;
  }
  // No CTA leaves while its sums may still be read; every value fetched above has gone into a
  // store, so the barrier need not order memory.
  if (S > 1) cluster_sync_relaxed();
}

template <class T, bool UP>
cudaError_t run(const FfnProduct& f, int num_sms, cudaStream_t stream) {
  FfnFew p = {};
  static_cast<FfnProduct&>(p) = f;
  p.tile_n = (f.M + 15) / 16 * 16;
  p.ksteps = (f.K + 63) / 64;
  p.tmem_cols = p.tile_n <= 32 ? 32 : p.tile_n <= 64 ? 64 : p.tile_n <= 128 ? 128 : 256;
  const int units = UP ? (f.N + 63) / 64 : (f.N + 127) / 128, stage = kWeightBytes + p.tile_n * 128;
  // Segments of two steps or more, four at most, as many as there are SMs for: more of them cost
  // the adding up what they save.  us a call in a graph by at most 2, 3, 4, 6 and 8 segments:
  //   48 tokens, 4096 x 1536: 18.0, 15.7, 14.8, 15.0, 15.0;  7168 x 2048: 26.5, 23.3, 22.5, 22.7, 23.0
  //   128 tokens, 4096 x 1536: 26.4, 21.8, 19.3, 20.2, 20.3;  7168 x 2048: 37.6, 31.7, 28.4, 28.7, 29.4
  p.splits = 1;
  while (p.splits < kMaxSplits && units * (p.splits + 1) <= num_sms &&
         p.ksteps >= 2 * (p.splits + 1))
    ++p.splits;
  const int limit = p.tile_n <= 128 ? kSmemHalf : kSmemLimit, other = 1024 + kCtrl;
  const int most = (limit - other) / stage;
  p.stages = most < kMaxStages ? most : kMaxStages;
  const int need = p.tile_n * 512;  // the sums
  p.ring_bytes = p.stages * stage > need ? p.stages * stage : need;
  Maps m = {};
  const T* w = reinterpret_cast<const T*>(f.b);
  bool ok = map_of(&m.x, f.dtype, f.a, f.M, f.K, f.lda, p.tile_n) &&
            map_of(&m.w, f.dtype, w, f.N, f.K, f.K, UP ? 64 : 128);
  m.w2 = m.w;
  if (UP) ok = ok && map_of(&m.w2, f.dtype, w + (size_t)f.N * f.K, f.N, f.K, f.K, 64);
  if (!ok) return cudaErrorInvalidValue;
  auto* k = ffn_few_kernel<T, UP>;
  cudaError_t e = allow_smem(k, kSmemLimit);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2] = {pdl_attribute()};
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(units * p.splits));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = other + p.ring_bytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = p.splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k, m, p);
}

}  // namespace

cudaError_t launch_ffn_few(const FfnProduct& f, int num_sms, cudaStream_t stream) {
  const bool up = f.op == FfnOp::kUp;
  if (f.dtype == QMOE_DTYPE_BF16)
    return up ? run<__nv_bfloat16, true>(f, num_sms, stream)
              : run<__nv_bfloat16, false>(f, num_sms, stream);
  return up ? run<__half, true>(f, num_sms, stream) : run<__half, false>(f, num_sms, stream);
}

}  // namespace qmoe
