// The first step of the projection with adapters: t[m] = scales[a] * (x[m] . A[a]^T), and the
// lists of the distinct adapters of each tile of tokens.
#include "lora.cuh"

namespace qmoe {
namespace {

// ------------------------------------------------------------------ shrink, few tokens
// A block per (token, 8 ranks) with a thread per 8 elements of K (up to 1024), so that a
// single token's latency is about one round trip to memory; the eight sums are reduced in
// a fixed order.  The blocks before them list the tiles' adapters (one block each) and zero
// the error word.
constexpr int kShrinkThreads = 256;

// The distinct valid ids of a tile's tokens, in order of first appearance, into list
// (shared, one entry per token of the tile); whole block of at least kShrinkThreads, after
// clear_lists and a barrier.  Returns their count; *mine is this thread's token's place in
// the list (-1: none), *bad whether any of the tile's ids is L or more.
//
// The first token of each id is the least that a table of ids ends up with, whatever order
// they arrive in; a warp enters each of its ids once.  (Every token against every other one
// took 2 us more at 240 tokens.)
constexpr int kTable = 2 * kShrinkThreads;  // entries, a power of two: at most half are taken
struct ListScratch {
  int key[kTable], first[kTable];
  int place[kShrinkThreads], warp_count[kShrinkThreads / 32];
};
__device__ __forceinline__ void clear_lists(ListScratch& w) {
  for (int i = threadIdx.x; i < kTable; i += blockDim.x) {
    w.key[i] = -1;
    w.first[i] = kShrinkThreads;
  }
}
__device__ __forceinline__ int list_adapters(const int32_t* __restrict__ ids, int m0, int rows,
                                             int L, ListScratch& w, int* list, int* mine,
                                             bool* bad) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool here = tid < kShrinkThreads;
  int id = tid < rows ? ids[m0 + tid] : -1;
  const bool high = id >= L;
  if (high || id < 0) id = -1;
  const unsigned same = __match_any_sync(0xffffffffu, id);
  const int head = __ffs(same) - 1;  // the warp's first token with this id
  int at = 0;
  if (id >= 0 && lane == head) {
    at = (int)((uint32_t)id * 2654435761u >> 16) & (kTable - 1);
    for (int probe = 0; probe < kTable; ++probe) {  // (no more ids than tokens: a place is found)
      const int was = atomicCAS(&w.key[at], -1, id);
      if (was == -1 || was == id) break;
      at = (at + 1) & (kTable - 1);
    }
    atomicMin(&w.first[at], tid);
  }
  at = __shfl_sync(0xffffffffu, at, head);
  *bad = __syncthreads_or(high);
  const int lead = w.first[at];  // the first token with this id
  const bool first = id >= 0 && lead == tid;
  const unsigned mask = __ballot_sync(0xffffffffu, first);
  if (here && lane == 0) w.warp_count[warp] = __popc(mask);
  __syncthreads();
  int before = 0, total = 0;
  for (int i = 0; i < kShrinkThreads / 32; ++i) {
    if (i < warp) before += w.warp_count[i];
    total += w.warp_count[i];
  }
  if (first) {
    w.place[tid] = before + __popc(mask & ((1u << lane) - 1u));
    list[w.place[tid]] = id;
  }
  __syncthreads();
  *mine = id >= 0 ? w.place[lead] : -1;
  return total;
}

// What the GEMM needs of the lists; by one block per tile.
__device__ __forceinline__ void publish_list(const LoraArgs& p, int t, const int* list, int n,
                                             int mine, bool bad) {
  const int tid = threadIdx.x;
  if (tid < p.tile_n) {
    p.place[(size_t)t * p.tile_n + tid] = mine;
    p.left[(size_t)t * p.tile_n + tid] = 0u;
  }
  if (t == 0 && tid == 0) p.err[0] = 0u;
  for (int i = tid; i < n; i += blockDim.x) p.list[(size_t)t * p.tile_n + i] = list[i];
  if (tid == 0) {
    p.count[t] = n;
    p.bad[t] = bad;
    p.any_left[t] = 0u;
  }
}

constexpr int kShrinkMost = 1024;  // threads of the plain shrink
template <class T>
__global__ void __launch_bounds__(kShrinkMost) lora_shrink_kernel(const LoraArgs p) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int kWarps = kShrinkMost / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if ((int)blockIdx.x < p.tiles) {
    __shared__ ListScratch scratch;
    __shared__ int list[kShrinkThreads];
    const int t = blockIdx.x, m0 = t * p.tile_n;
    clear_lists(scratch);
    __syncthreads();
    int mine;
    bool bad;
    const int n =
        list_adapters(p.ids, m0, min(p.tile_n, p.M - m0), p.L, scratch, list, &mine, &bad);
    publish_list(p, t, list, n, mine, bad);
    return;
  }
  __shared__ float part[8][kWarps + 1];
  using P_ = Pack<T, 8>;
  const int groups = p.R / 8;
  const long long it = (long long)blockIdx.x - p.tiles;
  const int m = (int)(it / groups), r0 = (int)(it % groups) * 8;
  const int id = p.ids[m];
  const bool has = id >= 0 && id < p.L;
  const float scale = has ? p.scales[id] : 0.f;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (has) {
    const uint4* x = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(p.x) + m * p.ldx);
    const uint4* a =
        reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(p.a) + ((size_t)id * p.R + r0) * p.K);
    const int chunks = p.K / 8;
    for (int c = tid; c < chunks; c += blockDim.x) {
      P_ xv, av[8];
      xv.raw = x[c];
#pragma unroll
      for (int r = 0; r < 8; ++r) av[r].raw = a[(size_t)r * chunks + c];
#pragma unroll
      for (int r = 0; r < 8; ++r)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[r] = fmaf(to_f32(xv.v[i]), to_f32(av[r].v[i]), acc[r]);
    }
  }
#pragma unroll
  for (int r = 0; r < 8; ++r) {
#pragma unroll
    for (int o = 16; o; o >>= 1) acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], o);
    if (lane == 0) part[r][warp] = acc[r];
  }
  __syncthreads();
  if (warp < 8) {  // a warp per rank: at least 8 warps a block, at most 32
    float s = lane < (int)(blockDim.x >> 5) ? part[warp][lane] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0 && has) p.t[(size_t)m * p.R + r0 + warp] = s * scale;
  }
}

// ----------------------------------------------------------------- shrink, many tokens
// A CTA per (token tile, K segment): D[rank of adapter][token] = A[a] . x^T on the tensor
// cores, with the 128 / R adapters of a pass stacked on the MMA's 128 rows, so that a tile
// of few adapters (requests one after another) takes one pass over its token rows.  Each
// token keeps the rows of its own adapter; the GEMM adds up the segments where it takes t
// up (adding them here, through a cluster's shared memory, cost more than the reads it
// saved, and 37 tiles of four segments did not fit as clusters: at M = 8192, K = 7168 31 us).
// gridDim.y CTAs share a tile's passes.
constexpr int kShrinkMostStages = 6;
constexpr int kShrinkRing = kSmemLimit - 10240;  // bytes at most, less the lists
__host__ __device__ constexpr int shrink_stage_bytes(int tile_n) { return kStageA + tile_n * 128; }
__host__ __device__ constexpr int shrink_stages(int tile_n) {
  const int n = kShrinkRing / shrink_stage_bytes(tile_n);
  return n < kShrinkMostStages ? n : kShrinkMostStages;
}

template <class T>
__global__ void __launch_bounds__(kShrinkThreads, 1)
    lora_shrink_mma_kernel(const __grid_constant__ CUtensorMap map_x,
                           const __grid_constant__ CUtensorMap map_a, const LoraArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ ListScratch scratch;
  __shared__ int list[kShrinkThreads];
  __shared__ __align__(16) int place[kShrinkThreads];
  __shared__ __align__(8) uint64_t full[kShrinkMostStages], empty[kShrinkMostStages], accf,
      acce, drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stage_bytes = shrink_stage_bytes(p.tile_n), stages = shrink_stages(p.tile_n);
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(&accf), 1);
    mbar_init(smem_u32(&acce), 4);
    mbar_init(smem_u32(&drain), 1);
    abort_word = 0;
    fence_mbar_init();
    prefetch_tmap(&map_x);
    prefetch_tmap(&map_a);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), kAccCols);
    tmem_relinquish();
  }
  clear_lists(scratch);
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  const int t = blockIdx.x / p.tsplits, seg = blockIdx.x - t * p.tsplits;
  const int m0 = t * p.tile_n, cols = min(p.tile_n, p.M - m0);
  const int ksteps = (p.K + 63) / 64;
  const int k0 = (int)((long long)ksteps * seg / p.tsplits);
  const int k1 = (int)((long long)ksteps * (seg + 1) / p.tsplits);
  const uint64_t pol = l2_policy_evict_last();  // the GEMM reads the token rows next
  // the first token rows are fetched while the list is made (their bytes count on a phase
  // that the adapters' copies have yet to arrive at)
  const int early = min(stages, k1 - k0);
  if (warp == 0) {
    __syncwarp();
    const uint32_t lead = elect_one();
    for (int i = 0; i < early; ++i)
      tma_load_2d_if(lead, smem_u32(smem) + i * stage_bytes + kStageA, &map_x, (k0 + i) * 64, m0,
                     smem_u32(&full[i]), pol);
  }
  int mine;
  bool bad;
  const int n = list_adapters(p.ids, m0, cols, p.L, scratch, list, &mine, &bad);
  place[threadIdx.x] = mine;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  if (seg == 0 && blockIdx.y == 0) publish_list(p, t, list, n, mine, bad);
  const int cap = 128 / p.R;
  const int passes = (n + cap - 1) / cap;
  if (warp == 0) {
    const uint32_t lead = elect_one();
    uint32_t s = 0, ph = 1;
    bool ok = true;
    int fetched = early;
    for (int ps = blockIdx.y; ps < passes && ok; ps += gridDim.y) {
      const int here = min(cap, n - ps * cap);
      for (int k = k0; k < k1; ++k) {
        if (!warp_wait(smem_u32(&empty[s]), ph, abort_flag, p.err)) {
          ok = false;
          break;
        }
        const uint32_t st = smem_u32(smem) + s * stage_bytes, fb = smem_u32(&full[s]);
        mbar_arrive_expect_tx_if(lead, fb, (uint32_t)(here * p.R * 128 + p.tile_n * 128));
        for (int i = 0; i < here; ++i)
          tma_load_3d_if(lead, st + i * p.R * 128, &map_a, k * 64, 0, list[ps * cap + i], fb, pol);
        if (fetched > 0)
          --fetched;
        else
          tma_load_2d_if(lead, st + kStageA, &map_x, k * 64, m0, fb, pol);
        if (++s == (uint32_t)stages) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    // no adapters in these passes: the early rows are awaited all the same
    for (int i = early - fetched; i < early; ++i) {
      mbar_arrive_expect_tx_if(lead, smem_u32(&full[i]), (uint32_t)p.tile_n * 128);
      warp_wait(smem_u32(&full[i]), 0, abort_flag, p.err);
    }
    if (!ok) {  // the copies of the last steps may still be landing
      const unsigned long long t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 2000000ull) {
      }
    }
  } else if (warp == 1) {
    const uint32_t lead = elect_one();
    const uint32_t idesc = idesc_16bit(128, p.tile_n, p.dtype);
    const uint64_t desc0 = sdesc_sw128(smem_u32(smem));
    uint32_t s = 0, ph = 0, aph = 1;
    bool ok = true;
    for (int ps = blockIdx.y; ps < passes && ok; ps += gridDim.y) {
      if (!warp_wait(smem_u32(&acce), aph, abort_flag, p.err)) break;
      aph ^= 1;
      tc_fence_after();
      for (int k = k0; k < k1; ++k) {
        if (!warp_wait(smem_u32(&full[s]), ph, abort_flag, p.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t a = desc0 + ((s * stage_bytes) >> 4);
        if (lead) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_ss(1, tmem, a + 2 * j, a + (kStageA >> 4) + 2 * j, idesc, k > k0 || j > 0);
        }
        tc_commit_if(lead, smem_u32(&empty[s]));
        if (++s == (uint32_t)stages) {
          s = 0;
          ph ^= 1;
        }
      }
      if (ok) tc_commit_if(lead, smem_u32(&accf));
    }
    tc_commit_if(lead, smem_u32(&drain));
    drain_wait(smem_u32(&drain), 0);
  } else if (warp >= 4) {
    const int q = warp & 3, row = q * 32 + lane;
    const int slot = row / p.R, r = row - slot * p.R;
    uint32_t ph = 0;
    for (int ps = blockIdx.y; ps < passes; ps += gridDim.y) {
      if (!warp_wait(smem_u32(&accf), ph, abort_flag, p.err)) break;
      ph ^= 1;
      tc_fence_after();
      const int want = slot < cap && ps * cap + slot < n ? ps * cap + slot : -2;
      const float scale = want >= 0 ? p.scales[list[want]] : 0.f;
      for (int c0 = 0; c0 < cols; c0 += 16) {
        uint32_t v[16];
        tmem_ld_x16(tmem + ((uint32_t)(q * 32) << 16) + c0, v);
        // the tokens' places ahead of the stores (looked up between them, each store waited
        // for its own: 71 cycles a token); tokens past the tile's end have none
        int4 at[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) at[k] = reinterpret_cast<const int4*>(place + c0)[k];
        tmem_wait_ld();
        tmem_ld_ready(v);
        float* dst = p.t + ((size_t)seg * p.M + m0 + c0) * p.R + r;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (at[k].x == want) dst[(4 * k) * p.R] = __uint_as_float(v[4 * k]) * scale;
          if (at[k].y == want) dst[(4 * k + 1) * p.R] = __uint_as_float(v[4 * k + 1]) * scale;
          if (at[k].z == want) dst[(4 * k + 2) * p.R] = __uint_as_float(v[4 * k + 2]) * scale;
          if (at[k].w == want) dst[(4 * k + 3) * p.R] = __uint_as_float(v[4 * k + 3]) * scale;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&acce));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kAccCols);
  }
}

cudaError_t shrink_maps(const LoraArgs& p, CUtensorMap* x, CUtensorMap* a) {
  const cudaError_t e = map_rows(x, p, p.x, p.K, p.M, p.ldx, p.tile_n);
  return e == cudaSuccess ? map_adapters(a, p, p.a, p.K, p.R, p.R) : e;
}

template <class T>
cudaError_t run(const LoraArgs& p, int num_sms, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (!p.tensor_shrink) {
    int threads = (p.K / 8 + 31) / 32 * 32;
    threads = threads < kShrinkThreads ? kShrinkThreads : threads > kShrinkMost ? kShrinkMost : threads;
    cfg.blockDim = dim3(threads);
    cfg.gridDim = dim3((unsigned)(p.tiles + (long long)p.M * (p.R / 8)));
    return cudaLaunchKernelEx(&cfg, lora_shrink_kernel<T>, p);
  }
  const int ctas = p.tiles * p.tsplits, cap = 128 / p.R;
  const int most = ((p.L < p.tile_n ? p.L : p.tile_n) + cap - 1) / cap;
  const int share = num_sms / ctas < 1 ? 1 : num_sms / ctas;
  cfg.blockDim = dim3(kShrinkThreads);
  cfg.gridDim = dim3(ctas, share < most ? share : most);
  cfg.dynamicSmemBytes = 1024 + shrink_stages(p.tile_n) * shrink_stage_bytes(p.tile_n);
  cudaError_t e = allow_smem(lora_shrink_mma_kernel<T>, 1024 + kShrinkRing);
  if (e != cudaSuccess) return e;
  CUtensorMap map_x, map_a;
  e = shrink_maps(p, &map_x, &map_a);
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, lora_shrink_mma_kernel<T>, map_x, map_a, p);
}

}  // namespace

cudaError_t launch_lora_shrink(const LoraArgs& p, int num_sms, cudaStream_t stream) {
  return p.dtype == QMOE_DTYPE_BF16 ? run<__nv_bfloat16>(p, num_sms, stream)
                                    : run<__half>(p, num_sms, stream);
}

}  // namespace qmoe
