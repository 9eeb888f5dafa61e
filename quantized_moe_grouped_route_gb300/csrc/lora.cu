// A shared projection with a low-rank adapter per token:
//   t[m] = scales[a] * (x[m] . A[a]^T),  out[m] = base[m] + x[m] . w^T + t[m] . B[a]^T
// with a = adapter_ids[m].
//
// Two kernels.  The first (shrink: plain fp32 products for few tokens, tensor cores for
// many) forms the sums x . A^T in fp32 and lists, for each tile
// of tokens, the distinct adapters its tokens use.  The second is one GEMM whose
// contraction runs over K and then over the ranks of the tile's adapters: the MMA's M side
// is 128 rows of w (or of B[a]), its N side a tile of up to 240 tokens, and for each of
// the tile's adapters the token operand is t with the rows of other adapters zero.  So the
// adapters cost a tile (distinct adapters) * ranks more of contraction length, whatever
// the order of the tokens, and the result is rounded once.
//
// t enters the tensor cores as the sum of two values of the activation type (t rounded,
// and what the rounding left): 16 (bf16) or 22 (fp16) significant bits for twice the MMAs
// of a contraction that is short, instead of a second rounding of the result's size.  The
// shrink kernel writes both.
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
// Few tokens of few ranks (VEC: at most 64 tokens, tokens * ranks at most 4096; a decode
// step's requests with an adapter each) do not take the adapters through the MMA: a step
// per adapter moves 128 rows of B[a] for one or two tokens, and the tensor copies took 0.24
// us a step (64-byte rows), 5.3 of the 15.9 us of 48 tokens of 43 adapters.  There warp 2
// brings in B[a]'s rows, which lie next to each other, as one bulk copy each, while w
// streams; the builder warps multiply them with t in fp32, and the
// epilogue adds what they leave in shared memory.
//
// Few tokens (one tile): one CTA per unit, w streamed once, HBM bound.  More: CTA pairs
// (cta_group::2, M = 256), each SM loading half of the token rows, since a 128 x 256 tile
// fed by one SM alone asks more of its L2 port (96 bytes a clock) than it has.
//
// One or two tokens run as plain products, warps per row of w (lora_gemv_kernel).
//
// Every wait is bounded, as in the layer's GEMMs.
#include <atomic>

#include "cluster.cuh"
#include "common.cuh"
#include "launch.h"
#include "pack.cuh"

namespace qmoe {
namespace {

// ------------------------------------------------------------------ shrink, few tokens
// A block per (token, 8 ranks) with a thread per 8 elements of K (up to 1024), so that a
// single token's latency is about one round trip to memory; the eight sums are reduced in
// a fixed order.  The blocks before them list the tiles' adapters (one block each) and zero
// the error word.
constexpr int kShrinkThreads = 256;

// The distinct valid ids of a tile's tokens, in order of first appearance, into list
// (shared, one entry per token of the tile); whole block of at least kShrinkThreads.  Returns their
// count; *mine is this thread's token's place in the list (-1: none), *bad whether its id
// is L or more.
struct __align__(16) ListScratch {
  int id[kShrinkThreads], place[kShrinkThreads], warp_count[kShrinkThreads / 32];
};
__device__ __forceinline__ int list_adapters(const int32_t* __restrict__ ids, int m0, int rows,
                                             int L, ListScratch& w, int* list, int* mine,
                                             bool* bad) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool here = tid < kShrinkThreads;
  int id = tid < rows ? ids[m0 + tid] : -1;
  *bad = id >= L;
  if (id >= L || id < 0) id = -1;
  if (here) w.id[tid] = id;
  __syncthreads();
  int lead = tid;  // the first token with this id
  const int4* four = reinterpret_cast<const int4*>(w.id);
#pragma unroll 4
  for (int i = (rows - 1) / 4; i >= 0; --i) {  // backwards: the last match found is the first
    const int4 v = four[i];
    if (v.w == id) lead = 4 * i + 3;
    if (v.z == id) lead = 4 * i + 2;
    if (v.y == id) lead = 4 * i + 1;
    if (v.x == id) lead = 4 * i;
  }
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
  if (tid < p.tile_n) p.place[(size_t)t * p.tile_n + tid] = mine;
  if (t == 0 && tid == 0) p.err[0] = 0u;
  for (int i = tid; i < n; i += blockDim.x) p.list[(size_t)t * p.tile_n + i] = list[i];
  const bool any = __syncthreads_or(bad);
  if (tid == 0) {
    p.count[t] = n;
    p.bad[t] = any;
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
    int mine;
    bool bad;
    const int n =
        list_adapters(p.ids, m0, min(p.tile_n, p.M - m0), p.L, scratch, list, &mine, &bad);
    publish_list(p, t, list, n, mine, bad);
    return;
  }
  __shared__ float part[kWarps][8];
  using P_ = Pack<T, 8>;
  const int groups = p.R / 8;
  const long long it = (long long)blockIdx.x - p.tiles;
  const int m = (int)(it / groups), r0 = (int)(it % groups) * 8;
  const int id = p.ids[m];
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (id >= 0 && id < p.L) {
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
    if (lane == 0) part[warp][r] = acc[r];
  }
  __syncthreads();
  if (tid < 8) {
    float s = 0.f;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) s += part[w][tid];
    if (id >= 0 && id < p.L) p.t[(size_t)m * p.R + r0 + tid] = s * p.scales[id];
  }
}

// Ranks r .. r + 7 of a token's t, over the shrink's segments of K in order.
__device__ __forceinline__ void load_t8(const LoraArgs& p, int m, int r, float (&t)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) t[e] = 0.f;
  const float* src = p.t + (size_t)m * p.R + r;
#pragma unroll 4
  for (int g = 0; g < p.tsplits; ++g) {
    const float4 a = reinterpret_cast<const float4*>(src + (size_t)g * p.M * p.R)[0];
    const float4 b = reinterpret_cast<const float4*>(src + (size_t)g * p.M * p.R)[1];
    t[0] += a.x, t[1] += a.y, t[2] += a.z, t[3] += a.w;
    t[4] += b.x, t[5] += b.y, t[6] += b.z, t[7] += b.w;
  }
}
// ... as their rounding and what that leaves.
template <class T>
__device__ __forceinline__ void load_t8_split(const LoraArgs& p, int m, int r, uint4* hi,
                                              uint4* lo) {
  float t[8];
  load_t8(p, m, r, t);
  Pack<T, 8> h, l;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    h.v[e] = from_f32<T>(t[e]);
    l.v[e] = from_f32<T>(t[e] - to_f32(h.v[e]));
  }
  *hi = h.raw;
  *lo = l.raw;
}

// ------------------------------------------------------------------------------- GEMM
constexpr int kBuilders = 8;  // warps
constexpr int kGemmThreads = 256 + 32 * kBuilders;
constexpr int kStageA = 128 * 128;  // 128 rows x 64 elements
constexpr int kMaxStages = 12;
constexpr int kAccCols = 256;  // TMEM columns of one accumulator
constexpr int kCtrl = 1024;
constexpr int kEpiStage = 4 * 2048;  // transpose tiles of the epilogue warps: 32 tokens x 32 rows
constexpr int kSmemLimit = 232448;
constexpr int kMostTokens = 240;  // of a tile: five stages of the ring; 256 leave room for four
constexpr int kMaxSplits = 8;  // CTAs of a cluster, at most

// Bytes of one step of a CTA's token rows; slots of the builders' operand (two of them
// each: t rounded, and the rest), fewer the wider the tile.
__host__ __device__ constexpr int token_bytes(int tile_n, int cg) { return tile_n / cg * 128; }
__host__ __device__ constexpr int token_slots(int tile_n, int cg) {
  return tile_n / cg <= 48 ? 8 : tile_n / cg <= 64 ? 4 : 2;
}
// The builders' copy of t for a CTA's token rows (both values), where it takes up to 16 KB:
// every row enters one adapter's step, and the steps then build from shared memory what
// they would each wait for from L2.
__host__ __device__ constexpr int t_copy_bytes(int tile_n, int cg, int R) {
  return cg == 1 && tile_n * R * 4 <= 16384 ? tile_n * R * 4 : 0;
}

// VEC: bytes of an adapter's 128 rows of B, and how many adapters are in flight (64 KB at
// most).  A power of two: step i's slot is i % vec_slots, and the kBuilders / vec_slots warps
// of a slot take all of its steps, since a wait on a phase's parity cannot tell it from the
// phase after the next (six slots among eight warps ran into that and timed out).
constexpr int kVecTokens = 64, kVecTokenRanks = 4096;
__host__ __device__ constexpr int vec_slot_bytes(int R) { return 128 * R * 2; }
__host__ __device__ constexpr int vec_slots(int R) { return R <= 32 ? 8 : R <= 64 ? 4 : 2; }

// Bytes of shared memory behind the ring (multiples of 1024 each): the builders' slots, their
// copy of t, and (VEC) what they leave for the epilogue [tokens][128] in fp32.
struct Behind {
  int slots, copy, delta;
};
__host__ __device__ constexpr int round_kb(int v) { return (v + 1023) / 1024 * 1024; }
__host__ __device__ constexpr Behind behind(bool vec, int tile_n, int cg, int R) {
  Behind b{};
  if (vec) {
    b.slots = round_kb(vec_slots(R) * vec_slot_bytes(R));
    b.copy = round_kb(tile_n * R * 4);
    b.delta = tile_n * 512;
  } else {
    b.slots = 2 * token_slots(tile_n, cg) * token_bytes(tile_n, cg);
    b.copy = round_kb(t_copy_bytes(tile_n, cg, R));
  }
  return b;
}

__device__ __forceinline__ void mma_ss(uint32_t cg, uint32_t d, uint64_t a, uint64_t b,
                                       uint32_t idesc, uint32_t accumulate) {
  if (cg == 1)
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, q;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, q;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor, kind::f16: A and B both bf16 or both fp16, fp32 D.
__device__ __forceinline__ uint32_t idesc_16bit(int M, int N, int dtype) {
  return idesc_bf16_f32(M, N) & (dtype == QMOE_DTYPE_BF16 ? ~0u : ~((1u << 7) | (1u << 10)));
}

// Barrier of the builder warps.
__device__ __forceinline__ void builders_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kBuilders) : "memory");
}

__device__ __forceinline__ void fence_proxy_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
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
constexpr int kShrinkSegments = 8;  // at most
__host__ __device__ constexpr int shrink_stage_bytes(int tile_n) { return kStageA + tile_n * 128; }
__host__ __device__ constexpr int shrink_stages(int tile_n) {
  const int n = (kSmemLimit - 8192) / shrink_stage_bytes(tile_n);  // less the static memory
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
  if (seg == 0 && blockIdx.y == 0) publish_list(p, t, list, n, mine, bad);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
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

template <class T, int CG, bool VEC>
__global__ void __launch_bounds__(kGemmThreads, 1)
    lora_gemm_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                     const __grid_constant__ CUtensorMap map_b, const LoraArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int rows_b = p.tile_n / CG;  // token rows of this CTA
  const int bytes_b = token_bytes(p.tile_n, CG);
  const int stage_bytes = kStageA + bytes_b;
  const int stages = p.stages;
  const int tslots = VEC ? vec_slots(p.R) : token_slots(p.tile_n, CG);
  const Behind behind_ring = behind(VEC, p.tile_n, CG, p.R);
  uint8_t* tbuf = smem + stages * stage_bytes;  // [tslots][2][bytes_b]; VEC [tslots][128][R]
  uint8_t* tcopy = tbuf + behind_ring.slots;    // [rows_b][2][R]; VEC fp32 [rows_b][R]
  const int copy_bytes = t_copy_bytes(p.tile_n, CG, p.R);
  float* delta = reinterpret_cast<float*>(tcopy + behind_ring.copy);  // VEC [tokens][128]
  uint8_t* ctrl = tcopy + behind_ring.copy + behind_ring.delta;
  uint8_t* epi_stage = ctrl + kCtrl;
  uint64_t* full = reinterpret_cast<uint64_t*>(ctrl);
  uint64_t* empty = full + kMaxStages;
  uint64_t* tfull = empty + kMaxStages;
  uint64_t* tempty = tfull + 8;
  uint64_t* accf = tempty + 8;
  uint64_t* acce = accf + 2;
  uint64_t* drain = acce + 2;
  uint64_t* dfull = drain + 1;  // VEC: delta complete (builder warps), read (epilogue warps)
  uint64_t* dempty = dfull + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(dempty + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  short* place = reinterpret_cast<short*>(ctrl + 512);  // [rows_b] the tokens' adapters

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // a cluster: S segments of CG CTAs
  const int S = p.splits;
  const bool clustered = CG * S > 1;
  const uint32_t crank = clustered ? cluster_rank() : 0u;
  const uint32_t rank = crank % CG, lead_rank = crank - rank;
  const int seg = (int)crank / CG;
  const int worker = clustered ? (int)cluster_index() : (int)blockIdx.x;
  const int workers = clustered ? (int)cluster_count() : (int)gridDim.x;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int i = 0; i < tslots; ++i) {
      mbar_init(smem_u32(&tfull[i]), VEC ? 1 : kBuilders / tslots * CG);
      mbar_init(smem_u32(&tempty[i]), VEC ? kBuilders / tslots : 1);
    }
    mbar_init(smem_u32(dfull), kBuilders);
    mbar_init(smem_u32(dempty), 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&accf[i]), 1);
      mbar_init(smem_u32(&acce[i]), 4 * CG);
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if (CG == 2) {
      tmem_alloc2(smem_u32(tmem_slot), 2 * kAccCols);
      tmem_relinquish2();
    } else {
      tmem_alloc(smem_u32(tmem_slot), 2 * kAccCols);
      tmem_relinquish();
    }
  }
  if (threadIdx.x == 0) {
    prefetch_tmap(&map_x);
    prefetch_tmap(&map_w);
    prefetch_tmap(&map_b);
  }
  grid_dep_launch();
  tc_fence_before();
  __syncthreads();
  if (clustered) cluster_sync_all();  // the peer's barriers exist before any remote arrival
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int ksteps = p.ksteps;  // of the shared product; 0 without w
  const int chunks = (p.R + 63) / 64;
  const int units = p.tiles * p.blocks;
  const int k0 = (int)((long long)ksteps * seg / S), k1 = (int)((long long)ksteps * (seg + 1) / S);
  // bounded waits; the pair's barriers take arrivals from both CTAs
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (CG == 2) return warp_wait_cl(smem_u32(bar), parity, abort_flag, p.err);
    return warp_wait(smem_u32(bar), parity, abort_flag, p.err);
  };
  // The tile's adapters d = seg, seg + S, .. < adapters(tile), one step per 64 ranks, follow
  // a segment's K steps.  The shrink kernel writes the lists, so it is awaited first.
  bool waited = false;
  auto adapters = [&](int tile) -> int {
    if (!waited) grid_dep_wait();
    waited = true;
    return p.count[tile];
  };
  // VEC: this CTA's tokens seg, seg + S, .. of a tile, numbered 0, 1, .., two a lane; their
  // ids (-1: none) come from the call's own input, so the rows of B are under way before the
  // shrink kernel is done.  for_adapters calls body(id, tokens lane, tokens lane + 32 as
  // ballots) for each distinct id in order of first appearance, until it returns false.
  const int own_rows = (p.tile_n - seg + S - 1) / S;
  auto own_id = [&](int tile, int c) -> int {
    const int m = tile * p.tile_n + c * S + seg;
    const int id = c < own_rows && m < p.M ? p.ids[m] : -1;
    return id < p.L ? id : -1;
  };
  auto for_adapters = [&](int tile, auto&& body) {
    const int a = own_id(tile, lane), b = own_id(tile, lane + 32);
    unsigned left_a = __ballot_sync(0xffffffffu, a >= 0), left_b = __ballot_sync(0xffffffffu, b >= 0);
    while (left_a | left_b) {
      const int id = left_a ? __shfl_sync(0xffffffffu, a, __ffs(left_a) - 1)
                            : __shfl_sync(0xffffffffu, b, __ffs(left_b) - 1);
      const unsigned in_a = __ballot_sync(0xffffffffu, a == id);
      const unsigned in_b = __ballot_sync(0xffffffffu, b == id);
      left_a &= ~in_a;
      left_b &= ~in_b;
      if (!body(id, in_a, in_b)) break;
    }
  };

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    const uint32_t lead = elect_one();
    const uint64_t pol_w = p.tiles == 1 ? l2_policy_evict_first() : l2_policy_evict_last();
    const uint64_t pol_x = l2_policy_evict_last();
    uint32_t s = 0, ph = 1;
    bool ok = true;
    // the leader's barriers as seen from this CTA (pair: both CTAs' copies count there)
    const uint32_t full0 = CG == 2 ? peer_addr(smem_u32(full), lead_rank) : smem_u32(full);
    auto next = [&]() {
      if (++s == (uint32_t)stages) {
        s = 0;
        ph ^= 1;
      }
    };
    for (int i = worker; i < units && ok; i += workers) {
      const int tile = i / p.blocks, block = i - tile * p.blocks;
      const int row = (block * CG + (int)rank) * 128;
      const int m = tile * p.tile_n + (int)rank * rows_b;
      for (int k = k0; k < k1; ++k) {
        if (!wait(&empty[s], ph)) {
          ok = false;
          break;
        }
        const uint32_t st = smem_u32(smem) + s * stage_bytes;
        if (rank == 0)
          mbar_arrive_expect_tx_if(lead, smem_u32(&full[s]), CG * (uint32_t)stage_bytes);
        if (CG == 2) {
          tma_load_2d_pair_if(lead, st, &map_w, k * 64, row, full0 + s * 8, pol_w);
          tma_load_2d_pair_if(lead, st + kStageA, &map_x, k * 64, m, full0 + s * 8, pol_x);
        } else {
          tma_load_2d_if(lead, st, &map_w, k * 64, row, full0 + s * 8, pol_w);
          tma_load_2d_if(lead, st + kStageA, &map_x, k * 64, m, full0 + s * 8, pol_x);
        }
        next();
      }
      const int n = ok && !VEC ? adapters(tile) : 0;
      for (int d = seg; d < n && ok; d += S) {
        const int id = p.list[(size_t)tile * p.tile_n + d];
        for (int h = 0; h < chunks; ++h) {
          if (!wait(&empty[s], ph)) {
            ok = false;
            break;
          }
          const uint32_t st = smem_u32(smem) + s * stage_bytes;
          if (rank == 0) mbar_arrive_expect_tx_if(lead, smem_u32(&full[s]), CG * (uint32_t)kStageA);
          if (CG == 2)
            tma_load_3d_pair_if(lead, st, &map_b, h * 64, row, id, full0 + s * 8, pol_x);
          else
            tma_load_3d_if(lead, st, &map_b, h * 64, row, id, full0 + s * 8, pol_x);
          next();
        }
      }
    }
    if (!ok) {  // the copies of the last steps may still be landing
      const unsigned long long t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 2000000ull) {
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // ------------------------------------------------------------------ MMA issue
      const uint32_t lead = elect_one();
      const uint32_t idesc = idesc_16bit(128 * CG, p.tile_n, p.dtype);
      const uint64_t desc0 = sdesc_sw128(smem_u32(smem));
      const uint32_t t0 = (uint32_t)(tbuf - smem) >> 4;
      uint32_t s = 0, ph = 0, ts = 0, tph = 0, local = 0;
      bool ok = true;
      auto commit = [&](uint64_t* bar) {
        if (CG == 2)
          tc_commit2_both_if(lead, smem_u32(bar), (uint16_t)(3u << lead_rank));
        else
          tc_commit_if(lead, smem_u32(bar));
      };
      auto next = [&]() {
        if (++s == (uint32_t)stages) {
          s = 0;
          ph ^= 1;
        }
      };
      for (int i = worker; i < units && ok; i += workers, ++local) {
        const int ab = local & 1;
        if (!wait(&acce[ab], ((local >> 1) & 1) ^ 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t dst = tmem + ab * kAccCols;
        uint32_t acc = 0;
        for (int k = k0; k < k1; ++k) {
          if (!wait(&full[s], ph)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t a = desc0 + ((s * stage_bytes) >> 4);
          if (lead) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_ss(CG, dst, a + 2 * j, a + (kStageA >> 4) + 2 * j, idesc, acc | (j > 0));
          }
          acc = 1;
          commit(&empty[s]);
          next();
        }
        const int n = ok && !VEC ? adapters(i / p.blocks) : 0;
        for (int d = seg; d < n && ok; d += S) {
          for (int h = 0; h < chunks; ++h) {
            const int slices = (min(64, p.R - h * 64) + 15) / 16;
            if (!wait(&full[s], ph) || !wait(&tfull[ts], tph)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t a = desc0 + ((s * stage_bytes) >> 4);
            const uint64_t hi = desc0 + t0 + ((2 * ts * bytes_b) >> 4), lo = hi + (bytes_b >> 4);
            if (lead)
              for (int j = 0; j < slices; ++j) {
                mma_ss(CG, dst, a + 2 * j, hi + 2 * j, idesc, acc | (j > 0));
                mma_ss(CG, dst, a + 2 * j, lo + 2 * j, idesc, 1u);
              }
            acc = 1;
            commit(&empty[s]);
            commit(&tempty[ts]);
            next();
            if (++ts == (uint32_t)tslots) {
              ts = 0;
              tph ^= 1;
            }
          }
        }
        if (ok) commit(&accf[ab]);
      }
      commit(drain);
    }
  } else if (VEC && warp == 2) {
    // ------------------------------------------------------- VEC: the adapters' rows of B
    const uint32_t lead = elect_one();
    const uint64_t pol = l2_policy_evict_last();
    uint32_t step = 0;
    bool ok = true;
    for (int i = worker; i < units && ok; i += workers) {
      const int tile = i / p.blocks, block = i - tile * p.blocks;
      const uint32_t bytes = (uint32_t)min(128, p.N - block * 128) * p.R * 2;
      for_adapters(tile, [&](int id, unsigned, unsigned) {
        const int s = step % tslots;
        ok = wait(&tempty[s], ((step / tslots) & 1) ^ 1);
        ++step;
        if (!ok) return false;
        mbar_arrive_expect_tx_if(lead, smem_u32(&tfull[s]), bytes);
        bulk_g2s_if(lead, smem_u32(tbuf) + s * vec_slot_bytes(p.R),
                    reinterpret_cast<const T*>(p.b) + ((size_t)id * p.N + block * 128) * p.R, bytes,
                    smem_u32(&tfull[s]), pol);
        return true;
      });
    }
    if (!ok) {  // the copies of the last steps may still be landing
      const unsigned long long t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 2000000ull) {
      }
    }
  } else if (VEC && warp >= 8) {
    // ------------------------------------------------------------- VEC: t . B^T in fp32
    // A slot's adapter is one to four warps' work (the more, the longer its rows), a lane
    // having four to one of the 128 rows: several adapters are in the making, with several
    // sums a lane in flight (two groups of four warps, a row a thread, took 0.65 us a step).
    // delta holds this CTA's tokens seg, seg + S, .. one after the other.  A row is read in
    // 16-byte chunks from a place of its own on, so that eight neighbouring rows' chunks lie
    // in different banks.
    const int group = kBuilders / tslots;
    const int own = (warp - 8) / group;
    const int rows_lane = 4 / group;
    const int row0 = (warp - 8) % group * rows_lane * 32 + lane;
    const int C = p.R / 8;  // chunks of a row
    // rows after which the chunks' banks repeat: 8 / gcd(C, 8)
    const int apart = C % 8 == 0 ? 1 : C % 4 == 0 ? 2 : C % 2 == 0 ? 4 : 8;
    const int turn = lane / apart % C;
    float* tf = reinterpret_cast<float*>(tcopy);
    uint32_t step = 0, dph = 1;
    bool ok = true;
    // (after a wait that gave up a warp still meets the others at their barriers)
    for (int i = worker; i < units; i += workers) {
      const int tile = i / p.blocks;
      const int m0 = tile * p.tile_n;
      adapters(tile);   // t is complete
      builders_sync();  // the previous unit's t has been used
      for (int u = threadIdx.x - 256; u < own_rows * C; u += 32 * kBuilders) {
        const int c = u / C, m = m0 + c * S + seg;
        if (m >= p.M) break;
        float t[8];
        load_t8(p, m, u % C * 8, t);
        reinterpret_cast<float4*>(tf)[2 * u] = make_float4(t[0], t[1], t[2], t[3]);
        reinterpret_cast<float4*>(tf)[2 * u + 1] = make_float4(t[4], t[5], t[6], t[7]);
      }
      if (ok && !wait(dempty, dph)) ok = false;  // the epilogue has read the previous delta
      dph ^= 1;
      builders_sync();
      // tokens without an adapter
      for (int c = warp - 8; c < own_rows; c += kBuilders)
        if (own_id(tile, c) < 0)
          reinterpret_cast<float4*>(delta + c * 128)[lane] = make_float4(0.f, 0.f, 0.f, 0.f);
      for_adapters(tile, [&](int, unsigned in_a, unsigned in_b) {
        if ((int)(step++ % tslots) != own || !ok) return true;
        ok = wait(&tfull[own], ((step - 1) / tslots) & 1);
        if (!ok) return true;
        const uint4* b =
            reinterpret_cast<const uint4*>(tbuf + own * vec_slot_bytes(p.R)) + row0 * C;
        for (uint64_t who = (uint64_t)in_b << 32 | in_a; who; who &= who - 1) {
          const int c = __ffsll(who) - 1;
          const float4* t4 = reinterpret_cast<const float4*>(tf + c * p.R);
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
          int j = turn;
#pragma unroll 2
          for (int k = 0; k < C; ++k) {
            const float4 x = t4[2 * j], y = t4[2 * j + 1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (i >= rows_lane) break;
              Pack<T, 8> v;
              v.raw = b[i * 32 * C + j];
              acc[i] = fmaf(to_f32(v.v[0]), x.x, acc[i]);
              acc[i] = fmaf(to_f32(v.v[1]), x.y, acc[i]);
              acc[i] = fmaf(to_f32(v.v[2]), x.z, acc[i]);
              acc[i] = fmaf(to_f32(v.v[3]), x.w, acc[i]);
              acc[i] = fmaf(to_f32(v.v[4]), y.x, acc[i]);
              acc[i] = fmaf(to_f32(v.v[5]), y.y, acc[i]);
              acc[i] = fmaf(to_f32(v.v[6]), y.z, acc[i]);
              acc[i] = fmaf(to_f32(v.v[7]), y.w, acc[i]);
            }
            if (++j == C) j = 0;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < rows_lane) delta[c * 128 + row0 + 32 * i] = acc[i];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&tempty[own]));
        return true;
      });
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(dfull));
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------------- builders
    // step i goes to the warps of slot i % tslots
    const int group = kBuilders / tslots;
    const int own = (warp - 8) / group;
    const int tid = (warp - 8) % group * 32 + lane;
    uint8_t* const dst = tbuf + 2 * own * bytes_b;
    uint32_t step = 0, tph = 1;
    bool ok = true;
    const uint32_t tfull0 = CG == 2 ? peer_addr(smem_u32(tfull), lead_rank) : smem_u32(tfull);
    // (after a wait that gave up a warp still meets the others at their barriers)
    for (int i = worker; i < units; i += workers) {
      const int tile = i / p.blocks;
      const int n = adapters(tile);
      const int m0 = tile * p.tile_n + (int)rank * rows_b;
      if (seg >= n) continue;    // the same for all builders
      builders_sync();           // the previous unit's rows have been used
      for (int r = threadIdx.x - 256; r < rows_b; r += 32 * kBuilders)
        place[r] = (short)p.place[(size_t)m0 + r];
      if (copy_bytes) {
        const int eights = p.R / 8;
        for (int u = threadIdx.x - 256; u < rows_b * eights; u += 32 * kBuilders) {
          const int row = u / eights, r = u % eights * 8;
          if (m0 + row >= p.M) break;
          T* dst = reinterpret_cast<T*>(tcopy) + row * 2 * p.R + r;
          load_t8_split<T>(p, m0 + row, r, reinterpret_cast<uint4*>(dst),
                           reinterpret_cast<uint4*>(dst + p.R));
        }
      }
      builders_sync();
      for (int d = seg; d < n && ok; d += S) {
        for (int h = 0; h < chunks; ++h, ++step) {
          if ((int)(step % tslots) != own) continue;
          const int units = (min(64, p.R - h * 64) + 15) / 16 * 2;  // 16-byte units of a row
          if (!wait(&tempty[own], tph)) {
            ok = false;
            break;
          }
          tph ^= 1;
          for (int u = tid; u < rows_b * units; u += group * 32) {
            const int row = u / units, j = u - row * units;
            const int r = h * 64 + j * 8;
            uint4 hi = make_uint4(0u, 0u, 0u, 0u), lo = hi;
            if (place[row] == d && r < p.R) {
              if (copy_bytes) {
                const T* src = reinterpret_cast<const T*>(tcopy) + row * 2 * p.R + r;
                hi = *reinterpret_cast<const uint4*>(src);
                lo = *reinterpret_cast<const uint4*>(src + p.R);
              } else {
                load_t8_split<T>(p, m0 + row, r, &hi, &lo);
              }
            }
            // rows of 128 bytes, 16-byte units swizzled by the row (128-byte swizzle)
            uint8_t* at = dst + row * 128 + ((j ^ (row & 7)) << 4);
            *reinterpret_cast<uint4*>(at) = hi;
            *reinterpret_cast<uint4*>(at + bytes_b) = lo;
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            if (CG == 2 && rank != 0)
              mbar_arrive_remote(tfull0 + own * 8);
            else
              mbar_arrive(smem_u32(&tfull[own]));
          }
        }
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------------- epilogue
    const int q = warp & 3;
    const uint32_t acce0 = CG == 2 ? peer_addr(smem_u32(acce), lead_rank) : smem_u32(acce);
    uint32_t local = 0;
    grid_dep_wait();  // the shrink kernel's lists
    if (worker == 0 && crank == 0 && warp == 4) {
      bool bad = false;
      for (int t = lane; t < p.tiles; t += 32) bad |= p.bad[t] != 0;
      bad = __any_sync(0xffffffffu, bad);
      if (lane == 0 && bad) atomicOr(p.err, QMOE_FLAG_BAD_ID);
    }
    T* stage = reinterpret_cast<T*>(epi_stage + q * 2048);  // [32 tokens][32 rows]
    for (int i = worker; i < units; i += workers, ++local) {
      const int tile = i / p.blocks, block = i - tile * p.blocks;
      const int ab = local & 1;
      const int m0 = tile * p.tile_n;
      const int cols = min(p.tile_n, p.M - m0);
      const int n0 = (block * CG + (int)rank) * 128 + q * 32;
      const bool any = k1 > k0 || (!VEC && p.count[tile] > seg);
      if (!wait(&accf[ab], (local >> 1) & 1)) break;
      if (VEC && !wait(dfull, local & 1)) break;
      tc_fence_after();
      const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16) + ab * kAccCols;
      for (int c0 = 0; c0 < cols; c0 += 32) {
        float v[32];
        if (any) {
          // (a tile's last 16 columns may be followed by columns of no meaning, within the
          // accumulator's 256)
          uint32_t r[2][16];
          tmem_ld_x16(tbase + c0, r[0]);
          tmem_ld_x16(tbase + c0 + 16, r[1]);
          tmem_wait_ld();
          tmem_ld_ready(r[0]);
          tmem_ld_ready(r[1]);
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(r[k >> 4][k & 15]);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = 0.f;
        }
        if (S > 1) {
          // this segment's sums [token][row], over the ring, which is idle: a CTA of a split
          // unit has this one unit, and its MMAs are complete
          float* sums = reinterpret_cast<float*>(smem) + (size_t)c0 * 128 + q * 32 + lane;
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (c0 + k < cols) sums[k * 128] = v[k];
        } else {
          if constexpr (VEC) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (c0 + k < cols) v[k] += delta[(c0 + k) * 128 + q * 32 + lane];
          }
          if (p.base) {
            const T* base = reinterpret_cast<const T*>(p.base) + (size_t)(m0 + c0) * p.ldbase + n0;
            const bool in = n0 + lane < p.N;
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (in && c0 + k < cols) v[k] += to_f32(base[(size_t)k * p.ldbase + lane]);
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 32; ++k) stage[k * 32 + lane] = from_f32<T>(v[k]);
          __syncwarp();
          T* out = reinterpret_cast<T*>(p.out) + (size_t)(m0 + c0) * p.N + n0;
          if (p.wide) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int tok = u * 8 + lane / 4, part = lane % 4 * 8;
              if (c0 + tok < cols && n0 + part < p.N)
                *reinterpret_cast<uint4*>(out + (size_t)tok * p.N + part) =
                    *reinterpret_cast<const uint4*>(stage + tok * 32 + part);
            }
          } else if (n0 + lane < p.N) {
            for (int k = 0; k < 32 && c0 + k < cols; ++k)
              out[(size_t)k * p.N + lane] = stage[k * 32 + lane];
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2 && rank != 0)
          mbar_arrive_remote(acce0 + ab * 8);
        else
          mbar_arrive(smem_u32(&acce[ab]));
        if (VEC) mbar_arrive(smem_u32(dempty));
      }
    }
  }

  // No MMA may still read this CTA's shared memory or write its TMEM, and no remote
  // arrival may be in flight, when it (or its peer) exits.
  if (warp == 1) {
    if (CG == 2)
      drain_wait_cl(smem_u32(drain), 0);
    else
      drain_wait(smem_u32(drain), 0);
  }
  tc_fence_before();
  __syncthreads();
  if (clustered) cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    if (CG == 2)
      tmem_dealloc2(tmem, 2 * kAccCols);
    else
      tmem_dealloc(tmem, 2 * kAccCols);
  }
  if (S > 1) {
    // the unit's tokens seg, seg + S, .. over all segments: a warp per token, four rows a
    // lane, the segments' values in flight together
    const int tile = worker / p.blocks, block = worker - tile * p.blocks;
    const int m0 = tile * p.tile_n, cols = min(p.tile_n, p.M - m0);
    const int n = (block * CG + (int)rank) * 128 + 4 * lane;
    const uint32_t sums0 = smem_u32(smem) + 16 * lane;
    for (int c = seg + S * warp; c < cols; c += S * (kGemmThreads / 32)) {
      float4 v[kMaxSplits];
#pragma unroll
      for (int g = 0; g < kMaxSplits; ++g)
        if (g < S) v[g] = ld_cluster_f32x4(peer_addr(sums0 + c * 512, g * CG + rank));
      float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int g = 0; g < kMaxSplits; ++g)
        if (g < S) t.x += v[g].x, t.y += v[g].y, t.z += v[g].z, t.w += v[g].w;
      if constexpr (VEC) {
        const float4 d = reinterpret_cast<const float4*>(delta + c / S * 128)[lane];
        t.x += d.x, t.y += d.y, t.z += d.z, t.w += d.w;
      }
      float f[4] = {t.x, t.y, t.z, t.w};
      const T* base = reinterpret_cast<const T*>(p.base) + (size_t)(m0 + c) * p.ldbase + n;
      T* out = reinterpret_cast<T*>(p.out) + (size_t)(m0 + c) * p.N + n;
      Pack<T, 4> o;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (p.base && n + e < p.N) f[e] += to_f32(base[e]);
        o.v[e] = from_f32<T>(f[e]);
      }
      if (p.wide && n < p.N) {
        *reinterpret_cast<uint2*>(out) = o.raw;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < p.N) out[e] = o.v[e];
      }
    }
    cluster_sync_all();  // no CTA leaves while its sums may still be read
  }
}

// --------------------------------------------------------------------- one or two tokens
// One, two or four warps (WPR, the more, the longer the row) per row of w: its product with
// up to MT token rows in fp32, w in 16-byte loads of which a lane has about eight in all, in
// flight together (one warp a row, 28 loads a lane at K = 7168, took 9.4 us); then the row
// of each token's B with t.
// HBM (or L2) bound, and there is nothing to set up: the tensor-core kernel spends 5 of its
// 10.3 us at M = 1, K = 7168, N = 2048 on barriers, TMEM, the cluster and the last sums.
// Whole calls at K = 7168, N = 2048, R = 16: one token 9.7 us (tensor cores 11.4), two 10.9
// (11.9), four 16.0 (12.0).
constexpr int kGemvThreads = 128, kGemvTokens = 2;

template <class T, int MT, int WPR>
__global__ void __launch_bounds__(kGemvThreads) lora_gemv_kernel(const LoraArgs p) {
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
    constexpr int kFlight = MT == 1 ? 8 : 6;
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

// Clusters of `size` CTAs of a kernel that the device holds at once: asked of the runtime
// once per size and kept (a property of the kernel and the device model).
template <class K>
int resident_clusters(K* kernel, int size, int threads, size_t smem, std::atomic<int>& kept,
                      int num_sms) {
  int n = kept.load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(num_sms / size * size);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) return 0;
    kept.store(n, std::memory_order_relaxed);
  }
  return n;
}

// Tensor maps: token rows in boxes of `rows`, [N][K] and [L][rows][cols] in boxes of 64
// columns.
cudaError_t map_rows(CUtensorMap* map, const LoraArgs& p, const void* base, int cols, int rows,
                     long long ld, int box_rows) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows}, strides[1] = {(uint64_t)ld * 2};
  const uint32_t box[2] = {64, (uint32_t)box_rows};
  return make_tmap16(map, p.dtype, base, 2, dims, strides, box) == QMOE_OK ? cudaSuccess
                                                                           : cudaErrorUnknown;
}
cudaError_t map_adapters(CUtensorMap* map, const LoraArgs& p, const void* base, int cols, int rows,
                         int box_rows) {
  const uint64_t dims[3] = {(uint64_t)cols, (uint64_t)rows, (uint64_t)p.L};
  const uint64_t strides[2] = {(uint64_t)cols * 2, (uint64_t)rows * cols * 2};
  const uint32_t box[3] = {64, (uint32_t)box_rows, 1};
  return make_tmap16(map, p.dtype, base, 3, dims, strides, box) == QMOE_OK ? cudaSuccess
                                                                           : cudaErrorUnknown;
}
cudaError_t shrink_maps(const LoraArgs& p, CUtensorMap* x, CUtensorMap* a) {
  const cudaError_t e = map_rows(x, p, p.x, p.K, p.M, p.ldx, p.tile_n);
  return e == cudaSuccess ? map_adapters(a, p, p.a, p.K, p.R, p.R) : e;
}
cudaError_t gemm_maps(const LoraArgs& p, CUtensorMap* x, CUtensorMap* w, CUtensorMap* b) {
  cudaError_t e = map_rows(x, p, p.x, p.K, p.M, p.ldx, p.tile_n / p.cg);
  if (e == cudaSuccess && p.w) e = map_rows(w, p, p.w, p.K, p.N, p.K, 128);
  if (!p.w) *w = *x;  // never read
  return e == cudaSuccess ? map_adapters(b, p, p.b, p.R, p.N, 128) : e;
}

template <class T>
cudaError_t run(LoraArgs& p, int num_sms, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0] = pdl_attribute();
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  if (!p.tensor_shrink) {
    int threads = (p.K / 8 + 31) / 32 * 32;
    threads = threads < kShrinkThreads ? kShrinkThreads : threads > kShrinkMost ? kShrinkMost : threads;
    cfg.blockDim = dim3(threads);
    cfg.gridDim = dim3((unsigned)(p.tiles + (long long)p.M * (p.R / 8)));
    e = cudaLaunchKernelEx(&cfg, lora_shrink_kernel<T>, p);
  } else {
    const int ctas = p.tiles * p.tsplits, cap = 128 / p.R;
    const int most = ((p.L < p.tile_n ? p.L : p.tile_n) + cap - 1) / cap;
    const int share = num_sms / ctas < 1 ? 1 : num_sms / ctas;
    cfg.blockDim = dim3(kShrinkThreads);
    cfg.gridDim = dim3(ctas, share < most ? share : most);
    cfg.dynamicSmemBytes = 1024 + shrink_stages(p.tile_n) * shrink_stage_bytes(p.tile_n);
    e = cudaFuncSetAttribute(lora_shrink_mma_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)cfg.dynamicSmemBytes);
    if (e != cudaSuccess) return e;
    CUtensorMap map_x, map_a;
    e = shrink_maps(p, &map_x, &map_a);
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, lora_shrink_mma_kernel<T>, map_x, map_a, p);
  }
  if (e != cudaSuccess) return e;
  if (p.M <= kGemvTokens) {
    return p.K <= 2048   ? gemv<T, 1>(p, cfg)
           : p.K <= 4096 ? gemv<T, 2>(p, cfg)
                         : gemv<T, 4>(p, cfg);
  }
  CUtensorMap map_x, map_w, map_b;
  e = gemm_maps(p, &map_x, &map_w, &map_b);
  if (e != cudaSuccess) return e;
  const int stage = kStageA + token_bytes(p.tile_n, p.cg);
  const bool vec = p.cg == 1 && p.tile_n <= kVecTokens && p.tile_n * p.R <= kVecTokenRanks;
  const Behind more = behind(vec, p.tile_n, p.cg, p.R);
  const int other = 1024 + kCtrl + kEpiStage + more.slots + more.copy + more.delta;
  const int most = (kSmemLimit - other) / stage;
  p.stages = most < kMaxStages ? most : kMaxStages;
  // every plan's shared memory leaves one CTA an SM
  const size_t smem = other + (size_t)p.stages * stage;
  auto* k = p.cg == 2 ? lora_gemm_kernel<T, 2, false>
            : vec     ? lora_gemm_kernel<T, 1, true>
                      : lora_gemm_kernel<T, 1, false>;
  e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int units = p.tiles * p.blocks;
  static std::atomic<int> kept[3][kMaxSplits + 1];
  auto clusters_of = [&](int splits) {
    const int size = p.cg * splits;
    if (size == 1) return num_sms;
    return resident_clusters(k, size, kGemmThreads, smem, kept[vec ? 2 : p.cg - 1][splits],
                             num_sms);
  };
  // Segments: where every unit's cluster is resident at once and each has 4 steps or more,
  // as many as there can be
  p.splits = 1;
  for (int s = kMaxSplits / p.cg; s > 1 && p.splits == 1; --s)
    if (4 * s <= p.ksteps && units <= num_sms / (p.cg * s) && units <= clusters_of(s)) p.splits = s;
  const int held = clusters_of(p.splits);
  if (held < 1) return cudaErrorInvalidConfiguration;
  const int size = p.cg * p.splits;
  cfg.gridDim = dim3((unsigned)((units < held ? units : held) * size));
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = smem;
  if (size > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = size;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, k, map_x, map_w, map_b, p);
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
  return p.dtype == QMOE_DTYPE_BF16 ? run<__nv_bfloat16>(p, num_sms, stream)
                                    : run<__half>(p, num_sms, stream);
}

}  // namespace qmoe
