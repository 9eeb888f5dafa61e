// A shared projection with a low-rank adapter per token:
//   t[m] = scales[a] * (x[m] . A[a]^T),  out[m] = base[m] + x[m] . w^T + t[m] . B[a]^T
// with a = adapter_ids[m].
//
// Two kernels.  The first (shrink: plain fp32 products for few tokens, tensor cores for
// many) forms the sums x . A^T in fp32 and lists, for each tile
// of tokens, the distinct adapters its tokens use.  The second is one GEMM whose
// contraction runs over K and then over the ranks of the tile's adapters: the MMA's M side
// is 128 rows of w (or of B[a]), its N side a tile of up to 256 tokens, and for each of
// the tile's adapters the token operand is t with the rows of other adapters zero.  So the
// adapters cost a tile (distinct adapters) * ranks more of contraction length, whatever
// the order of the tokens, and the result is rounded once.
//
// t enters the tensor cores as the sum of two values of the activation type (t rounded,
// and what the rounding left): 16 (bf16) or 22 (fp16) significant bits for twice the MMAs
// of a contraction that is short, instead of a second rounding of the result's size.
//
// GEMM pipeline (a unit is 128 rows of w per CTA x one token tile, its contraction split
// into S segments when there are fewer units than SMs):
//   warp 0      TMA producer: steps of 64 of K, [128 rows of w | token rows], then per
//               adapter and 64 ranks twice [128 rows of B[a]]
//   warp 1      MMA issue: 4 x tcgen05.mma kind::f16 per step, fp32 accumulator in TMEM,
//               two accumulators, so that the epilogue overlaps the next unit
//   warps 4-7   epilogue: TMEM -> registers -> base, rounding, global stores; with S > 1
//               the segments' partial sums are added in K order by the last to arrive
//   warps 8-11  builders: the token operand of the adapter steps into two slots of their
//               own
// Few tokens (one tile): one CTA per unit, w streamed once, HBM bound.  More: CTA pairs
// (cta_group::2, M = 256), each SM loading half of the token rows, since a 128 x 256 tile
// fed by one SM alone asks more of its L2 port (96 bytes a clock) than it has.
//
// Every wait is bounded, as in the layer's GEMMs.
#include "cluster.cuh"
#include "common.cuh"
#include "launch.h"
#include "pack.cuh"

namespace qmoe {
namespace {

// ------------------------------------------------------------------ shrink, few tokens
// A block per (token, 8 ranks): its warps share out K, and the eight sums are reduced in a
// fixed order.  The blocks before them list the tiles' adapters (one block each) and zero
// the error word and the arrival counters.
constexpr int kShrinkThreads = 256;

// The distinct valid ids of a tile's tokens, in order of first appearance, into list
// (shared, one entry per token of the tile); whole block of kShrinkThreads.  Returns their
// count; *mine is this thread's token's place in the list (-1: none), *bad whether its id
// is L or more.
struct ListScratch {
  int id[kShrinkThreads], place[kShrinkThreads], warp_count[kShrinkThreads / 32];
};
__device__ __forceinline__ int list_adapters(const int32_t* __restrict__ ids, int m0, int rows,
                                             int L, ListScratch& w, int* list, int* mine,
                                             bool* bad) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int id = tid < rows ? ids[m0 + tid] : -1;
  *bad = id >= L;
  if (id >= L || id < 0) id = -1;
  w.id[tid] = id;
  __syncthreads();
  int lead = tid;  // the first token with this id
  if (id >= 0)
    for (int i = 0; i < tid; ++i)
      if (w.id[i] == id) {
        lead = i;
        break;
      }
  const bool first = id >= 0 && lead == tid;
  const unsigned mask = __ballot_sync(0xffffffffu, first);
  if (lane == 0) w.warp_count[warp] = __popc(mask);
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

// What the GEMM needs of the lists, and zeros where it counts; by one block per tile.
__device__ __forceinline__ void publish_list(const LoraArgs& p, int t, const int* list, int n,
                                             bool bad) {
  const int tid = threadIdx.x;
  if (t == 0) {
    if (tid == 0) p.err[0] = 0u;
    for (int i = tid; i < p.n_cnt; i += kShrinkThreads) p.cnt[i] = 0;
  }
  for (int i = tid; i < n; i += kShrinkThreads) p.list[(size_t)t * p.tile_n + i] = list[i];
  const bool any = __syncthreads_or(bad);
  if (tid == 0) {
    p.count[t] = n;
    p.bad[t] = any;
  }
}

template <class T>
__global__ void __launch_bounds__(kShrinkThreads) lora_shrink_kernel(const LoraArgs p) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int kWarps = kShrinkThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if ((int)blockIdx.x < p.tiles) {
    __shared__ ListScratch scratch;
    __shared__ int list[kShrinkThreads];
    const int t = blockIdx.x, m0 = t * p.tile_n;
    int mine;
    bool bad;
    const int n =
        list_adapters(p.ids, m0, min(p.tile_n, p.M - m0), p.L, scratch, list, &mine, &bad);
    publish_list(p, t, list, n, bad);
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
    for (int c = tid; c < chunks; c += kShrinkThreads) {
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
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += part[w][tid];
    p.t[(size_t)m * p.R + r0 + tid] = s;
  }
}

// ------------------------------------------------------------------------------- GEMM
constexpr int kGemmThreads = 384;
constexpr int kStageA = 128 * 128;  // 128 rows x 64 elements
constexpr int kMaxStages = 12;
constexpr int kAccCols = 256;  // TMEM columns of one accumulator
constexpr int kCtrl = 1024;
constexpr int kSmemLimit = 232448;

// Token rows per CTA of a tile, and the bytes of one step of them.
__host__ __device__ constexpr int token_bytes(int tile_n, int cg) { return tile_n / cg * 128; }

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

__device__ __forceinline__ void fence_proxy_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ----------------------------------------------------------------- shrink, many tokens
// A CTA per (token tile, K segment): D[rank of adapter][token] = A[a] . x^T on the tensor
// cores, with the 128 / R adapters of a pass stacked on the MMA's 128 rows, so that a tile
// of few adapters (requests one after another) takes one pass over its token rows.  Each
// token keeps the rows of its own adapter; the segments' sums are added by the GEMM's
// builders.  gridDim.y CTAs share a tile's passes.
__host__ __device__ constexpr int shrink_stages(int tile_n) { return tile_n > 128 ? 4 : 6; }

template <class T>
__global__ void __launch_bounds__(kShrinkThreads, 1)
    lora_shrink_mma_kernel(const __grid_constant__ CUtensorMap map_x,
                           const __grid_constant__ CUtensorMap map_a, const LoraArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ ListScratch scratch;
  __shared__ int list[kShrinkThreads], place[kShrinkThreads];
  __shared__ __align__(8) uint64_t full[6], empty[6], accf, acce, drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stages = shrink_stages(p.tile_n);
  const int stage_bytes = kStageA + p.tile_n * 128;
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
  int mine;
  bool bad;
  const int n = list_adapters(p.ids, m0, cols, p.L, scratch, list, &mine, &bad);
  place[threadIdx.x] = mine;
  if (seg == 0 && blockIdx.y == 0) publish_list(p, t, list, n, bad);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int cap = 128 / p.R;
  const int passes = (n + cap - 1) / cap;
  const int ksteps = (p.K + 63) / 64;
  const int k0 = (int)((long long)ksteps * seg / p.tsplits);
  const int k1 = (int)((long long)ksteps * (seg + 1) / p.tsplits);

  if (warp == 0) {
    const uint32_t lead = elect_one();
    const uint64_t pol = l2_policy_evict_last();  // the GEMM reads the token rows next
    uint32_t s = 0, ph = 1;
    bool ok = true;
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
        tma_load_2d_if(lead, st + kStageA, &map_x, k * 64, m0, fb, pol);
        if (++s == (uint32_t)stages) {
          s = 0;
          ph ^= 1;
        }
      }
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
    float* dst = p.t + ((size_t)seg * p.M + m0) * p.R + r;
    uint32_t ph = 0;
    for (int ps = blockIdx.y; ps < passes; ps += gridDim.y) {
      if (!warp_wait(smem_u32(&accf), ph, abort_flag, p.err)) break;
      ph ^= 1;
      tc_fence_after();
      const int want = slot < cap ? ps * cap + slot : -2;
      for (int c0 = 0; c0 < cols; c0 += 16) {
        uint32_t v[16];
        tmem_ld_x16(tmem + ((uint32_t)(q * 32) << 16) + c0, v);
        tmem_wait_ld();
        tmem_ld_ready(v);
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (c0 + k < cols && place[c0 + k] == want)
            dst[(size_t)(c0 + k) * p.R] = __uint_as_float(v[k]);
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

template <class T, int CG>
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
  uint8_t* tbuf = smem + stages * stage_bytes;  // [2][bytes_b]
  uint8_t* ctrl = tbuf + 2 * bytes_b;
  uint64_t* full = reinterpret_cast<uint64_t*>(ctrl);
  uint64_t* empty = full + kMaxStages;
  uint64_t* tfull = empty + kMaxStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* accf = tempty + 2;
  uint64_t* acce = accf + 2;
  uint64_t* drain = acce + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const int worker = CG == 2 ? (int)cluster_index() : (int)blockIdx.x;
  const int workers = CG == 2 ? (int)cluster_count() : (int)gridDim.x;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&tfull[i]), 4 * CG);
      mbar_init(smem_u32(&tempty[i]), 1);
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
  if (CG == 2) cluster_sync_all();  // the peer's barriers exist before any remote arrival
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int ksteps = p.ksteps;  // of the shared product; 0 without w
  const int chunks = (p.R + 63) / 64;
  const int S = p.splits;
  const int pieces = p.tiles * p.blocks * S;
  // piece = (tile, block, segment), segments of a unit next to each other
  struct Piece {
    int tile, block, seg, k0, k1;
  };
  auto piece_of = [&](int i) {
    Piece c;
    const int u = i / S;
    c.seg = i - u * S;
    c.tile = u / p.blocks;
    c.block = u - c.tile * p.blocks;
    c.k0 = (int)((long long)ksteps * c.seg / S);
    c.k1 = (int)((long long)ksteps * (c.seg + 1) / S);
    return c;
  };
  // bounded waits; the pair's barriers take arrivals from both CTAs
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (CG == 2) return warp_wait_cl(smem_u32(bar), parity, abort_flag, p.err);
    return warp_wait(smem_u32(bar), parity, abort_flag, p.err);
  };
  // Adapter steps of a tile (twice per adapter and 64 ranks), in a unit's last segment.
  // The shrink kernel writes the lists, so its completion is awaited first.
  bool waited = false;
  auto adapters = [&](const Piece& c) -> int {
    if (c.seg != S - 1) return 0;
    if (!waited) grid_dep_wait();
    waited = true;
    return p.count[c.tile];
  };

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    const uint32_t lead = elect_one();
    const uint64_t pol_w = p.tiles == 1 ? l2_policy_evict_first() : l2_policy_evict_last();
    const uint64_t pol_x = l2_policy_evict_last();
    uint32_t s = 0, ph = 1;
    bool ok = true;
    // the leader's barriers as seen from this CTA (pair: both CTAs' copies count there)
    const uint32_t full0 = CG == 2 ? peer_addr(smem_u32(full), 0) : smem_u32(full);
    auto next = [&]() {
      if (++s == (uint32_t)stages) {
        s = 0;
        ph ^= 1;
      }
    };
    for (int i = worker; i < pieces && ok; i += workers) {
      const Piece c = piece_of(i);
      const int row = (c.block * CG + (int)rank) * 128;
      const int m = c.tile * p.tile_n + (int)rank * rows_b;
      for (int k = c.k0; k < c.k1; ++k) {
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
      const int n = ok ? adapters(c) : 0;
      for (int d = 0; d < n && ok; ++d) {
        const int id = p.list[(size_t)c.tile * p.tile_n + d];
        for (int h = 0; h < 2 * chunks; ++h) {
          if (!wait(&empty[s], ph)) {
            ok = false;
            break;
          }
          const uint32_t st = smem_u32(smem) + s * stage_bytes;
          if (rank == 0) mbar_arrive_expect_tx_if(lead, smem_u32(&full[s]), CG * (uint32_t)kStageA);
          if (CG == 2)
            tma_load_3d_pair_if(lead, st, &map_b, (h >> 1) * 64, row, id, full0 + s * 8, pol_x);
          else
            tma_load_3d_if(lead, st, &map_b, (h >> 1) * 64, row, id, full0 + s * 8, pol_x);
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
          tc_commit2_both_if(lead, smem_u32(bar));
        else
          tc_commit_if(lead, smem_u32(bar));
      };
      auto next = [&]() {
        if (++s == (uint32_t)stages) {
          s = 0;
          ph ^= 1;
        }
      };
      for (int i = worker; i < pieces && ok; i += workers, ++local) {
        const Piece c = piece_of(i);
        const int ab = local & 1;
        if (!wait(&acce[ab], ((local >> 1) & 1) ^ 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + ab * kAccCols;
        uint32_t acc = 0;
        for (int k = c.k0; k < c.k1; ++k) {
          if (!wait(&full[s], ph)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t a = desc0 + ((s * stage_bytes) >> 4);
          if (lead) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_ss(CG, d, a + 2 * j, a + (kStageA >> 4) + 2 * j, idesc, acc | (j > 0));
          }
          acc = 1;
          commit(&empty[s]);
          next();
        }
        const int n = ok ? adapters(c) : 0;
        for (int h = 0; h < n * 2 * chunks && ok; ++h) {
          const int c0 = ((h >> 1) % chunks) * 64;
          const int slices = (min(64, p.R - c0) + 15) / 16;
          if (!wait(&full[s], ph) || !wait(&tfull[ts], tph)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t a = desc0 + ((s * stage_bytes) >> 4);
          const uint64_t b = desc0 + t0 + ((ts * bytes_b) >> 4);
          if (lead)
            for (int j = 0; j < slices; ++j) mma_ss(CG, d, a + 2 * j, b + 2 * j, idesc, acc | (j > 0));
          acc = 1;
          commit(&empty[s]);
          commit(&tempty[ts]);
          next();
          ts ^= 1;
          if (ts == 0) tph ^= 1;
        }
        if (ok) commit(&accf[ab]);
      }
      commit(drain);
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------------- builders
    const int tid = threadIdx.x - 256;
    uint32_t ts = 0, tph = 1;
    bool ok = true;
    const uint32_t tfull0 = CG == 2 ? peer_addr(smem_u32(tfull), 0) : smem_u32(tfull);
    for (int i = worker; i < pieces && ok; i += workers) {
      const Piece c = piece_of(i);
      const int n = adapters(c);
      const int m0 = c.tile * p.tile_n + (int)rank * rows_b;
      for (int d = 0; d < n && ok; ++d) {
        const int id = p.list[(size_t)c.tile * p.tile_n + d];
        const float scale = p.scales[id];
        for (int h = 0; h < 2 * chunks; ++h) {
          if (!wait(&tempty[ts], tph)) {
            ok = false;
            break;
          }
          uint8_t* dst = tbuf + ts * bytes_b;
          for (int u = tid; u < rows_b * 8; u += 128) {
            const int row = u >> 3, j = u & 7;
            const int m = m0 + row, r = (h >> 1) * 64 + j * 8;
            Pack<T, 8> o;
            o.raw = make_uint4(0u, 0u, 0u, 0u);
            if (m < p.M && r < p.R && p.ids[m] == id) {
              float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
              for (int g = 0; g < p.tsplits; ++g) {
                const float4* src =
                    reinterpret_cast<const float4*>(p.t + ((size_t)g * p.M + m) * p.R + r);
                const float4 v0 = src[0], v1 = src[1];
                v[0] += v0.x, v[1] += v0.y, v[2] += v0.z, v[3] += v0.w;
                v[4] += v1.x, v[5] += v1.y, v[6] += v1.z, v[7] += v1.w;
              }
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float f = v[e] * scale;
                const T hi = from_f32<T>(f);
                o.v[e] = (h & 1) ? from_f32<T>(f - to_f32(hi)) : hi;
              }
            }
            // rows of 128 bytes, 16-byte units swizzled by the row (128-byte swizzle)
            *reinterpret_cast<uint4*>(dst + row * 128 + ((j ^ (row & 7)) << 4)) = o.raw;
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            if (CG == 2 && rank != 0)
              mbar_arrive_remote(tfull0 + ts * 8);
            else
              mbar_arrive(smem_u32(&tfull[ts]));
          }
          ts ^= 1;
          if (ts == 0) tph ^= 1;
        }
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------------- epilogue
    const int q = warp & 3;
    const uint32_t acce0 = CG == 2 ? peer_addr(smem_u32(acce), 0) : smem_u32(acce);
    uint32_t local = 0;
    T* out = reinterpret_cast<T*>(p.out);
    const T* base = reinterpret_cast<const T*>(p.base);
    grid_dep_wait();  // the counters are the shrink kernel's to clear
    if (worker == 0 && rank == 0 && warp == 4) {
      bool bad = false;
      for (int t = lane; t < p.tiles; t += 32) bad |= p.bad[t] != 0;
      bad = __any_sync(0xffffffffu, bad);
      if (lane == 0 && bad) atomicOr(p.err, QMOE_FLAG_BAD_ID);
    }
    for (int i = worker; i < pieces; i += workers, ++local) {
      const Piece c = piece_of(i);
      const int ab = local & 1;
      const int m0 = c.tile * p.tile_n;
      const int cols = min(p.tile_n, p.M - m0);
      const int n = (c.block * CG + (int)rank) * 128 + q * 32 + lane;
      const bool any = c.k1 > c.k0 || (c.seg == S - 1 && p.count[c.tile] > 0);
      if (!wait(&accf[ab], (local >> 1) & 1)) break;
      tc_fence_after();
      const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16) + ab * kAccCols;
      auto load = [&](int c0, float (&v)[16]) {
        if (!any) {
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = 0.f;
          return;
        }
        uint32_t r[16];
        tmem_ld_x16(tbase + c0, r);
        tmem_wait_ld();
        tmem_ld_ready(r);
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(r[k]);
      };
      bool last = true;
      const size_t slot0 = ((size_t)(i / S) * S * CG + rank) * 128 * p.tile_n;
      const size_t slot_step = (size_t)CG * 128 * p.tile_n;
      if (S > 1) {
        // this segment's sums, [column][row] so that a warp's stores are contiguous
        float* mine = p.part + slot0 + c.seg * slot_step + q * 32 + lane;
        for (int c0 = 0; c0 < cols; c0 += 16) {
          float v[16];
          load(c0, v);
#pragma unroll
          for (int k = 0; k < 16; ++k) mine[(size_t)(c0 + k) * 128] = v[k];
        }
        __threadfence();
        __syncwarp();
        int old = 0;
        if (lane == 0) old = atomicAdd(p.cnt + ((size_t)(i / S) * CG + rank) * 4 + q, 1);
        last = __shfl_sync(0xffffffffu, old, 0) == S - 1;
        __threadfence();
      }
      if (last) {
        for (int c0 = 0; c0 < cols; c0 += 16) {
          float v[16];
          if (S == 1) {
            load(c0, v);
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = 0.f;
            for (int g = 0; g < S; ++g) {
              const float* src = p.part + slot0 + g * slot_step + q * 32 + lane;
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] += __ldcg(src + (size_t)(c0 + k) * 128);
            }
          }
          if (n < p.N) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int m = m0 + c0 + k;
              if (c0 + k < cols) {
                float f = v[k];
                if (base) f += to_f32(base[(size_t)m * p.ldbase + n]);
                out[(size_t)m * p.N + n] = from_f32<T>(f);
              }
            }
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
  if (CG == 2) cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    if (CG == 2)
      tmem_dealloc2(tmem, 2 * kAccCols);
    else
      tmem_dealloc(tmem, 2 * kAccCols);
  }
}

template <class T>
cudaError_t run(LoraArgs& p, const LoraMaps& maps, int num_sms, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0] = pdl_attribute();
  cfg.blockDim = dim3(kShrinkThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  if (p.tsplits == 0) {
    p.tsplits = 1;
    cfg.gridDim = dim3((unsigned)(p.tiles + (long long)p.M * (p.R / 8)));
    e = cudaLaunchKernelEx(&cfg, lora_shrink_kernel<T>, p);
  } else {
    const int ctas = p.tiles * p.tsplits, cap = 128 / p.R;
    const int most = ((p.L < p.tile_n ? p.L : p.tile_n) + cap - 1) / cap;
    const int share = num_sms / ctas < 1 ? 1 : num_sms / ctas;
    cfg.gridDim = dim3(ctas, share < most ? share : most);
    cfg.dynamicSmemBytes = 1024 + (size_t)shrink_stages(p.tile_n) * (kStageA + p.tile_n * 128);
    e = cudaFuncSetAttribute(lora_shrink_mma_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)cfg.dynamicSmemBytes);
    if (e == cudaSuccess)
      e = cudaLaunchKernelEx(&cfg, lora_shrink_mma_kernel<T>, maps.xs, maps.a, p);
  }
  if (e != cudaSuccess) return e;
  const int stage = kStageA + token_bytes(p.tile_n, p.cg);
  const int rest = kSmemLimit - 1024 - kCtrl - 2 * token_bytes(p.tile_n, p.cg);
  p.stages = rest / stage < kMaxStages ? rest / stage : kMaxStages;
  const size_t smem = 1024 + kCtrl + (size_t)p.stages * stage + 2 * token_bytes(p.tile_n, p.cg);
  auto* k = p.cg == 2 ? lora_gemm_kernel<T, 2> : lora_gemm_kernel<T, 1>;
  e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const long long pieces = (long long)p.tiles * p.blocks * p.splits;
  const int workers = num_sms / p.cg;
  cfg.gridDim = dim3((unsigned)((pieces < workers ? (int)pieces : workers) * p.cg));
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = smem;
  if (p.cg == 2) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    int clusters = 0;
    e = cudaOccupancyMaxActiveClusters(&clusters, k, &cfg);
    if (e != cudaSuccess) return e;
    if (clusters < 1) return cudaErrorInvalidConfiguration;
    if (2 * clusters < (int)cfg.gridDim.x) cfg.gridDim = dim3((unsigned)(2 * clusters));
  }
  return cudaLaunchKernelEx(&cfg, k, maps.x, maps.w, maps.b, p);
}

}  // namespace

// Tiles, pairs and splits for a problem (SMs of a GB300: the workspace size must not depend
// on the device).  Up to 256 tokens are one tile and one CTA a unit; more go to CTA pairs,
// with the tile width whose last round of units leaves the least idle.  A unit is split
// along K when there are fewer units than workers, into segments of at least 4 steps; the
// tensor-core shrink likewise, into at most 8.
LoraPlan lora_plan(int M, int K, int N, int R, bool has_w) {
  LoraPlan L;
  const int sms = 152;
  const int ksteps = (K + 63) / 64;
  L.ksteps = has_w ? ksteps : 0;
  if (M <= 256) {
    L.cg = 1;
    L.tile_n = (M + 15) / 16 * 16;
    L.tiles = 1;
  } else {
    L.cg = 2;
    long long best = -1;
    for (int tn = 256; tn >= 128; tn -= 16) {
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
  const long long units = (long long)L.tiles * L.blocks;
  L.splits = 1;
  if (units * 2 <= sms / L.cg) {
    L.splits = (int)(sms / L.cg / units);
    if (L.splits > L.ksteps / 4) L.splits = L.ksteps / 4 > 0 ? L.ksteps / 4 : 1;
  }
  // the fp32 shrink reads a token's adapter anew for each token: up to 16 MB of such reads
  L.tsplits = 0;
  if ((long long)M * R * K * 2 > (16LL << 20)) {
    int s = sms / L.tiles;
    if (s > ksteps / 4) s = ksteps / 4;
    L.tsplits = s < 1 ? 1 : s > 8 ? 8 : s;
  }
  return L;
}

cudaError_t launch_lora(LoraArgs& p, const LoraMaps& maps, int num_sms, cudaStream_t stream) {
  return p.dtype == QMOE_DTYPE_BF16 ? run<__nv_bfloat16>(p, maps, num_sms, stream)
                                    : run<__half>(p, maps, num_sms, stream);
}

}  // namespace qmoe
