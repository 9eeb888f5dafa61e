// The GEMM of the projection with adapters (lora.cu describes it).
#include <type_traits>

#include "cluster.cuh"
#include "lora.cuh"

namespace qmoe {
namespace {

constexpr int kBuilders = 8;  // warps
constexpr int kGemmThreads = 256 + 32 * kBuilders;
constexpr int kMaxStages = 12;
constexpr int kCtrl = 2048;
constexpr int kEpiStage = 4 * 2048;  // transpose tiles of the epilogue warps: 32 tokens x 32 rows
constexpr int kMaxSplits = 8;  // CTAs of a cluster, at most

// Bytes of one step of a CTA's token rows.
__host__ __device__ constexpr int token_bytes(int tile_n, int cg) { return tile_n / cg * 128; }
// The builders' operand (two of them a slot: t rounded, and the rest) has rows as long as an
// adapter's ranks ask for, in the swizzle of that length, so that more adapters are in the
// making where their steps are short (256 tokens of 64 adapters, K = N = 4096, R = 16: 33.4 us
// a call, with rows of 128 bytes 38.4; 2047 tokens of a few requests, R = 32: 54.1 and 57.6).
__host__ __device__ constexpr int t_pitch(int R) { return R <= 16 ? 32 : R <= 32 ? 64 : 128; }
__host__ __device__ constexpr int t_bytes(int tile_n, int cg, int R) {
  return tile_n / cg * t_pitch(R);
}
__host__ __device__ constexpr int token_slots(int tile_n, int cg, int R) {
  const int bytes = t_bytes(tile_n, cg, R);
  return bytes <= 48 * 128 ? 8 : bytes <= 64 * 128 ? 4 : 2;
}

// VEC: bytes of an adapter's 128 rows of B, and how many adapters are in flight (64 KB at
// most).  A power of two: step i's slot is i % vec_slots, and the kBuilders / vec_slots warps
// of a slot take all of its steps, since a wait on a phase's parity cannot tell it from the
// phase after the next (six slots among eight warps ran into that and timed out).
//
// Where it is taken: up to 64 tokens and 512 token-ranks, 1024 where at least as many adapters
// are loaded as there are tokens.  How many of them the tokens use is not known on the host: VEC
// pays for tokens, MMAs for distinct adapters.  Time of a call against the MMA form's, by the
// adapters that 16 to 64 tokens of K = N = 4096 and of K = 2048, N = 7168 use:
//   token-ranks   512          768          1024         1536         2048
//   one each      0.70 - 0.91  0.79 - 0.81  0.77 - 0.89  0.81 - 0.82  0.82 - 0.98
//   0.4 a token   0.87 - 0.96  0.92 - 1.01  0.91 - 1.03  0.99 - 1.07  0.97 - 1.16
//   four          0.96 - 1.07  1.02 - 1.18  0.98 - 1.25  1.16 - 1.31  1.11 - 1.41
// so 1024 loses least at worst: 1.25 inside, 1 / 0.81 outside.
constexpr int kVecTokens = 64;
__host__ constexpr int vec_token_ranks(int tokens, int L) { return L >= tokens ? 1024 : 512; }
__host__ __device__ constexpr int vec_slot_bytes(int R) { return 128 * R * 2; }
__host__ __device__ constexpr int vec_slots(int R) { return R <= 32 ? 8 : 4; }

// Bytes of shared memory behind the ring (multiples of 1024 each): the builders' slots, and
// (VEC) their copy of t and what they leave for the epilogue [tokens][128] in fp32.
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
    b.slots = round_kb(2 * token_slots(tile_n, cg, R) * t_bytes(tile_n, cg, R));
  }
  return b;
}

// Barrier of the builder warps.
__device__ __forceinline__ void builders_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kBuilders) : "memory");
}

__device__ __forceinline__ void fence_proxy_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ bool all_finite(const float (&f)[4]) {
  return fabsf(f[0]) < INFINITY && fabsf(f[1]) < INFINITY && fabsf(f[2]) < INFINITY &&
         fabsf(f[3]) < INFINITY;
}

// The spoiled rows (lora.cuh) of a CTA's unsplit units, which their epilogues left out; whole CTA.
template <class T>
__device__ __noinline__ void redo_units(const LoraArgs& p, int worker, int workers, int cg,
                                        int rank) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int first = warp >> 2, step = kGemmThreads / 128;
  for (int i = worker; i < p.tiles * p.blocks; i += workers) {
    const int tile = i / p.blocks, block = i - tile * p.blocks;
    const int n0 = (block * cg + rank) * 128 + (warp & 3) * 32, m0 = tile * p.tile_n;
    const int cols = min(p.tile_n, p.M - m0);
    const unsigned spoiled = __ballot_sync(0xffffffffu, spoiled_row<T>(p, tile, n0 + lane));
    if (spoiled && first < cols)
      redo_rows<T>(p, spoiled, n0, m0 + first, step, (cols - first + step - 1) / step);
  }
}

// What a CTA of a split unit left out: four rows n .. n + 3 of a token (n a multiple of 4) with a
// sum that is not finite.  Rows that are spoiled (lora.cuh) are made anew for all of the CTA's
// tokens, and the others get their sums.  n0: the CTA's first row; whole CTA.
template <class T>
__device__ __noinline__ void finish_odd(const LoraArgs& p, int tile, int n0, int seg, int cg,
                                        int rank, uint32_t sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, S = p.splits;
  const int m0 = tile * p.tile_n, cols = min(p.tile_n, p.M - m0);
  const int block = warp & 3, row = 32 * block + lane, n = n0 + row;
  const int first = seg + S * (warp >> 2), step = S * (kGemmThreads / 128);
  const unsigned spoiled = __ballot_sync(0xffffffffu, spoiled_row<T>(p, tile, n));
  const bool left = __ldcg(&p.any_left[tile]) != 0u;
  for (int c = first; c < cols; c += step) {
    float f = 0.f;
    for (int g = 0; g < S; ++g)
      f += ld_cluster_f32(peer_addr(sums + (c * 128 + row) * 4, g * cg + rank));
    if (left) f += left_products<T>(p, m0 + c, n);
    const unsigned bad = __ballot_sync(0xffffffffu, !(fabsf(f) < INFINITY));
    if ((bad >> (lane & ~3) & 15u) == 0u || n >= p.N || (spoiled >> lane & 1u)) continue;
    if (p.base) f += to_f32(reinterpret_cast<const T*>(p.base)[(m0 + c) * p.ldbase + n]);
    reinterpret_cast<T*>(p.out)[(size_t)(m0 + c) * p.N + n] = from_f32<T>(f);
  }
  __syncwarp();
  if (spoiled && first < cols)
    redo_rows<T>(p, spoiled, n0 + 32 * block, m0 + first, step, (cols - first + step - 1) / step);
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
  const int tslots = VEC ? vec_slots(p.R) : token_slots(p.tile_n, CG, p.R);
  const int pitch = t_pitch(p.R), half_slot = t_bytes(p.tile_n, CG, p.R);
  const Behind behind_ring = behind(VEC, p.tile_n, CG, p.R);
  uint8_t* tbuf = smem + stages * stage_bytes;  // [tslots][2][rows_b][pitch]; VEC [tslots][128][R]
  uint8_t* tcopy = tbuf + behind_ring.slots;    // VEC: fp32 [rows_b][R]
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
  volatile int* any_spoiled = abort_flag + 1;  // rows of this CTA's units are left out (below)
  // whether the builders (of the pair) left any of t to the epilogue, in whichever unit
  volatile int* any_left = any_spoiled + 1;
  short* place = reinterpret_cast<short*>(ctrl + 512);  // [rows_b] the tokens' adapters
  int* counts = reinterpret_cast<int*>(ctrl + 768);     // [kBuilders] the builders' lists of
  uint8_t* listed = ctrl + 1024;                        // [kBuilders][128] rows

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
    *any_spoiled = 0;
    *any_left = 0;
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
      const uint64_t tdesc0 = sdesc_swizzled(smem_u32(tbuf), pitch);
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
            const uint64_t hi = tdesc0 + ((2 * ts * half_slot) >> 4), lo = hi + (half_slot >> 4);
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
    // A slot's adapter is one or two warps' work, a lane having four or two of the 128 rows:
    // several adapters are in the making, with several sums a lane in flight (two groups of four
    // warps, a row a thread, took 0.65 us a step).
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
    // Step i goes to the warps of slot i % tslots, 32 of its rows a warp at a time.  Of a slot
    // only the rows of the step's adapter are written, and those of the step before it that
    // it has not are cleared: with an adapter a token a step is a row or two (128 tokens of 64
    // adapters, K = N = 4096, R = 64: 33.2 us a call, writing whole slots 42.7).  A lane's first
    // ranks of t are on their way before the slot is free.  This chain of instructions is what
    // a step costs, hence the row lengths at compile time (512 such tokens, R = 128: 124
    // us, at run time 144).
    // A unit of no more steps than slots has its rows written by all builders together: a tile
    // of one adapter would leave them to the warps of one slot (128 tokens, K = N = 4096,
    // R = 64: 20.1 us a call, by that slot's 23.3).
    auto build = [&](auto log_units) {
      constexpr int LG = decltype(log_units)::value, kUnits = 1 << LG;  // of 16 bytes a row
      constexpr int kWords = LG == 3 ? 2 : LG == 2 ? 3 : 4;  // 32 rows each, by the slots' sizes
      constexpr int kPitch = 16 << LG;
      const int group = kBuilders / tslots;
      const int own = (warp - 8) / group, part = (warp - 8) % group;
      uint8_t* const own_slot = tbuf + 2 * own * half_slot;
      uint8_t* const rows = listed + (warp - 8) * 128;  // this warp's rows of a step
      unsigned held[kWords] = {};                       // rows in the slot that are not zero,
      int held_units = 0;                               // and how many units of 16 bytes they have
      auto row0 = [&](int w) { return 32 * (part + w * group); };
      // a row's units of 16 bytes, swizzled by the 128-byte line that it is in
      auto put = [&](uint8_t* slot, int row, int j, uint4 hi, uint4 lo) {
        uint8_t* at = slot + row * kPitch + ((j ^ (row >> (3 - LG) & (kUnits - 1))) << 4);
        *reinterpret_cast<uint4*>(at) = hi;
        *reinterpret_cast<uint4*>(at + half_slot) = lo;
      };
      auto units_of = [&](int h) { return min(64, p.R - h * 64) / 8; };  // with ranks in them
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      for (int w = 0; row0(w) < rows_b; ++w)
        for (int u = lane; u < 32 * kUnits; u += 32)
          if (row0(w) + u / kUnits < rows_b)
            put(own_slot, row0(w) + u / kUnits, u % kUnits, zero, zero);
      uint32_t step = 0, tph = 1;
      bool ok = true;
      const uint32_t tfull0 = CG == 2 ? peer_addr(smem_u32(tfull), lead_rank) : smem_u32(tfull);
      auto arrive = [&]() {
        if (lane != 0) return;
        if (CG == 2 && rank != 0)
          mbar_arrive_remote(tfull0 + own * 8);
        else
          mbar_arrive(smem_u32(&tfull[own]));
      };
      auto tell = [&]() {
        *any_left = 1;
        if (CG == 2) st_cluster_u32(peer_addr(smem_u32((const void*)any_left), crank ^ 1u), 1u);
      };
      unsigned now[kWords];
      // this warp's rows of adapter d, times the units of a row
      auto list_rows = [&](int d) -> int {
        int found = 0;
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          const int row = row0(w) + lane;
          const bool in = row < rows_b && place[row] == d;
          now[w] = __ballot_sync(0xffffffffu, in);
          if (in) rows[found + __popc(now[w] & ((1u << lane) - 1u))] = (uint8_t)row;
          found += __popc(now[w]);
        }
        __syncwarp();
        return found * kUnits;
      };
      // waits until the slot's previous step has been used and clears what it leaves
      auto take_slot = [&](int units) {
        if (!wait(&tempty[own], tph)) return false;
        tph ^= 1;
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          unsigned left = held_units > units ? held[w] : held[w] & ~now[w];
          for (; left; left &= left - 1)
            if (lane < kUnits) put(own_slot, row0(w) + __ffs(left) - 1, lane, zero, zero);
          held[w] = now[w];
        }
        held_units = units;
        __syncwarp();
        return true;
      };
      // (after a wait that gave up a warp still meets the others at their barriers)
      for (int i = worker; i < units; i += workers) {
        const int tile = i / p.blocks;
        const int n = adapters(tile);
        const int m0 = tile * p.tile_n + (int)rank * rows_b;
        if (seg >= n) continue;    // the same for all builders
        builders_sync();           // the previous unit's rows have been used
        for (int r = threadIdx.x - 256; r < rows_b; r += 32 * kBuilders)
          place[r] = (short)p.place[(size_t)m0 + r];
        builders_sync();
        const int steps = (n - seg + S - 1) / S * chunks;
        if (steps <= tslots) {
          const int turn = step & (tslots - 1);
          auto step_of = [&](int slot) { return (slot - turn) & (tslots - 1); };
          const int j = step_of(own);
          int found = 0;
          if (j < steps && ok) {
            found = list_rows(seg + j / chunks * S);
            ok = take_slot(units_of(j % chunks));
          }
          if (lane == 0) counts[warp - 8] = ok ? found : 0;
          builders_sync();
          int ends[kBuilders];
#pragma unroll
          for (int o = 0; o < kBuilders; ++o) ends[o] = counts[o] + (o ? ends[o - 1] : 0);
          for (int v = threadIdx.x - 256; v < ends[kBuilders - 1]; v += 32 * kBuilders) {
            int o = 0, begin = 0;
#pragma unroll
            for (int e = 0; e < kBuilders - 1; ++e)
              if (v >= ends[e]) o = e + 1, begin = ends[e];
            const int row = listed[o * 128 + (v - begin) / kUnits], u = (v - begin) % kUnits;
            const int slot = o / group, h = step_of(slot) % chunks;
            uint4 hi, lo;
            if (u >= units_of(h)) continue;
            load_t8_split<T>(p, tile, m0 + row, h * 64 + u * 8, &hi, &lo, tell);
            put(tbuf + 2 * slot * half_slot, row, u, hi, lo);
          }
          fence_proxy_async();
          builders_sync();
          if (j < steps && ok) arrive();
          step += steps;
          continue;
        }
        for (int d = seg; d < n && ok; d += S) {
          for (int h = 0; h < chunks; ++h, ++step) {
            if ((int)(step & (tslots - 1)) != own) continue;
            const int found = list_rows(d), units = units_of(h);
            uint4 hi, lo;
            auto fetch = [&](int u) {
              load_t8_split<T>(p, tile, m0 + rows[u / kUnits], h * 64 + u % kUnits * 8, &hi, &lo,
                               tell);
            };
            const bool mine = lane % kUnits < units;  // (32 is a multiple of kUnits)
            if (mine && lane < found) fetch(lane);
            ok = take_slot(units);
            if (!ok) break;
            for (int u = lane; mine && u < found; u += 32) {
              if (u != lane) fetch(u);
              put(own_slot, rows[u / kUnits], u % kUnits, hi, lo);
            }
            fence_proxy_async();
            __syncwarp();
            arrive();
          }
        }
      }
    };
    if (pitch == 32)
      build(std::integral_constant<int, 1>{});
    else if (pitch == 64)
      build(std::integral_constant<int, 2>{});
    else
      build(std::integral_constant<int, 3>{});
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
      // (the builders' word came before the MMAs that the barrier stands for)
      const bool left = !VEC && S == 1 && *any_left && __ldcg(&p.any_left[tile]) != 0u;
      const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16) + ab * kAccCols;
      // the warp's rows that infinities or NaN in some B spoiled (lora.cuh): looked for where the
      // first token's sum is not finite
      unsigned spoiled = 0u;
      if (!VEC && S == 1 && any) {
        uint32_t first[16];
        tmem_ld_x16(tbase, first);
        tmem_wait_ld();
        tmem_ld_ready(first);
        if (__builtin_expect(
                __any_sync(0xffffffffu, !(fabsf(__uint_as_float(first[0])) < INFINITY)), 0))
          spoiled = __ballot_sync(0xffffffffu, spoiled_row<T>(p, tile, n0 + lane));
      }
      auto write_tile = [&](auto with_rest) {
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
            } else if constexpr (decltype(with_rest)::value) {
              if (left)
                add_left<T>(p, m0 + c0, cols - c0, n0 + lane, reinterpret_cast<float4*>(stage), v);
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
            if (p.wide && !(decltype(with_rest)::value && spoiled)) {
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const int tok = u * 8 + lane / 4, part = lane % 4 * 8;
                if (c0 + tok < cols && n0 + part < p.N)
                  *reinterpret_cast<uint4*>(out + (size_t)tok * p.N + part) =
                      *reinterpret_cast<const uint4*>(stage + tok * 32 + part);
              }
            } else if (n0 + lane < p.N && !(decltype(with_rest)::value && (spoiled >> lane & 1u))) {
              for (int k = 0; k < 32 && c0 + k < cols; ++k)
                out[(size_t)k * p.N + lane] = stage[k * 32 + lane];
            }
          }
        }
      };
      // (a loop of its own, since its registers cost the usual one 2 %)
      if (__builtin_expect(!VEC && (left || spoiled != 0u), 0))
        write_tile(std::true_type{});
      else
        write_tile(std::false_type{});
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2 && rank != 0)
          mbar_arrive_remote(acce0 + ab * 8);
        else
          mbar_arrive(smem_u32(&acce[ab]));
        if (VEC) mbar_arrive(smem_u32(dempty));
      }
      if (!VEC && spoiled) *any_spoiled = 1;
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
  if (!VEC && S == 1 && *any_spoiled) redo_units<T>(p, worker, workers, CG, (int)rank);
  if (S > 1) {
    // the unit's tokens seg, seg + S, .. over all segments: a warp per token, four rows a
    // lane, the segments' values in flight together
    const int tile = worker / p.blocks, block = worker - tile * p.blocks;
    const int m0 = tile * p.tile_n, cols = min(p.tile_n, p.M - m0);
    const int n = (block * CG + (int)rank) * 128 + 4 * lane;
    const bool left = !VEC && __ldcg(&p.any_left[tile]) != 0u;
    const uint32_t sums0 = smem_u32(smem) + 16 * lane;
    constexpr int kAtOnce = 2;  // tokens a warp
    bool odd = false;           // a sum that is not finite: looked at below
    const int stride = S * (kGemmThreads / 32);
    for (int c0 = seg + S * warp; c0 < cols; c0 += kAtOnce * stride) {
      float4 v[kAtOnce][kMaxSplits];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
        for (int g = 0; g < kMaxSplits; ++g)
          if (g < S && c0 + u * stride < cols && n < p.N)
            v[u][g] = ld_cluster_f32x4(peer_addr(sums0 + (c0 + u * stride) * 512, g * CG + rank));
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int c = c0 + u * stride;
        if (c >= cols || n >= p.N) break;
        float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int g = 0; g < kMaxSplits; ++g)
          if (g < S) t.x += v[u][g].x, t.y += v[u][g].y, t.z += v[u][g].z, t.w += v[u][g].w;
        if constexpr (VEC) {
          const float4 d = reinterpret_cast<const float4*>(delta + c / S * 128)[lane];
          t.x += d.x, t.y += d.y, t.z += d.z, t.w += d.w;
        }
        float f[4] = {t.x, t.y, t.z, t.w};
        if (!VEC && left)
          for (int e = 0; e < 4; ++e) f[e] += left_products<T>(p, m0 + c, n + e);
        if (!VEC && !all_finite(f)) {
          odd = true;
          continue;
        }
        const T* base = reinterpret_cast<const T*>(p.base) + (size_t)(m0 + c) * p.ldbase + n;
        T* out = reinterpret_cast<T*>(p.out) + (size_t)(m0 + c) * p.N + n;
        Pack<T, 4> o;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (p.base && n + e < p.N) f[e] += to_f32(base[e]);
          o.v[e] = from_f32<T>(f[e]);
        }
        if (p.wide) {
          *reinterpret_cast<uint2*>(out) = o.raw;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n + e < p.N) out[e] = o.v[e];
        }
      }
    }
    if (!VEC && __syncthreads_or(odd))
      finish_odd<T>(p, tile, (block * CG + (int)rank) * 128, seg, CG, (int)rank, smem_u32(smem));
    // No CTA leaves while its sums may still be read.  Every value fetched above has gone into
    // a store by now, so the barrier need not order memory (waiting for those stores took
    // 0.4 to 1 us: 128 tokens, K = N = 4096, R = 16: 16.6 us a call for 17.4).
    cluster_sync_relaxed();
  }
}

// Clusters of `size` CTAs of a kernel that the current device holds at once, 0 if it cannot say.
template <class K>
int resident_clusters(K* kernel, int size, int threads, size_t smem, int num_sms) {
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
  int n = 0;
  return cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess ? n : 0;
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
  cudaLaunchAttribute attr[2] = {pdl_attribute()};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  CUtensorMap map_x, map_w, map_b;
  cudaError_t e = gemm_maps(p, &map_x, &map_w, &map_b);
  if (e != cudaSuccess) return e;
  const int stage = kStageA + token_bytes(p.tile_n, p.cg);
  const bool vec = p.cg == 1 && p.tile_n <= kVecTokens &&
                   p.tile_n * p.R <= vec_token_ranks(p.M, p.L);
  const Behind more = behind(vec, p.tile_n, p.cg, p.R);
  const int other = 1024 + kCtrl + kEpiStage + more.slots + more.copy + more.delta;
  const int most = (kSmemLimit - other) / stage;
  p.stages = most < kMaxStages ? most : kMaxStages;
  // every plan's shared memory leaves one CTA an SM
  const size_t smem = other + (size_t)p.stages * stage;
  auto* k = p.cg == 2 ? lora_gemm_kernel<T, 2, false>
            : vec     ? lora_gemm_kernel<T, 1, true>
                      : lora_gemm_kernel<T, 1, false>;
  e = allow_smem(k, kSmemLimit);
  if (e != cudaSuccess) return e;
  const int units = p.tiles * p.blocks;
  int dev = -1;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  // asked of the runtime once per device, kernel and size (devices of one model can have their
  // SMs in clusters of different sizes)
  static PerDevice<3 * (kMaxSplits + 1)> clusters;
  auto clusters_of = [&](int splits) {
    const int size = p.cg * splits;
    if (size == 1) return num_sms;
    return clusters.get(dev, (vec ? 2 : p.cg - 1) * (kMaxSplits + 1) + splits, [&] {
      return resident_clusters(k, size, kGemmThreads, smem, num_sms);
    });
  };
  // Segments: where every unit's cluster is resident at once, each has 4 steps or more and a
  // CTA's sums fit over its ring, as many as there can be
  p.splits = 1;
  const bool sums_fit = p.tile_n * 512 <= p.stages * stage;
  for (int s = sums_fit ? kMaxSplits / p.cg : 1; s > 1 && p.splits == 1; --s)
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

cudaError_t launch_lora_gemm(LoraArgs& p, int num_sms, cudaStream_t stream) {
  return p.dtype == QMOE_DTYPE_BF16 ? run<__nv_bfloat16>(p, num_sms, stream)
                                    : run<__half>(p, num_sms, stream);
}

}  // namespace qmoe
