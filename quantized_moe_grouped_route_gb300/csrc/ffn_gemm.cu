// The products of the gated feed-forward block for many tokens, forward and backward, on the
// tensor cores: one persistent kernel on CTA pairs whose operands are taken as they lie in memory,
// rows along the contraction (K) or across it, and whose epilogues do the rest of the block.
//
//   up      [u | g] = x . W13^T, h = act(g) u         x: K, W13: K     (W13 [2I][H], rows 0..I-1 up)
//   plain   out = h . W2^T                            h: K, W2: K      (W2 [H][I])
//   dh      dh = dout . W2, then du, dg and h again   dout: K, W2: across
//   plain   dx = [du | dg] . W13                      [du | dg]: K, W13: across
//   plain   dW13 = [du | dg]^T . x, dW2 = dout^T . h  both across, K are the tokens
//
// A tile is 256 rows x tile_n columns of the accumulator, half of the rows in each SM of the pair
// (tcgen05 cta_group::2, M = 256; each SM loads its own 128 rows of A and half of B's columns, so
// an operand passes the memory system once a pair).  Steps of 64 of K go through a ring of
// TMA-loaded stages; two accumulators in TMEM let a tile's epilogue run under the next one's MMAs.
// The up tile holds tile_n / 2 columns of u beside the same columns of g: one SM loads the rows of
// W13 for u and the other those for g, and the epilogue finds both of a pair in one TMEM lane.
// Epilogues write through swizzled staging tiles and TMA stores, which cut at the matrix's edges.
// Bound by the tensor cores: 8192 tokens, H = 7168, I = 2048, 436 to 450 us a call by the power left
// (1.60 to 1.65 PFLOP/s, the tensor pipes 87 to 92 % active), backward 927 to 970 us; smaller batches
// by the last round of tiles and what a launch costs to begin and end.
#include <type_traits>

#include "checkpoint.cuh"
#include "cluster.cuh"
#include "ffn.cuh"
#include "ffn_tiles.h"
#include "mma.cuh"

namespace qmoe {
namespace {

constexpr int kEpiWarps = 8;  // two a lane quarter of TMEM, 32 columns in turn
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr int kMaxStages = 12;
constexpr int kCtrl = 1024;
constexpr int kAccCols = 256;
constexpr int kABytes = 128 * 128;  // a stage's A: 128 rows x 64 of K
constexpr int kStageTile = 2048;    // an epilogue warp's staging tile: 32 rows x 32 columns
constexpr int kSmemLimit = 232448;

// kMany: up to three products of their own sizes and operands' lie in one launch, plain epilogues.
enum class Op { kUp, kDh, kMany };
constexpr int kMost = 3;
// Staging tiles of an epilogue warp.
__host__ __device__ constexpr int staging(Op op) { return op == Op::kMany ? 2 : 3; }

struct Maps {
  CUtensorMap a, b, b2, o, o2, o3;
  CUtensorMap a_edge, b_edge, b2_edge;  // the operands in boxes of a last block's rows
};
template <int N>
struct Launch {
  int count, stages, stage_bytes;
  FfnGemm p[N];
  Maps maps[N];
};
constexpr int problems(Op op) { return op == Op::kMany ? kMost : 1; }

__device__ __forceinline__ uint64_t l2_policy_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void store_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void store_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// Descriptor of an operand that lies across K: boxes of 64 elements (128 bytes, swizzled) x 64
// of K.  Eight of K are 1024 bytes apart (stride offset), the next 64 elements a box (leading).
__device__ __forceinline__ uint64_t sdesc_across(uint32_t saddr) {
  return (sdesc_sw128(saddr) & ~((uint64_t)0x3fff << 16)) | (uint64_t)(64 * 128 >> 4) << 16;
}

// 16 values of a lane's row into half `half` of a staging tile (64-byte rows, swizzled as the
// store's tensor map has it).
template <class T>
__device__ __forceinline__ void stage_half(uint8_t* tile, int half, const float* v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    Pack<T, 8> p;
#pragma unroll
    for (int e = 0; e < 8; ++e) p.v[e] = from_f32<T>(v[8 * j + e]);
    *reinterpret_cast<uint4*>(tile + lane * 64 + (((half * 2 + j) ^ (lane >> 1 & 3)) << 4)) = p.raw;
  }
}
template <class T>
__device__ __forceinline__ void stage_row(uint8_t* tile, const float (&v)[32]) {
  stage_half<T>(tile, 0, v);
  stage_half<T>(tile, 1, v + 16);
}
// ... of u or g, which is kept within T's finite range: a gate past it is open or closed, where an
// infinity's product with sigmoid's 0 would leave NaN.
template <class T>
__device__ __forceinline__ void stage_kept(uint8_t* tile, const float (&v)[32]) {
  float f[32];
#pragma unroll
  for (int k = 0; k < 32; ++k) f[k] = within<T>(v[k]);
  stage_row<T>(tile, f);
}

__device__ __forceinline__ void load_acc16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  tmem_ld_x16(taddr, r);
  tmem_wait_ld();
  tmem_ld_ready(r);
#pragma unroll
  for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(r[k]);
}
__device__ __forceinline__ void load_acc32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[2][16];
  tmem_ld_x16(taddr, r[0]);
  tmem_ld_x16(taddr + 16, r[1]);
  tmem_wait_ld();
  tmem_ld_ready(r[0]);
  tmem_ld_ready(r[1]);
#pragma unroll
  for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(r[k >> 4][k & 15]);
}

// A row's 32 values as 8-bit codes and their scale (checkpoint.cuh); n <= 32 of them exist, a
// multiple of 8.
__device__ __forceinline__ void save_block(const float (&v)[32], int n, int8_t* codes,
                                           uint8_t* scale) {
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < 32; ++k)
    if (k < n) top = max(top, __float_as_uint(v[k]) & 0x7fffffffu);
  const uint32_t byte = ck_byte(top);
  const float inverse = ck_inverse(byte);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (8 * j >= n) break;
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w[i] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[i] |= (uint32_t)(ck_code(v[8 * j + 4 * i + e], inverse) & 255) << (8 * e);
    }
    *reinterpret_cast<uint2*>(codes + 8 * j) = make_uint2(w[0], w[1]);
  }
  *scale = (uint8_t)byte;
}

// A row's 32 kept values of u or g on their way: 16-bit or codes with a scale.
struct Kept {
  uint4 raw[4];
  uint32_t byte;
};
// 16 bytes, or zeros.  (Two lie in a sector, so they may stay in L1: past it each would fetch the sector,
// twice the bytes through L2's ports, which the operands need: 8192 tokens, H = 7168, I = 2048, the
// kernel 172 us, past L1 183.)
__device__ __forceinline__ uint4 load_l1_if(const uint4* p, bool there) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
      "@p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"((int)there));
  return v;
}
template <class T, bool CODES>
__device__ __forceinline__ void fetch_kept(Kept& k, const FfnGemm& p, int row, int col, int half) {
  const size_t at = (size_t)row * 2 * p.N + (size_t)half * p.N + col;
  const bool in = row < p.M;
  if constexpr (CODES) {
    const uint8_t* src = reinterpret_cast<const uint8_t*>(p.kept) + at;
    uint2 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = load_if(reinterpret_cast<const uint2*>(src + 8 * j), in && col + 8 * j < p.N);
    k.raw[0] = make_uint4(v[0].x, v[0].y, v[1].x, v[1].y);
    k.raw[1] = make_uint4(v[2].x, v[2].y, v[3].x, v[3].y);
    const int blocks = (p.N + kCkBlock - 1) / kCkBlock;
    k.byte = in && col < p.N ? p.kept_scales[((size_t)row * 2 + half) * blocks + col / kCkBlock] : 0u;
  } else {
    const T* src = reinterpret_cast<const T*>(p.kept) + at;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      k.raw[j] = load_l1_if(reinterpret_cast<const uint4*>(src + 8 * j), in && col + 8 * j < p.N);
  }
}
template <class T, bool CODES>
__device__ __forceinline__ float kept_value(const Kept& k, int i, float value) {
  const uint32_t w[16] = {k.raw[0].x, k.raw[0].y, k.raw[0].z, k.raw[0].w, k.raw[1].x, k.raw[1].y,
                          k.raw[1].z, k.raw[1].w, k.raw[2].x, k.raw[2].y, k.raw[2].z, k.raw[2].w,
                          k.raw[3].x, k.raw[3].y, k.raw[3].z, k.raw[3].w};
  if constexpr (CODES) {
    return ck_restore<T>((int)(int8_t)(w[i >> 2] >> (8 * (i & 3)) & 255u), value);
  } else {
    Pack<T, 2> v;
    v.raw = w[i >> 1];
    return to_f32(v.v[i & 1]);
  }
}

// Tile i of a matrix of tiles: groups of eight rows of tiles, a group column by column, so that
// the tiles in the making at one time share few rows of A and of B (both stay in L2).
__device__ __forceinline__ void tile_of(const FfnGemm& p, int i, int* tm, int* tn) {
  const int group = 8 * p.tiles_n, first = i / group * 8;
  const int rows = min(8, p.tiles_m - first), r = i - first * p.tiles_n;
  *tn = r / rows;
  *tm = first + r - *tn * rows;
}
// Unit i of a launch: a tile of one of its products, and of K the segment `seg`.
struct Unit {
  int problem, tm, tn, seg, k0, k1;
};
template <int N>
__device__ __forceinline__ Unit unit_of(const Launch<N>& L, int i) {
  Unit u;
  u.problem = 0;
#pragma unroll
  for (int j = 1; j < N; ++j)
    if (j < L.count && i >= L.p[j].first) u.problem = j;
  const FfnGemm& p = L.p[u.problem];
  i -= p.first;
  const int tile = i / p.splits;
  u.seg = i - tile * p.splits;
  u.k0 = (int)((long long)p.ksteps * u.seg / p.splits);
  u.k1 = (int)((long long)p.ksteps * (u.seg + 1) / p.splits);
  tile_of(p, tile, &u.tm, &u.tn);
  return u;
}

// A product whose K is cut into segments leaves each segment's sums in p.part [splits][M][columns]
// (u's columns before g's) for the kernels of ffn_finish.cu; PART: whether kUp's and kDh's does.
template <class T, Op OP, bool CODES, bool PART>
__global__ void __launch_bounds__(kThreads, 1)
    ffn_gemm_kernel(const __grid_constant__ Launch<problems(OP)> L) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int stage_bytes = L.stage_bytes, stages = L.stages;
  uint8_t* epi = smem + stages * stage_bytes;
  uint8_t* ctrl = epi + kEpiWarps * staging(OP) * kStageTile;
  uint64_t* full = reinterpret_cast<uint64_t*>(ctrl);
  uint64_t* empty = full + kMaxStages;
  uint64_t* accf = empty + kMaxStages;
  uint64_t* acce = accf + 2;
  uint64_t* drain = acce + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  unsigned int* const err = L.p[0].err;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int worker = (int)cluster_index(), workers = (int)cluster_count();
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&accf[i]), 1);
      mbar_init(smem_u32(&acce[i]), 2 * kEpiWarps);  // of both SMs
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    fence_mbar_init();
    for (int j = 0; j < L.count; ++j) {
      prefetch_tmap(&L.maps[j].a);
      prefetch_tmap(&L.maps[j].b);
      if (OP == Op::kUp) prefetch_tmap(&L.maps[j].b2);
      prefetch_tmap(&L.maps[j].o);
    }
  }
  if (warp == 1) {
    tmem_alloc2(smem_u32(tmem_slot), 2 * kAccCols);
    tmem_relinquish2();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the peer's barriers exist before any remote arrival
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dep_wait();  // (all threads: what they read was written by the kernel before)
  grid_dep_launch();
  if (L.p[0].clear_err && blockIdx.x == 0 && threadIdx.x == 0) *err = 0;

  const FfnGemm& last = L.p[L.count - 1];
  const int units = last.first + last.tiles_m * last.tiles_n * last.splits;
  // the operands' lie
  auto a_across = [&](const FfnGemm& p) { return OP == Op::kMany && p.op == FfnOp::kTN; };
  auto b_across = [&](const FfnGemm& p) {
    return OP == Op::kDh || (OP == Op::kMany && p.op != FfnOp::kNT);
  };
  // f with the lie of both operands as constants
  auto by_lie = [&](bool across_a, bool across_b, auto&& f) {
    if constexpr (OP == Op::kUp) {
      f(std::false_type{}, std::false_type{});
    } else if constexpr (OP == Op::kDh) {
      f(std::false_type{}, std::true_type{});
    } else if (across_a) {
      f(std::true_type{}, std::true_type{});
    } else if (across_b) {
      f(std::false_type{}, std::true_type{});
    } else {
      f(std::false_type{}, std::false_type{});
    }
  };
  // columns of the result, a tile
  auto tile_cols = [&](const FfnGemm& p) { return OP == Op::kUp ? p.tile_n / 2 : p.tile_n; };
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return warp_wait_cl(smem_u32(bar), parity, abort_flag, err);
  };

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    const uint32_t lead = elect_one();
    const uint64_t pol = l2_policy_normal();
    const uint32_t full0 = peer_addr(smem_u32(full), 0);  // the leader's: both SMs' copies count
    uint32_t s = 0, ph = 1;
    bool ok = true;
    for (int i = worker; i < units && ok; i += workers) {
      const Unit u = unit_of(L, i);
      const FfnGemm& p = L.p[u.problem];
      const Maps& maps = L.maps[u.problem];
      const bool across_a = a_across(p), across_b = b_across(p);
      const int rows_b = p.tile_n / 2, K = p.K;
      const uint32_t bytes = 2u * (kABytes + rows_b * 128);  // of a whole step, both SMs
      const Share shares[2] = {share_of(p.M, p.N, p.tile_n, OP == Op::kUp, u.tm, u.tn, 0),
                               share_of(p.M, p.N, p.tile_n, OP == Op::kUp, u.tm, u.tn, 1)};
      const Share own = rank == 0 ? shares[0] : shares[1];
      const int row = own.row, col = own.col, na = own.rows, nb = own.cols;
      const bool second = OP == Op::kUp && rank != 0;  // the SM with the rows of g
      const CUtensorMap* const map_b = second ? &maps.b2 : &maps.b;
      // steps of whole boxes (a tile whose second half is whole is whole), one copy an operand, two
      // across K: the issue is what paces a step
      const int k_whole =
          shares[1].rows == 128 && shares[1].cols == rows_b ? min(u.k1, K / 64) : u.k0;
      auto steps = [&](auto lie_a, auto lie_b) {
        constexpr bool kA = decltype(lie_a)::value, kB = decltype(lie_b)::value;
        for (int k = u.k0; k < u.k1; ++k) {
          if (!wait(&empty[s], ph)) {
            ok = false;
            break;
          }
          const uint32_t sa = smem_u32(smem) + s * stage_bytes, sb = sa + kABytes;
          const uint32_t bar = full0 + s * 8;
          if (k < k_whole) {
            if (rank == 0) mbar_arrive_expect_tx_if(lead, smem_u32(&full[s]), bytes);
            if constexpr (kA) {
              tma_load_2d_pair_if(lead, sa, &maps.a, row, k * 64, bar, pol);
              tma_load_2d_pair_if(lead, sa + 8192, &maps.a, row + 64, k * 64, bar, pol);
            } else {
              tma_load_2d_pair_if(lead, sa, &maps.a, k * 64, row, bar, pol);
            }
            if constexpr (kB) {
              tma_load_2d_pair_if(lead, sb, map_b, col, k * 64, bar, pol);
              if (rows_b > 64) tma_load_2d_pair_if(lead, sb + 8192, map_b, col + 64, k * 64, bar, pol);
            } else {
              tma_load_2d_pair_if(lead, sb, map_b, k * 64, col, bar, pol);
            }
          } else {
            const bool deep = k < K / 64;  // a whole step of K
            const int depth = deep ? 64 : last_deep(K);
            if (rank == 0) {
              uint32_t rows = 0;  // of 128 bytes, of both SMs
#pragma unroll
              for (int r = 0; r < 2; ++r)
                rows += (kA ? (shares[r].rows + 63) / 64 * depth : shares[r].rows) +
                        (kB ? (shares[r].cols + 63) / 64 * depth : shares[r].cols);
              mbar_arrive_expect_tx_if(lead, smem_u32(&full[s]), rows * 128u);
            }
            if constexpr (kA) {
              for (int c = 0; c < na; c += 64)
                tma_load_2d_pair_if(lead, sa + c * 128, deep ? &maps.a : &maps.a_edge, row + c, k * 64,
                                    bar, pol);
            } else {
              if (na > 0)
                tma_load_2d_pair_if(lead, sa, na == 128 ? &maps.a : &maps.a_edge, k * 64, row, bar, pol);
            }
            if constexpr (kB) {
              for (int c = 0; c < nb; c += 64)
                tma_load_2d_pair_if(lead, sb + c * 128, deep ? &maps.b : &maps.b_edge, col + c, k * 64,
                                    bar, pol);
            } else {
              const CUtensorMap* b = nb == rows_b ? map_b : second ? &maps.b2_edge : &maps.b_edge;
              if (nb > 0) tma_load_2d_pair_if(lead, sb, b, k * 64, col, bar, pol);
            }
          }
          if (++s == (uint32_t)stages) {
            s = 0;
            ph ^= 1;
          }
        }
      };
      by_lie(across_a, across_b, steps);
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
      const uint32_t base = smem_u32(smem);
      uint32_t s = 0, ph = 0, local = 0;
      bool ok = true;
      for (int i = worker; i < units && ok; i += workers, ++local) {
        const Unit u = unit_of(L, i);
        const FfnGemm& p = L.p[u.problem];
        const bool across_a = a_across(p), across_b = b_across(p);
        uint32_t idesc = idesc_16bit(256, p.tile_n, p.dtype);
        idesc |= (across_a ? 1u << 15 : 0u) | (across_b ? 1u << 16 : 0u);
        const uint64_t a0 = across_a ? sdesc_across(base) : sdesc_sw128(base);
        const uint64_t b0 = across_b ? sdesc_across(base + kABytes) : sdesc_sw128(base + kABytes);
        const int k0 = u.k0, whole = p.K / 64;
        const int ab = local & 1;
        if (!wait(&acce[ab], ((local >> 1) & 1) ^ 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t dst = tmem + ab * kAccCols;
        auto steps = [&](auto lie_a, auto lie_b) {
          // 16 of K further on: 32 bytes of a row, or 16 rows of 128 bytes
          constexpr uint32_t step_a = decltype(lie_a)::value ? 128 : 2;
          constexpr uint32_t step_b = decltype(lie_b)::value ? 128 : 2;
          for (int k = k0; k < u.k1; ++k) {
            if (!wait(&full[s], ph)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t off = (s * stage_bytes) >> 4;
            if (k < whole) {
              if (lead) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  mma_ss(2, dst, a0 + off + step_a * j, b0 + off + step_b * j, idesc, (k > k0) | (j > 0));
              }
            } else if (lead) {  // the slices of 16 that there are
              for (int j = 0; j < (p.K - k * 64 + 15) / 16; ++j)
                mma_ss(2, dst, a0 + off + step_a * j, b0 + off + step_b * j, idesc, (k > k0) | (j > 0));
            }
            tc_commit2_both_if(lead, smem_u32(&empty[s]));
            if (++s == (uint32_t)stages) {
              s = 0;
              ph ^= 1;
            }
          }
        };
        by_lie(across_a, across_b, steps);
        if (ok) tc_commit2_both_if(lead, smem_u32(&accf[ab]));
      }
      tc_commit2_both_if(lead, smem_u32(drain));
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------------- epilogue
    const int q = warp & 3, first_col = 32 * ((warp - 4) >> 2);
    constexpr int kApart = 32 * (kEpiWarps / 4);  // a warp's columns
    const uint32_t acce0 = peer_addr(smem_u32(acce), 0);
    uint8_t* stage = epi + (warp - 4) * staging(OP) * kStageTile;
    const uint32_t stage0 = smem_u32(stage);
    const bool gelu = L.p[0].activation == QMOE_ACT_GELU;
    uint32_t local = 0;
    int turn = 0;
    for (int i = worker; i < units; i += workers, ++local) {
      const Unit unit = unit_of(L, i);
      const FfnGemm& p = L.p[unit.problem];
      const Maps& maps = L.maps[unit.problem];
      const bool part = OP == Op::kMany ? p.splits > 1 : PART;
      const int ab = local & 1, cols = tile_cols(p);
      const int row0 = unit.tm * 256 + (int)rank * 128 + q * 32, col0 = unit.tn * cols;
      const int n = min(cols, p.N - col0);  // columns of this tile
      Kept ku, kg;
      if constexpr (OP == Op::kDh && !PART) {
        fetch_kept<T, CODES>(ku, p, row0 + lane, col0 + first_col, 0);
        fetch_kept<T, CODES>(kg, p, row0 + lane, col0 + first_col, 1);
      }
      if (!wait(&accf[ab], (local >> 1) & 1)) break;
      tc_fence_after();
      const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16) + ab * kAccCols;
      const bool rows_in = row0 < p.M;
      for (int c = first_col; c < n; c += kApart) {
        if (part) {
          // a lane's row in pieces of 128 bytes
          const int width = OP == Op::kUp ? 2 * p.N : p.N;
          float* to = p.part + ((size_t)unit.seg * p.M + row0 + lane) * width + col0 + c;
#pragma unroll
          for (int half = 0; half < (OP == Op::kUp ? 2 : 1); ++half) {
            float v[32];
            load_acc32(tbase + half * (p.tile_n / 2) + c, v);
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              if (row0 + lane < p.M && c + k < n)
                *reinterpret_cast<float4*>(to + half * p.N + k) =
                    make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
          }
        } else if constexpr (!PART) {
          // the staging tiles are free again
          const int t = OP == Op::kUp || OP == Op::kDh ? 0 : turn;
          turn ^= 1;
          if (lane == 0) {
            if (OP == Op::kUp || OP == Op::kDh)
              store_wait_read<0>();
            else
              store_wait_read<1>();
          }
          __syncwarp();
          if constexpr (OP == Op::kUp) {
            float u[32], g[32];
            load_acc32(tbase + c, u);
            load_acc32(tbase + p.tile_n / 2 + c, g);
            if (p.save == 8 && row0 + lane < p.M) {
              const int blocks = (p.N + kCkBlock - 1) / kCkBlock;
              const size_t at = (size_t)(row0 + lane) * 2 * p.N + col0 + c;
              const size_t sat = (size_t)(row0 + lane) * 2 * blocks + (col0 + c) / kCkBlock;
              save_block(u, min(32, n - c), p.codes + at, p.scales + sat);
              save_block(g, min(32, n - c), p.codes + at + p.N, p.scales + sat + blocks);
            }
            if (p.save == 16) {
              stage_kept<T>(stage + kStageTile, u);
              stage_kept<T>(stage + 2 * kStageTile, g);
            }
#pragma unroll
            for (int k = 0; k < 32; ++k) u[k] = gated(gelu, p.limit, u[k], g[k]);
            stage_row<T>(stage, u);
          } else if constexpr (OP == Op::kDh) {
            const float su = CODES ? ck_value(ku.byte) : 0.f, sg = CODES ? ck_value(kg.byte) : 0.f;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              float v[16], du[16], dg[16];
              load_acc16(tbase + c + 16 * half, v);
#pragma unroll
              for (int k = 0; k < 16; ++k)
                v[k] = gated_backward(gelu, p.limit, kept_value<T, CODES>(ku, 16 * half + k, su),
                                      kept_value<T, CODES>(kg, 16 * half + k, sg), v[k], &du[k],
                                      &dg[k]);
              stage_half<T>(stage, half, v);
              stage_half<T>(stage + kStageTile, half, du);
              stage_half<T>(stage + 2 * kStageTile, half, dg);
            }
            if (c + kApart < n) {
              fetch_kept<T, CODES>(ku, p, row0 + lane, col0 + c + kApart, 0);
              fetch_kept<T, CODES>(kg, p, row0 + lane, col0 + c + kApart, 1);
            }
          } else {
            float v[32];
            load_acc32(tbase + c, v);
            stage_row<T>(stage + t * kStageTile, v);
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0 && rows_in) {
            tma_store_2d(&maps.o, stage0 + t * kStageTile, col0 + c, row0);
            if (OP == Op::kDh || (OP == Op::kUp && p.save == 16)) {
              tma_store_2d(&maps.o2, stage0 + kStageTile, col0 + c, row0);
              tma_store_2d(&maps.o3, stage0 + 2 * kStageTile, col0 + c, row0);
            }
          }
          if (lane == 0) store_commit();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank != 0)
          mbar_arrive_remote(acce0 + ab * 8);
        else
          mbar_arrive(smem_u32(&acce[ab]));
      }
    }
    if (lane == 0) store_wait_all();
  }

  // No MMA may still read this SM's shared memory or write its TMEM, and no remote arrival may be
  // in flight, when it (or its peer) exits.
  if (warp == 1) drain_wait_cl(smem_u32(drain), 0);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc2(tmem, 2 * kAccCols);
  }
}

// An output [rows][cols], rows ld elements apart, in the epilogue's staging tiles.
bool map_out(CUtensorMap* map, int dtype, const void* base, long long rows, int cols, long long ld) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows}, strides[1] = {(uint64_t)ld * 2};
  const uint32_t box[2] = {32, 32};
  return make_tmap16(map, dtype, base, 2, dims, strides, box, 64) == QMOE_OK;
}

template <class T, Op OP, bool CODES, bool PART>
cudaError_t run_as(Launch<problems(OP)>& L, int num_sms, cudaStream_t stream) {
  auto* k = ffn_gemm_kernel<T, OP, CODES, PART>;
  int tile_n = 0, units = 0;
  for (int j = 0; j < L.count; ++j) {
    FfnGemm& p = L.p[j];
    p.first = units;
    units += p.tiles_m * p.tiles_n * p.splits;
    if (p.tile_n > tile_n) tile_n = p.tile_n;
  }
  L.stage_bytes = kABytes + tile_n / 2 * 128;
  const int other = 1024 + kCtrl + kEpiWarps * staging(OP) * kStageTile;
  const int most = (kSmemLimit - other) / L.stage_bytes;
  L.stages = most < kMaxStages ? most : kMaxStages;
  cudaError_t e = allow_smem(k, kSmemLimit);
  if (e != cudaSuccess) return e;
  int dev = -1;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  // asked of the runtime once per device: all plans leave one pair two SMs
  static PerDevice<1> clusters;
  const int held = clusters.get(dev, 0, [&] {
    return resident_clusters(k, 2, kThreads, kSmemLimit, num_sms);
  });
  if (held < 1) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2] = {pdl_attribute()};
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)((units < held ? units : held) * 2));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = other + (size_t)L.stages * L.stage_bytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, k, L);
  for (int j = 0; j < L.count && e == cudaSuccess; ++j)
    if (L.p[j].splits > 1) e = launch_ffn_finish(L.p[j], stream);
  return e;
}

template <class T, Op OP, bool CODES>
cudaError_t run(Launch<problems(OP)>& L, int num_sms, cudaStream_t stream) {
  if constexpr (OP != Op::kMany)
    if (L.p[0].splits > 1) return run_as<T, OP, false, true>(L, num_sms, stream);
  return run_as<T, OP, CODES, false>(L, num_sms, stream);
}

constexpr int kPairs = 76;  // of SMs of a GB300: results are the same on every part

// How a product alone in its launch is cut: tiles of 256 or 128 columns, and their K steps into
// segments where the tiles are far fewer than the pairs of SMs.  By an estimate of the time in units
// of a step of a wide tile (0.27 us): a step of a tile of 128 columns takes 0.75 (its operands come at
// the rate at which L2 feeds an SM), a tile's last epilogue about 8, segments another kernel of about
// 12 and their sums written and read again in L2.  (3000 tokens, H = 7168, I = 2048: 166 us a call,
// with 0.55 182; backward of 1023 tokens, 4096 x 1000: 66 us, without segments in its first product 74.)
void cut_alone(FfnGemm& p) {
  const bool up = p.op == FfnOp::kUp;
  double best = 0;
  for (int n = 256; n >= 128; n /= 2) {
    const int cols = up ? n / 2 : n, tiles_n = (p.N + cols - 1) / cols;
    const long long tiles = (long long)p.tiles_m * tiles_n;
    for (int s = 1; s <= kFfnMaxSplits && (s == 1 || (tiles * s <= kPairs && p.ksteps >= 4 * s)); ++s) {
      const double waves = (double)((tiles * s + kPairs - 1) / kPairs);
      const double steps = (p.ksteps + s - 1) / s * (n == 256 ? 1.0 : 0.75);
      const double sums = (double)s * p.M * p.N * (up ? 2 : 1) * 8;
      const double cost = waves * steps + (n == 256 ? 8 : 4) + (s > 1 ? 12 + sums / 2.7e6 : 0);
      if (best != 0 && cost >= best) continue;
      best = cost;
      p.tile_n = n;
      p.tiles_n = tiles_n;
      p.splits = s;
    }
  }
}

// Products that share a launch: narrow tiles where wide ones are fewer than two for each pair of SMs,
// and K in segments where a tile has more steps than twice a pair's share of all of them.
void cut_together(FfnGemm* p, int count) {
  auto tiles = [&](int j, int n) { return (long long)p[j].tiles_m * ((p[j].N + n - 1) / n); };
  long long wide = 0;
  double steps = 0;
  for (int j = 0; j < count; ++j) wide += tiles(j, 256);
  for (int j = 0; j < count; ++j) {
    p[j].tile_n = wide >= 2 * kPairs ? 256 : 128;
    p[j].tiles_n = (p[j].N + p[j].tile_n - 1) / p[j].tile_n;
    steps += (double)tiles(j, p[j].tile_n) * p[j].ksteps;
  }
  const double share = steps / kPairs;
  for (int j = 0; j < count; ++j) {
    const long long n = tiles(j, p[j].tile_n);
    int s = 1;
    while (s < kFfnMaxSplits && p[j].ksteps > 2 * s * (share > 16 ? share : 16) &&
           n * (s + 1) <= kPairs && p[j].ksteps >= 4 * (s + 1))
      ++s;
    p[j].splits = s;
  }
}

// The tensor maps of a product.
template <class T>
bool maps_of(const FfnGemm& p, Maps* m) {
  const bool across_a = p.op == FfnOp::kTN;
  const bool across_b = p.op == FfnOp::kTN || p.op == FfnOp::kNN || p.op == FfnOp::kDh;
  bool ok = across_a ? map_of(&m->a, p.dtype, p.a, p.K, p.M, p.lda, 64) &&
                           map_of(&m->a_edge, p.dtype, p.a, p.K, p.M, p.lda, last_deep(p.K))
                     : map_of(&m->a, p.dtype, p.a, p.M, p.K, p.lda, 128) &&
                           map_of(&m->a_edge, p.dtype, p.a, p.M, p.K, p.lda, last_rows(p.M, 128));
  const int half = p.tile_n / 2, edge = last_rows(p.N, half);
  ok = ok && (across_b ? map_of(&m->b, p.dtype, p.b, p.K, p.N, p.ldb, 64) &&
                             map_of(&m->b_edge, p.dtype, p.b, p.K, p.N, p.ldb, last_deep(p.K))
                       : map_of(&m->b, p.dtype, p.b, p.N, p.K, p.ldb, half) &&
                             map_of(&m->b_edge, p.dtype, p.b, p.N, p.K, p.ldb, edge));
  m->b2 = m->b;
  m->b2_edge = m->b_edge;
  if (p.op == FfnOp::kUp) {  // w13's rows for g
    const T* g = reinterpret_cast<const T*>(p.b) + (size_t)p.N * p.ldb;
    ok = ok && map_of(&m->b2, p.dtype, g, p.N, p.K, p.ldb, half) &&
         map_of(&m->b2_edge, p.dtype, g, p.N, p.K, p.ldb, edge);
  }
  ok = ok && map_out(&m->o, p.dtype, p.out, p.M, p.N, p.N);
  m->o2 = m->o3 = m->o;
  if (p.op == FfnOp::kDh || (p.op == FfnOp::kUp && p.save == 16)) {  // at a pitch of both halves
    T* ug = reinterpret_cast<T*>(p.ug);
    ok = ok && map_out(&m->o2, p.dtype, ug, p.M, p.N, 2LL * p.N) &&
         map_out(&m->o3, p.dtype, ug + p.N, p.M, p.N, 2LL * p.N);
  }
  return ok;
}

void prepare(FfnGemm& p, const FfnProduct& f) {
  static_cast<FfnProduct&>(p) = f;
  p.tiles_m = (f.M + 255) / 256;
  p.ksteps = (f.K + 63) / 64;
}

template <class T>
cudaError_t one(const FfnProduct& f, int num_sms, cudaStream_t stream) {
  Launch<1> L = {};
  L.count = 1;
  prepare(L.p[0], f);
  cut_alone(L.p[0]);
  if (!maps_of<T>(L.p[0], &L.maps[0])) return cudaErrorInvalidValue;
  if (f.op == FfnOp::kUp) return run<T, Op::kUp, false>(L, num_sms, stream);
  return f.kept_scales ? run<T, Op::kDh, true>(L, num_sms, stream)
                       : run<T, Op::kDh, false>(L, num_sms, stream);
}

template <class T>
cudaError_t many(const FfnProduct* f, int count, int num_sms, cudaStream_t stream) {
  Launch<kMost> L = {};
  L.count = count;
  for (int j = 0; j < count; ++j) prepare(L.p[j], f[j]);
  if (count == 1)
    cut_alone(L.p[0]);
  else
    cut_together(L.p, count);
  for (int j = 0; j < count; ++j)
    if (!maps_of<T>(L.p[j], &L.maps[j])) return cudaErrorInvalidValue;
  return run<T, Op::kMany, false>(L, num_sms, stream);
}

}  // namespace

cudaError_t launch_ffn_product(const FfnProduct& f, int num_sms, cudaStream_t stream) {
  if (f.op != FfnOp::kUp && f.op != FfnOp::kDh) return launch_ffn_products(&f, 1, num_sms, stream);
  return f.dtype == QMOE_DTYPE_BF16 ? one<__nv_bfloat16>(f, num_sms, stream)
                                    : one<__half>(f, num_sms, stream);
}

cudaError_t launch_ffn_products(const FfnProduct* f, int count, int num_sms, cudaStream_t stream) {
  if (count < 1 || count > kMost) return cudaErrorInvalidValue;
  return f[0].dtype == QMOE_DTYPE_BF16 ? many<__nv_bfloat16>(f, count, num_sms, stream)
                                       : many<__half>(f, count, num_sms, stream);
}

}  // namespace qmoe
