// Host-side launchers shared between the translation units of libqmoe (internal).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace qmoe {

constexpr int kMaxDevices = 64;
// Positive numbers that are looked up once per device, N of them; atomics, since several host
// threads may make their first calls at the same time.
template <int N>
struct PerDevice {
  std::atomic<int> kept[kMaxDevices][N] = {};  // 0: not yet known
  // Number i of a device; look() gives it, or 0 or less if it cannot.
  template <class F>
  int get(int dev, int i, F&& look) {
    if (dev < 0 || dev >= kMaxDevices) return 0;
    int v = kept[dev][i].load(std::memory_order_relaxed);
    if (v == 0) {
      v = look();
      if (v < 1) return 0;
      kept[dev][i].store(v, std::memory_order_relaxed);
    }
    return v;
  }
};

// route.cu
constexpr int kRouteThreads = 512;
size_t route_smem_bytes(int E);
// scratch: route_scratch_bytes(P, E) bytes of device memory (none below 8193 pairs)
size_t route_scratch_bytes(long long P, int E);
// order (optional, needs small_rows < tile_n): the tile indices with the tiles of more
// than small_rows pairs first, then the others; n_tiles[1] = the count of the first part
// The route zeroes clear_words 32-bit words from err on (the error word and any counters
// the caller places after it) before it raises a bad-id bit there: no memset is needed.
// pdl: launch its kernels with programmatic stream serialization.
int route_blocks(long long P);
cudaError_t launch_route(const int32_t* ids, int P, int E, int tile_n, int32_t* offsets,
                         int32_t* sorted_pair, int32_t* pair_pos, int32_t* tiles, int32_t* n_tiles,
                         unsigned int* err, void* scratch, cudaStream_t stream,
                         int32_t* order = nullptr, int small_rows = 0, int clear_words = 1,
                         bool pdl = false);

// Route of moe_sort_tokens: as launch_route, without tiles; more than kSortSmallPairs pairs
// (fewer are placed by the kernel that copies their rows, launch_sort_small)
constexpr int kSortSmallPairs = 1024;
size_t sort_scratch_bytes(long long P, int E);
cudaError_t launch_sort_route(const int32_t* ids, int P, int E, int32_t* offsets,
                              int32_t* sorted_pair, int32_t* pair_pos, unsigned int* err,
                              void* scratch, cudaStream_t stream);

// api.cu
// SM count of the current device; QMOE_ERR_ARCH unless it runs sm_103a code
int device_info(int* num_sms);
// Tensor map of 16-bit elements (QMOE_DTYPE_BF16 or _FP16), 128- or 64-byte swizzle, zeros out of
// bounds; strides in bytes, of all dimensions but the innermost
int make_tmap16(CUtensorMap* map, int dtype, const void* base, int rank, const uint64_t* dims,
                const uint64_t* strides, const uint32_t* box, int swizzle = 128);

// misc.cu
// scale_layout: QMOE_SCALES_PLAIN, _SWIZZLED_128X4 or _PACKED_U32
cudaError_t launch_repack(const uint8_t* w, const uint8_t* s, int E, int N, int K, bool w13,
                          int scale_layout, uint8_t* out_codes, uint8_t* out_scales,
                          cudaStream_t stream);
// pdl: launch with programmatic stream serialization (see pdl_attribute)
// xs[pair_pos[i]] = x[i / top_k] for every routed pair i (pair_pos[i] >= 0)
cudaError_t launch_gather(const void* x, const int32_t* pair_pos, int M, int top_k, int H,
                          void* xs, int num_sms, cudaStream_t stream, bool pdl);
cudaError_t launch_combine(const float* ypart, const int32_t* ids, int M, int top_k, int E, int H,
                           void* out, int num_sms, cudaStream_t stream, bool pdl);
cudaError_t launch_selftest_dequant(uint16_t* out, cudaStream_t stream);
cudaError_t launch_selftest_timeout(unsigned int* err, long long limit_ns, cudaStream_t stream);

// gemm.cu
struct GemmParams {
  const uint8_t* wcodes;      // repacked codes
  const uint8_t* wscales;     // repacked scales
  const float* gscale;        // [E]
  const int32_t* tiles;       // [n_tiles][3]
  const int32_t* n_tiles;     // [1]
  int K;                      // contraction length
  int nrb;                    // 128-row weight blocks per expert
  // FC1 output: h [rows][I] bf16; the SwiGLU limit (+infinity: none)
  void* h;
  int I;
  float swiglu_limit;
  // FC2 output: ypart [pairs][H] fp32
  float* ypart;
  const int32_t* sorted_pair;
  const float* topk_w;
  int H;
  unsigned int* err;
  // decode schedule (stream-K): fp32 partial accumulators of units split between CTAs,
  // [CTA][2 slots][128 rows][16 pairs], and one arrival counter per (split unit, TMEM
  // lane quarter), [CTA holding the unit's first step][4], zero at launch
  float* sk_part;
  int* sk_cnt;
  uint32_t dq_mul[2];  // the dequant's multipliers 64, 4 (dequant_mul), as runtime values
  // which tiles the launch covers: 0 all, in tile order; with the split prefill
  // schedule's order (tile_order, n_tiles[1] = tiles of its first part) 1 the first
  // part (tiles of more than kSmallTileRows pairs), 2 the second
  const int32_t* tile_order;
  int tile_part;
};

// Largest grid of the decode schedule (its partial buffer has a slot pair per CTA).
constexpr int kMaxSkCtas = 192;
// Bytes of the decode schedule's partial buffer and of its counters for one GEMM.
inline size_t sk_part_bytes() { return (size_t)kMaxSkCtas * 2 * 128 * 16 * sizeof(float); }
inline size_t sk_cnt_bytes(int max_ctas) { return (size_t)max_ctas * 4 * sizeof(int); }

// Lets a kernel have up to `bytes` of dynamic shared memory.  Always the kernel's most, not the
// launch's own need: the limit belongs to the kernel in the whole process, and another thread
// must not find it lowered between its own call here and its launch.
template <class K>
cudaError_t allow_smem(K* kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
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

// A launch without attributes, whose own error is its answer: cudaGetLastError would hand over what an
// earlier call has left.
template <class... Params, class... Args>
cudaError_t launch_plain(void (*kernel)(Params...), int grid, int threads, cudaStream_t stream,
                         Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Launch attribute that lets a kernel start while the previous kernel on the stream
// finishes (it must then call grid_dep_wait before reading that kernel's outputs).
// The forward uses it on every schedule but the wide prefill one, where kernels that
// take SMs early (and start their weight streams) slowed the layer by about 2%:
// measured 4.63 against 4.54 ms on the large prefill workload, while decode (0.515
// against 0.526 ms) and the narrow prefill schedule gain from the overlap.
bool forward_uses_pdl(int sched);
inline cudaLaunchAttribute pdl_attribute() {
  cudaLaunchAttribute a;
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}

enum class GemmKind { kFc1, kFc2 };
cudaError_t launch_gemm(GemmKind kind, int sched, const CUtensorMap& tmap_b, const GemmParams& p,
                        int num_sms, cudaStream_t stream);
// Internal schedules.  kSchedPrefillNarrow: PREFILL when experts average fewer than 192
// pairs; the route cuts tiles of up to 192 pairs and orders them into two parts, and
// each GEMM runs as two launches: the tiles of more than kSmallTileRows pairs on the
// prefill kernel (two accumulators), the others on kSchedPrefillSmall, the decode
// kernel's weight-streaming pipeline with tiles of up to 64 pairs.
constexpr int kSchedPrefillNarrow = 16;
constexpr int kSchedPrefillSmall = 17;
constexpr int kSmallTileRows = 64;
int gemm_tile_n(int sched);  // max pairs per tile for a schedule
// Prefill GEMM on CTA pairs (two SMs per M = 256 tile, gemm2.cu); needs an even number
// of 128-row weight blocks (p.nrb).
cudaError_t launch_gemm2(GemmKind kind, const CUtensorMap& tmap_b, const GemmParams& p, int num_sms,
                         cudaStream_t stream);
// Rows and 64-wide slabs of the pair-row box the GEMM of a schedule loads: a 3-D box
// {64 elements, rows, slabs} per pipeline step, or (slabs 0) 2-D boxes of rows x 64
// elements.
int gemm_b_box_rows(int sched);
int gemm_b_box_slabs(int sched);

// gate.cu
struct GateArgs {
  const void* logits;  // [M][E], rows ld elements apart
  long long ld;
  int M, E, top_k;
  int scoring;  // QMOE_GATE_*
  const float* bias;
  int n_group, topk_group;
  int group_lanes;  // set at launch
  int renormalize;
  float scale;
  int32_t* ids;  // forward's outputs
  float* weights;
  const float* dweights;  // backward's inputs and output
  const int32_t* ids_in;
  void* dlogits;
};
cudaError_t launch_gate(const GateArgs& p, int dtype, int num_sms, cudaStream_t stream);
// vec: the output rows are 16-byte aligned and a multiple of 16 bytes long
cudaError_t launch_gate_backward(const GateArgs& p, int dtype, bool vec, int num_sms,
                                 cudaStream_t stream);

// tokens.cu
// xs[pair_pos[i]] = x[i / top_k] in chunks of chunk_bytes (16, 8, 4 or 2, dividing the rows,
// their stride and the pointers), zeros from row n_routed[0] on
cudaError_t launch_sort_copy(const void* x, long long ldx_bytes, const int32_t* pair_pos,
                             const int32_t* n_routed, int M, int top_k, long long row_bytes,
                             int chunk_bytes, void* xs, cudaStream_t stream);
// the same with the route in one launch, at most kSortSmallPairs pairs
cudaError_t launch_sort_small(const void* x, long long ldx_bytes, const int32_t* ids, int M,
                              int top_k, int E, long long row_bytes, int chunk_bytes, void* xs,
                              int32_t* offsets, int32_t* sorted_pair, int32_t* pair_pos,
                              unsigned int* err, cudaStream_t stream);
struct TokenArgs {
  const void* y;  // pair rows [M * top_k][H], rows ldy elements apart
  long long ldy;
  const void* dout;  // token rows [M][H], rows ldd elements apart (unsort backward)
  long long ldd;
  const int32_t* sorted_pair;
  const int32_t* pair_pos;
  const float* weights;  // NULL: all ones
  int M, H, top_k;
  void* out;
  float* dweights;
};
// chunk: elements that move together (1, 2, 4, or for 16-bit types 8), dividing every row,
// stride and pointer
cudaError_t launch_unsort(const TokenArgs& a, int dtype, int chunk, cudaStream_t stream);
cudaError_t launch_unsort_backward(const TokenArgs& a, int dtype, int chunk, int num_sms,
                                   cudaStream_t stream);

// lora.cu
// How a problem is cut: token tiles of tile_n (a multiple of 16, at most 256), units of one
// tile x 128 * cg rows of w (cg: CTAs per unit), each of ksteps steps of 64 of K; the shrink
// with plain products or on the tensor cores, in tsplits segments of K.
struct LoraPlan {
  int cg, tile_n, tiles, blocks, ksteps, tensor_shrink, tsplits;
};
constexpr int kLoraLeastTile = 128;  // tokens of a tile, of more than one; at most
constexpr int kLoraMostTile = 256;
LoraPlan lora_plan(int M, int K, int N, int R, bool has_w);
// The most M' * tsplits of any plan of M' <= M tokens.
size_t lora_segment_rows(int M, int K, int R);
struct LoraArgs : LoraPlan {
  int dtype;
  const void* x;  // [M][K], rows ldx elements apart
  long long ldx;
  const void* w;  // [N][K] or NULL
  const void* a;  // [L][R][K]
  const void* b;  // [L][N][R]
  const int32_t* ids;
  const float* scales;
  const void* base;  // [M][N], rows ldbase elements apart, or NULL
  long long ldbase;
  void* out;  // [M][N]
  int M, K, N, R, L;
  int wide;    // rows of out move in 16-byte chunks
  int stages, splits;  // of the GEMM's ring, of a unit's steps (set at launch)
  unsigned int* err;
  int* count;  // [tiles] distinct adapters of a tile
  int* bad;    // [tiles] whether an id of the tile is L or more
  int* list;   // [tiles][tile_n] the distinct adapters
  int* place;  // [tiles][tile_n] each token's adapter's place in the list, -1: none
  float* t;    // [tsplits][M][R] scales[a] * (x . A^T) over a segment of K
  // what of t the activation type does not hold, for the GEMM's epilogue (lora.cuh):
  unsigned int* left;      // [tiles][tile_n] a bit per eight ranks of a token
  unsigned int* any_left;  // [tiles] whether the tile has any
  float* tleft;            // [M][R] t of those ranks, over all segments
};
cudaError_t launch_lora(LoraArgs& p, int num_sms, cudaStream_t stream);
// its two steps (the second for more than eight tokens): lora_shrink.cu, lora_gemm.cu
cudaError_t launch_lora_shrink(const LoraArgs& p, int num_sms, cudaStream_t stream);
cudaError_t launch_lora_gemm(LoraArgs& p, int num_sms, cudaStream_t stream);

// norm.cu, norm_backward.cu
struct NormArgs {
  int M, H;
  int threads, units;  // of a row; rows of sums over the tokens (backward)
  // matrices a row is read from, rows on their way, vectors in shared memory (set at launch)
  int mats, depth, vectors;
  const void* y;       // [M][H], rows ldy elements apart (likewise the others)
  long long ldy;
  const void* residual;
  long long ldr;
  float residual_scale;
  const void* gate;
  int gate_form, gating, gate_fp32;
  long long ldgate;
  const void* post_weight;  // [H], NULL: no such norm
  const void* pre_weight;
  int weight_fp32;
  float weight_offset, eps;
  float* post_rstd;  // [M]
  float* pre_rstd;
  void* out;  // forward: outputs, NULL where not wanted
  void* normed;
  const void* dout;  // backward: gradients in, and what the forward pass left
  long long lddout;
  const void* dnormed;
  long long lddnormed;
  const void* out_in;
  long long ldout;
  void* dy;  // gradients out, NULL where not wanted
  void* dresidual;
  void* dgate;
  int dgate_fp32;  // of a full gate
  float* dpost_weight;
  float* dpre_weight;
  float* partial;  // [units][3][H]
};
constexpr int kNormRingBytes = 231424;       // of shared memory for rows and vectors, at most
constexpr int kNormRegisterColumns = 8192;  // whose sums over the tokens stay in registers
// chunk: elements that move together (1, 2, 4, or for 16-bit types 8), dividing every row, stride
// and pointer
cudaError_t launch_norm(const NormArgs& a, int dtype, int chunk, int sms, cudaStream_t stream);
// Rows of sums that M tokens leave.
int norm_units(int M, int H);
cudaError_t launch_norm_backward(const NormArgs& a, int dtype, int chunk, cudaStream_t stream);

// checkpoint.cu
struct CheckpointArgs {
  const void* x;  // [M][C], rows ldx elements apart
  long long ldx;
  int M, C, blocks;  // of 32 columns, of a row
  int8_t* codes;     // [M][C]
  uint8_t* scales;   // [M][blocks]
  void* out;         // [M][C]
};
// x to codes and scales, or (restore) those to out
cudaError_t launch_checkpoint(const CheckpointArgs& a, int dtype, int chunk, bool restore, int sms,
                              cudaStream_t stream);

// ffn_gemm.cu: one product of the gated feed-forward block, D [M][N] over K
enum class FfnOp {
  kUp,  // a [M][K], b = w13 [2N][K] -> out = h [M][N]
  kDh,  // a [M][K], b = w2 [K][N], kept u and g -> out = h [M][N], ug = [du | dg] [M][2N]
  kNT,  // a [M][K], b [N][K]
  kNN,  // a [M][K], b [K][N]
  kTN   // a [K][M], b [K][N]
};
struct FfnProduct {
  FfnOp op;
  int dtype;
  const void* a;
  long long lda;
  const void* b;
  long long ldb;
  int M, N, K;
  void* out;
  int save;         // kUp: keep u and g in ug (16) or codes and scales (8)
  void* ug;         // [M][2N]
  int8_t* codes;    // [M][2N]
  uint8_t* scales;  // [M][2][blocks of 32 of N]
  const void* kept;  // kDh: what kUp kept, codes where there are scales
  const uint8_t* kept_scales;
  int activation;
  float limit;
  unsigned int* err;
  int clear_err;  // the first product of a call
  float* part;    // ffn_part_bytes
};
struct FfnGemm : FfnProduct {
  int tile_n, tiles_m, tiles_n, ksteps;
  int splits;  // segments of K
  int first;   // of its launch's units
};
// Bytes of the sums of segments of a product with `rows` x `columns` of them, or fewer rows: as
// many tiles as there are pairs of SMs are the most, and as many segments.
constexpr int kFfnMaxSplits = 16;
inline size_t ffn_part_bytes(long long rows, long long columns) {
  const long long most = 76LL * 256 * 256 * 4, all = kFfnMaxSplits * rows * columns * 4;
  return (size_t)(all < most ? all : most);
}
// ffn_finish.cu: the segments' sums added up, and what a tile's epilogue does
cudaError_t launch_ffn_finish(const FfnGemm& p, cudaStream_t stream);
cudaError_t launch_ffn_product(const FfnProduct& f, int num_sms, cudaStream_t stream);
// ... and up to three plain ones of one type in one launch, the longest K first
cudaError_t launch_ffn_products(const FfnProduct* f, int count, int num_sms, cudaStream_t stream);
// ffn_stream.cu, ffn_few.cu: kUp (nothing kept) and kNT for few tokens, which are the columns of an
// MMA whose rows are the weights'
constexpr int kFfnStreamTokens = 8;
cudaError_t launch_ffn_stream(const FfnProduct& f, cudaStream_t stream);
struct FfnFew : FfnProduct {
  int tile_n;  // tokens, in whole MMA columns
  int ksteps, splits, stages, ring_bytes, tmem_cols;
};
// As many as an MMA has columns: up to there one pass over the weights is not slower than tiles of
// 256 tokens are.  us a call in a graph of 9, 128, 144, 192 and 256 tokens by ffn_few.cu, and
// (behind it) by ffn_gemm.cu:
//   4096 x 1536: 13.3 (23.0), 19.3 (25.4), 19.3 (25.4), 21.1 (25.6), 24.9 (25.9)
//   7168 x 2048: 20.6 (30.6), 28.4 (37.5), 26.7 (37.6), 29.6 (38.3), 34.9 (39.6)
//   2048 x 1024: 8.9 (16.5), 14.2 (19.7), 14.6 (19.7), 16.1 (19.8), 19.4 (19.5)
constexpr int kFfnFewTokens = 256;
cudaError_t launch_ffn_few(const FfnProduct& f, int num_sms, cudaStream_t stream);

}  // namespace qmoe
