// C-ABI boundary of a block's dense side (norms with gate and residual, gated feed-forward block,
// activation checkpoints): argument checks, workspace layout and launches.
#include <math.h>

#include <utility>

#include "common.cuh"
#include "launch.h"
#include "rows.h"

using namespace qmoe;

namespace {

constexpr int kMostColumns = 65536;
bool some_rows(int M) { return M >= 0 && M < (1 << 27); }

// Alignment at which `chunk` elements of `es` bytes of a vector in memory are read.
int vector_bytes(int chunk, int es) { return chunk * es < 16 ? chunk * es : 16; }

struct Gate {
  const void* p;
  int dtype, form;
  long long ld;
  int gating;
};

int check_norm(int dtype, int M, int H, const Gate& g, const void* post, const void* pre,
               int weight_dtype, float scale, float offset) {
  if (!known_dtype(dtype)) return QMOE_ERR_ARG;
  if (!some_rows(M) || H < 1 || H > kMostColumns) return QMOE_ERR_SHAPE;
  if (!isfinite(scale) || !isfinite(offset)) return QMOE_ERR_ARG;
  if ((post || pre) && weight_dtype != dtype && weight_dtype != QMOE_DTYPE_FP32)
    return QMOE_ERR_ARG;
  if (g.p) {
    if (g.dtype != dtype && g.dtype != QMOE_DTYPE_FP32) return QMOE_ERR_ARG;
    if (g.form < QMOE_GATE_TOKEN || g.form > QMOE_GATE_FULL) return QMOE_ERR_ARG;
    if (g.gating != QMOE_GATING_LINEAR && g.gating != QMOE_GATING_SIGMOID) return QMOE_ERR_ARG;
    if (g.form == QMOE_GATE_TOKEN && g.ld < 0) return QMOE_ERR_SHAPE;
    if (g.form == QMOE_GATE_FULL && bad_ld(g.ld, H)) return QMOE_ERR_SHAPE;
    if (misaligned(g.p, elem_size(g.dtype))) return QMOE_ERR_ARG;
  }
  const int ws = elem_size(weight_dtype);
  if (misaligned(post, ws) || misaligned(pre, ws)) return QMOE_ERR_ARG;
  return QMOE_OK;
}

// What the forward and backward kernels are both given.
NormArgs norm_args(int M, int H, const void* y, long long ldy, float residual_scale, const Gate& g,
                   const void* post, const void* pre, int weight_dtype, float weight_offset,
                   float* post_rstd, float* pre_rstd) {
  NormArgs a = {};
  a.M = M;
  a.H = H;
  a.y = y;
  a.ldy = ldy;
  a.residual_scale = residual_scale;
  a.gate = g.p;
  a.gate_form = g.form;
  a.gating = g.gating;
  a.gate_fp32 = g.dtype == QMOE_DTYPE_FP32;
  a.ldgate = g.ld;
  a.post_weight = post;
  a.pre_weight = pre;
  a.weight_fp32 = weight_dtype == QMOE_DTYPE_FP32;
  a.weight_offset = weight_offset;
  a.post_rstd = post_rstd;
  a.pre_rstd = pre_rstd;
  return a;
}

// The widest chunk of elements in which a norm's rows and vectors move.
int norm_chunk(int dtype, int H, const Gate& g, const void* post, const void* pre, int weight_dtype,
               Chunk chunk) {
  const int es = elem_size(dtype);
  if (g.p && g.form == QMOE_GATE_FULL) chunk.rows(g.p, g.dtype == dtype ? g.ld : H, H, es);
  int n = chunk.bytes / es;
  auto fits = [&](const void* p, int size, long long ld) {
    while (p && n > 1 && (misaligned(p, vector_bytes(n, size)) ||
                          ld * size % vector_bytes(n, size) != 0 || H % n != 0))
      n >>= 1;
  };
  fits(post, elem_size(weight_dtype), 0);
  fits(pre, elem_size(weight_dtype), 0);
  if (g.p && g.form != QMOE_GATE_TOKEN)
    fits(g.p, elem_size(g.dtype), g.form == QMOE_GATE_FULL ? g.ld : 0);
  return n;
}

}  // namespace

extern "C" {

int qmoe_block_norm(const void* y_dev, int dtype, long long ldy, const void* residual_dev,
                    long long ldr, float residual_scale, const void* gate_dev, int gate_dtype,
                    int gate_form, long long ldgate, int gating, const void* post_weight_dev,
                    const void* pre_weight_dev, int weight_dtype, float weight_offset, float eps,
                    int M, int H, void* out_dev, void* normed_dev, float* post_rstd_dev,
                    float* pre_rstd_dev, void* stream) {
  const Gate g = {gate_dev, gate_dtype, gate_form, ldgate, gating};
  int rc = check_norm(dtype, M, H, g, post_weight_dev, pre_weight_dev, weight_dtype, residual_scale,
                      weight_offset);
  if (rc != QMOE_OK) return rc;
  if (!(eps >= 0.f) || !isfinite(eps)) return QMOE_ERR_ARG;
  if (bad_ld(ldy, H) || (residual_dev && bad_ld(ldr, H))) return QMOE_ERR_SHAPE;
  if ((pre_weight_dev == nullptr) != (normed_dev == nullptr) && M > 0) return QMOE_ERR_ARG;
  if (M == 0) return QMOE_OK;
  const int es = elem_size(dtype);
  if (!y_dev || (!out_dev && !normed_dev)) return QMOE_ERR_ARG;
  if (misaligned(y_dev, es) || misaligned(residual_dev, es) || misaligned(out_dev, es) ||
      misaligned(normed_dev, es) || misaligned(post_rstd_dev, 4) || misaligned(pre_rstd_dev, 4))
    return QMOE_ERR_ARG;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != QMOE_OK) return rc;
  NormArgs a = norm_args(M, H, y_dev, ldy, residual_scale, g, post_weight_dev, pre_weight_dev,
                         weight_dtype, weight_offset, post_rstd_dev, pre_rstd_dev);
  a.residual = residual_dev;
  a.ldr = ldr;
  a.eps = eps;
  a.out = out_dev;
  a.normed = normed_dev;
  Chunk chunk;
  chunk.rows(y_dev, ldy, H, es);
  if (residual_dev) chunk.rows(residual_dev, ldr, H, es);
  if (out_dev) chunk.rows(out_dev, H, H, es);
  if (normed_dev) chunk.rows(normed_dev, H, H, es);
  return cuda_rc(launch_norm(
      a, dtype, norm_chunk(dtype, H, g, post_weight_dev, pre_weight_dev, weight_dtype, chunk), sms,
      reinterpret_cast<cudaStream_t>(stream)));
}

size_t qmoe_block_norm_backward_workspace_size(int M, int H) {
  if (!some_rows(M) || H < 1 || H > kMostColumns) return 0;
  return kWsHeaderBytes + 3 * sizeof(float) * (size_t)norm_units(M, H) * H;
}

int qmoe_block_norm_backward(const void* dout_dev, long long lddout, const void* dnormed_dev,
                             long long lddnormed, const void* y_dev, int dtype, long long ldy,
                             const void* out_dev, long long ldout, float residual_scale,
                             const void* gate_dev, int gate_dtype, int gate_form, long long ldgate,
                             int gating, const void* post_weight_dev, const void* pre_weight_dev,
                             int weight_dtype, float weight_offset, const float* post_rstd_dev,
                             const float* pre_rstd_dev, int M, int H, void* dy_dev,
                             void* dresidual_dev, void* dgate_dev, float* dpost_weight_dev,
                             float* dpre_weight_dev, void* workspace_dev, size_t ws_bytes,
                             void* stream) {
  int dgate_dtype = dtype;  // of a full gate's
  if (gate_form == QMOE_GATE_FULL + QMOE_GATE_OWN_GRADIENT) {
    gate_form = QMOE_GATE_FULL;
    dgate_dtype = gate_dtype;
  }
  const Gate g = {gate_dev, gate_dtype, gate_form, ldgate, gating};
  int rc = check_norm(dtype, M, H, g, post_weight_dev, pre_weight_dev, weight_dtype, residual_scale,
                      weight_offset);
  if (rc != QMOE_OK) return rc;
  if (bad_ld(ldy, H) || (dout_dev && bad_ld(lddout, H)) ||
      (dnormed_dev && bad_ld(lddnormed, H)) || (out_dev && bad_ld(ldout, H)))
    return QMOE_ERR_SHAPE;
  if (dgate_dev && !gate_dev) return QMOE_ERR_ARG;
  if ((dpost_weight_dev && !post_weight_dev) || (dpre_weight_dev && !pre_weight_dev))
    return QMOE_ERR_ARG;
  if (misaligned(dpost_weight_dev, 4) || misaligned(dpre_weight_dev, 4)) return QMOE_ERR_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) {  // sums over no tokens
    int sms = 0;
    float* sums[3] = {dpost_weight_dev, dpre_weight_dev,
                      gate_form == QMOE_GATE_CHANNEL ? reinterpret_cast<float*>(dgate_dev) : nullptr};
    for (float* p : sums) {
      if (!p) continue;
      rc = device_info(&sms);
      if (rc != QMOE_OK) return rc;
      if (cudaMemsetAsync(p, 0, sizeof(float) * H, s) != cudaSuccess) return QMOE_ERR_CUDA;
    }
    return QMOE_OK;
  }
  const int es = elem_size(dtype);
  if (!y_dev || !dy_dev || !workspace_dev || (pre_weight_dev == nullptr) != (dnormed_dev == nullptr) ||
      (!dout_dev && !dnormed_dev))
    return QMOE_ERR_ARG;
  if ((post_weight_dev && !post_rstd_dev) || (pre_weight_dev && !pre_rstd_dev)) return QMOE_ERR_ARG;
  // without what the norm was taken of, that is y itself
  if (pre_weight_dev && !out_dev && (post_weight_dev || gate_dev || dresidual_dev))
    return QMOE_ERR_ARG;
  if (misaligned(dout_dev, es) || misaligned(dnormed_dev, es) || misaligned(y_dev, es) ||
      misaligned(out_dev, es) || misaligned(dy_dev, es) || misaligned(dresidual_dev, es) ||
      misaligned(dgate_dev, gate_form == QMOE_GATE_FULL ? elem_size(dgate_dtype) : 4) ||
      misaligned(post_rstd_dev, 4) ||
      misaligned(pre_rstd_dev, 4) || misaligned(workspace_dev, 256))
    return QMOE_ERR_ARG;
  if (ws_bytes < qmoe_block_norm_backward_workspace_size(M, H)) return QMOE_ERR_WORKSPACE;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != QMOE_OK) return rc;
  NormArgs a = norm_args(M, H, y_dev, ldy, residual_scale, g, post_weight_dev, pre_weight_dev,
                         weight_dtype, weight_offset, const_cast<float*>(post_rstd_dev),
                         const_cast<float*>(pre_rstd_dev));
  a.units = norm_units(M, H);
  a.dout = dout_dev;
  a.lddout = lddout;
  a.dnormed = dnormed_dev;
  a.lddnormed = lddnormed;
  a.out_in = out_dev;
  a.ldout = ldout;
  a.dy = dy_dev;
  a.dresidual = dresidual_dev;
  a.dgate = dgate_dev;
  a.dgate_fp32 = dgate_dtype == QMOE_DTYPE_FP32;
  a.dpost_weight = dpost_weight_dev;
  a.dpre_weight = dpre_weight_dev;
  a.partial = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(workspace_dev) + kWsHeaderBytes);
  Chunk chunk;
  chunk.rows(y_dev, ldy, H, es);
  if (dout_dev) chunk.rows(dout_dev, lddout, H, es);
  if (dnormed_dev) chunk.rows(dnormed_dev, lddnormed, H, es);
  if (out_dev) chunk.rows(out_dev, ldout, H, es);
  chunk.rows(dy_dev, H, H, es);
  if (dresidual_dev) chunk.rows(dresidual_dev, H, H, es);
  const bool dgate_rows = dgate_dev && gate_form == QMOE_GATE_FULL;
  if (dgate_rows && dgate_dtype == dtype) chunk.rows(dgate_dev, H, H, es);
  int n = norm_chunk(dtype, H, g, post_weight_dev, pre_weight_dev, weight_dtype, chunk);
  if (dgate_rows)  // (n divides H)
    while (n > 1 && misaligned(dgate_dev, vector_bytes(n, elem_size(dgate_dtype)))) n >>= 1;
  return cuda_rc(launch_norm_backward(a, dtype, n, s));
}

static int check_checkpoint(int dtype, int M, int C) {
  if (!known_dtype(dtype)) return QMOE_ERR_ARG;
  if (!some_rows(M) || C < 1 || C > (1 << 20)) return QMOE_ERR_SHAPE;
  return QMOE_OK;
}

int qmoe_checkpoint8(const void* x_dev, int dtype, long long ldx, int M, int C, int8_t* codes_dev,
                     uint8_t* scales_dev, void* stream) {
  int rc = check_checkpoint(dtype, M, C);
  if (rc != QMOE_OK) return rc;
  if (bad_ld(ldx, C)) return QMOE_ERR_SHAPE;
  if (M == 0) return QMOE_OK;
  const int es = elem_size(dtype);
  if (!x_dev || !codes_dev || !scales_dev || misaligned(x_dev, es)) return QMOE_ERR_ARG;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != QMOE_OK) return rc;
  CheckpointArgs a = {};
  a.x = x_dev;
  a.ldx = ldx;
  a.M = M;
  a.C = C;
  a.blocks = (C + 31) / 32;
  a.codes = codes_dev;
  a.scales = scales_dev;
  Chunk chunk;
  chunk.rows(x_dev, ldx, C, es);
  int n = chunk.bytes / es;
  while (n > 1 && (misaligned(codes_dev, n) || C % n != 0)) n >>= 1;
  return cuda_rc(launch_checkpoint(a, dtype, n, false, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int qmoe_checkpoint8_restore(const int8_t* codes_dev, const uint8_t* scales_dev, int dtype, int M,
                             int C, void* out_dev, void* stream) {
  int rc = check_checkpoint(dtype, M, C);
  if (rc != QMOE_OK) return rc;
  if (M == 0) return QMOE_OK;
  const int es = elem_size(dtype);
  if (!codes_dev || !scales_dev || !out_dev || misaligned(out_dev, es)) return QMOE_ERR_ARG;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != QMOE_OK) return rc;
  CheckpointArgs a = {};
  a.M = M;
  a.C = C;
  a.blocks = (C + 31) / 32;
  a.codes = const_cast<int8_t*>(codes_dev);
  a.scales = const_cast<uint8_t*>(scales_dev);
  a.out = out_dev;
  Chunk chunk;
  chunk.rows(out_dev, C, C, es);
  int n = chunk.bytes / es;
  while (n > 1 && (misaligned(codes_dev, n) || C % n != 0)) n >>= 1;
  return cuda_rc(launch_checkpoint(a, dtype, n, true, sms, reinterpret_cast<cudaStream_t>(stream)));
}

static int check_ffn(int dtype, int M, int H, int I, int activation, float limit) {
  if (dtype != QMOE_DTYPE_BF16 && dtype != QMOE_DTYPE_FP16) return QMOE_ERR_ARG;
  if (activation != QMOE_ACT_SILU && activation != QMOE_ACT_GELU) return QMOE_ERR_ARG;
  if (!(limit > 0.f)) return QMOE_ERR_ARG;
  if (!some_rows(M) || H < 8 || I < 8 || H % 8 || I % 8 || H > kMostColumns || I > kMostColumns)
    return QMOE_ERR_SHAPE;
  return QMOE_OK;
}

static bool ffn_shape(int M, int H, int I) {
  return check_ffn(QMOE_DTYPE_BF16, M, H, I, QMOE_ACT_SILU, 1.f) == QMOE_OK;
}

// Workspaces: the error word's block, the rows between the products, the sums of segments; each as
// large as any batch of up to M tokens needs.
static size_t ffn_forward_part(int M, int I) {
  return kWsHeaderBytes + align_up((size_t)M * I * 2, 256);
}

size_t qmoe_gated_ffn_workspace_size(int M, int H, int I) {
  if (!ffn_shape(M, H, I)) return 0;
  const size_t up = ffn_part_bytes(M, 2LL * I), down = ffn_part_bytes(M, H);
  return ffn_forward_part(M, I) + align_up(up > down ? up : down, 256);
}

int qmoe_gated_ffn(const void* x_dev, int dtype, long long ldx, const void* w13_dev,
                   const void* w2_dev, int activation, float limit, int M, int H, int I,
                   void* out_dev, void* kept_dev, uint8_t* kept_scales_dev, void* workspace_dev,
                   size_t ws_bytes, void* stream) {
  return qmoe_gated_ffn_error_at(x_dev, dtype, ldx, w13_dev, w2_dev, activation, limit, M, H, I,
                                 out_dev, kept_dev, kept_scales_dev, workspace_dev, ws_bytes,
                                 reinterpret_cast<uint32_t*>(workspace_dev), stream);
}

int qmoe_gated_ffn_error_at(const void* x_dev, int dtype, long long ldx, const void* w13_dev,
                            const void* w2_dev, int activation, float limit, int M, int H, int I,
                            void* out_dev, void* kept_dev, uint8_t* kept_scales_dev,
                            void* workspace_dev, size_t ws_bytes, uint32_t* error_dev,
                            void* stream) {
  int rc = check_ffn(dtype, M, H, I, activation, limit);
  if (rc != QMOE_OK) return rc;
  if (ldx < H || ldx % 8) return QMOE_ERR_SHAPE;
  if (kept_scales_dev && !kept_dev) return QMOE_ERR_ARG;
  if (M == 0) return QMOE_OK;
  if (!x_dev || !w13_dev || !w2_dev || !out_dev || !workspace_dev || !error_dev ||
      misaligned(error_dev, 4))
    return QMOE_ERR_ARG;
  if (misaligned(x_dev, 16) || misaligned(w13_dev, 16) || misaligned(w2_dev, 16) ||
      misaligned(out_dev, 16) || misaligned(kept_dev, 16) || misaligned(workspace_dev, 256))
    return QMOE_ERR_ARG;
  if (ws_bytes < qmoe_gated_ffn_workspace_size(M, H, I)) return QMOE_ERR_WORKSPACE;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != QMOE_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace_dev);
  FfnProduct up = {};
  up.op = FfnOp::kUp;
  up.dtype = dtype;
  up.a = x_dev;
  up.lda = ldx;
  up.b = w13_dev;
  up.ldb = H;
  up.M = M;
  up.N = I;
  up.K = H;
  up.out = ws + kWsHeaderBytes;
  up.save = !kept_dev ? 0 : kept_scales_dev ? 8 : 16;
  up.ug = kept_dev;
  up.codes = reinterpret_cast<int8_t*>(kept_dev);
  up.scales = kept_scales_dev;
  up.activation = activation;
  up.limit = limit;
  up.err = error_dev;
  up.clear_err = 1;
  up.part = reinterpret_cast<float*>(ws + ffn_forward_part(M, I));
  auto launch = [&](const FfnProduct& f) {
    if (!kept_dev && M <= kFfnStreamTokens) return launch_ffn_stream(f, s);
    if (!kept_dev && M <= kFfnFewTokens) return launch_ffn_few(f, sms, s);
    return launch_ffn_product(f, sms, s);
  };
  cudaError_t e = launch(up);
  if (e != cudaSuccess) return QMOE_ERR_CUDA;
  FfnProduct down = {};
  down.op = FfnOp::kNT;
  down.dtype = dtype;
  down.a = up.out;
  down.lda = I;
  down.b = w2_dev;
  down.ldb = I;
  down.M = M;
  down.N = H;
  down.K = I;
  down.out = out_dev;
  down.err = up.err;
  down.part = up.part;
  return cuda_rc(launch(down));
}

// Workspace of the backward pass: [du | dg], h, x out of its codes, the sums of segments.
struct FfnBackwardLayout {
  size_t dug, h, x, part[3], total;
};
static FfnBackwardLayout ffn_backward_layout(int M, int H, int I, bool codes) {
  FfnBackwardLayout L;
  L.dug = kWsHeaderBytes;
  L.h = align_up(L.dug + (size_t)M * I * 4, 256);
  L.x = align_up(L.h + (size_t)M * I * 2, 256);
  L.part[0] = align_up(L.x + (codes ? (size_t)M * H * 2 : 0), 256);
  // of [du | dg] and h, then of any three of the others
  size_t most = 0;
  for (size_t b : {ffn_part_bytes(M, I), ffn_part_bytes(M, H), ffn_part_bytes(2LL * I, H)})
    most = b > most ? b : most;
  L.part[1] = align_up(L.part[0] + most, 256);
  L.part[2] = align_up(L.part[1] + most, 256);
  L.total = align_up(L.part[2] + most, 256);
  return L;
}

size_t qmoe_gated_ffn_backward_workspace_size(int M, int H, int I, int checkpoint) {
  if (!ffn_shape(M, H, I) || (checkpoint != 8 && checkpoint != 16)) return 0;
  return ffn_backward_layout(M, H, I, checkpoint == 8).total;
}

int qmoe_gated_ffn_backward(const void* dout_dev, int dtype, long long lddout, const void* x_dev,
                            long long ldx, const uint8_t* x_scales_dev, const void* w13_dev,
                            const void* w2_dev, const void* kept_dev,
                            const uint8_t* kept_scales_dev, int activation, float limit, int M,
                            int H, int I, void* dx_dev, void* dw13_dev, void* dw2_dev,
                            void* workspace_dev, size_t ws_bytes, void* stream) {
  return qmoe_gated_ffn_backward_error_at(
      dout_dev, dtype, lddout, x_dev, ldx, x_scales_dev, w13_dev, w2_dev, kept_dev, kept_scales_dev,
      activation, limit, M, H, I, dx_dev, dw13_dev, dw2_dev, workspace_dev, ws_bytes,
      reinterpret_cast<uint32_t*>(workspace_dev), stream);
}

int qmoe_gated_ffn_backward_error_at(const void* dout_dev, int dtype, long long lddout,
                                     const void* x_dev, long long ldx, const uint8_t* x_scales_dev,
                                     const void* w13_dev, const void* w2_dev, const void* kept_dev,
                                     const uint8_t* kept_scales_dev, int activation, float limit,
                                     int M, int H, int I, void* dx_dev, void* dw13_dev, void* dw2_dev,
                                     void* workspace_dev, size_t ws_bytes, uint32_t* error_dev,
                                     void* stream) {
  int rc = check_ffn(dtype, M, H, I, activation, limit);
  if (rc != QMOE_OK) return rc;
  if ((x_scales_dev == nullptr) != (kept_scales_dev == nullptr)) return QMOE_ERR_ARG;
  const bool codes = x_scales_dev != nullptr;
  if (lddout < H || lddout % 8 || (codes ? ldx != H : ldx < H || ldx % 8)) return QMOE_ERR_SHAPE;
  if (misaligned(dx_dev, 16) || misaligned(dw13_dev, 16) || misaligned(dw2_dev, 16))
    return QMOE_ERR_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int sms = 0;
  if (M == 0) {  // sums over no tokens
    void* sums[2] = {dw13_dev, dw2_dev};
    for (int i = 0; i < 2; ++i) {
      if (!sums[i]) continue;
      rc = device_info(&sms);
      if (rc != QMOE_OK) return rc;
      if (cudaMemsetAsync(sums[i], 0, (size_t)H * I * (i == 0 ? 4 : 2), s) != cudaSuccess)
        return QMOE_ERR_CUDA;
    }
    return QMOE_OK;
  }
  if (!dout_dev || !x_dev || !w13_dev || !w2_dev || !kept_dev || !workspace_dev || !error_dev ||
      misaligned(error_dev, 4))
    return QMOE_ERR_ARG;
  if (misaligned(dout_dev, 16) || misaligned(x_dev, codes ? 8 : 16) || misaligned(w13_dev, 16) ||
      misaligned(w2_dev, 16) || misaligned(kept_dev, 16) || misaligned(workspace_dev, 256))
    return QMOE_ERR_ARG;
  if (ws_bytes < qmoe_gated_ffn_backward_workspace_size(M, H, I, codes ? 8 : 16))
    return QMOE_ERR_WORKSPACE;
  if (!dx_dev && !dw13_dev && !dw2_dev) return QMOE_OK;
  rc = device_info(&sms);
  if (rc != QMOE_OK) return rc;
  const FfnBackwardLayout L = ffn_backward_layout(M, H, I, codes);
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace_dev);
  const void* x = x_dev;
  if (codes && dw13_dev) {
    rc = qmoe_checkpoint8_restore(reinterpret_cast<const int8_t*>(x_dev), x_scales_dev, dtype, M, H,
                                  ws + L.x, stream);
    if (rc != QMOE_OK) return rc;
    x = ws + L.x;
  }
  FfnProduct f = {};
  f.dtype = dtype;
  f.err = error_dev;
  f.activation = activation;
  f.limit = limit;
  int parts = 0;
  auto product = [&](FfnOp op, const void* a, long long lda, const void* b, long long ldb, int m,
                     int n, int k, void* out) {
    FfnProduct g = f;
    g.op = op;
    g.a = a;
    g.lda = lda;
    g.b = b;
    g.ldb = ldb;
    g.M = m;
    g.N = n;
    g.K = k;
    g.out = out;
    g.part = reinterpret_cast<float*>(ws + L.part[parts++]);
    return g;
  };
  FfnProduct dh = product(FfnOp::kDh, dout_dev, lddout, w2_dev, I, M, I, H, ws + L.h);
  parts = 0;  // (its segments' sums have been used when the others' are written)
  dh.ug = ws + L.dug;
  dh.kept = kept_dev;
  dh.kept_scales = kept_scales_dev;
  dh.clear_err = 1;
  const cudaError_t e = launch_ffn_product(dh, sms, s);
  if (e != cudaSuccess) return QMOE_ERR_CUDA;
  FfnProduct rest[3];
  int n = 0;
  if (dx_dev) rest[n++] = product(FfnOp::kNN, ws + L.dug, 2LL * I, w13_dev, H, M, H, 2 * I, dx_dev);
  if (dw13_dev)
    rest[n++] = product(FfnOp::kTN, ws + L.dug, 2LL * I, x, codes ? H : ldx, 2 * I, H, M, dw13_dev);
  if (dw2_dev) rest[n++] = product(FfnOp::kTN, dout_dev, lddout, ws + L.h, I, H, I, M, dw2_dev);
  // the longest K first, so that the launch ends with short tiles
  for (int i = 1; i < n; ++i)
    for (int j = i; j > 0 && rest[j].K > rest[j - 1].K; --j) std::swap(rest[j], rest[j - 1]);
  return cuda_rc(launch_ffn_products(rest, n, sms, s));
}

}  // extern "C"
