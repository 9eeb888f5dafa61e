// C-ABI boundary of the operators around the layer (gate, token sort and its inverse,
// projection with adapters): argument checks, workspace layout and launches.
#include <math.h>

#include "common.cuh"
#include "launch.h"
#include "rows.h"

namespace qmoe {
namespace {

int check_tokens(int dtype, int M, int H, int top_k) {
  if (!known_dtype(dtype)) return QMOE_ERR_ARG;
  if (M < 0 || H < 1 || H > (1 << 20) || top_k < 1 || top_k > 64) return QMOE_ERR_SHAPE;
  if ((long long)M * top_k >= (1LL << 31) / 16) return QMOE_ERR_SHAPE;
  return QMOE_OK;
}

}  // namespace
}  // namespace qmoe

using namespace qmoe;

extern "C" {

static int check_gate(int dtype, long long ld, int M, int E, int top_k, int scoring, float scale) {
  if (!known_dtype(dtype)) return QMOE_ERR_ARG;
  if (scoring != QMOE_GATE_SOFTMAX && scoring != QMOE_GATE_SIGMOID) return QMOE_ERR_ARG;
  if (!isfinite(scale)) return QMOE_ERR_ARG;
  if (E < 1 || E > 2048 || top_k > E || bad_ld(ld, E)) return QMOE_ERR_SHAPE;
  return check_tokens(dtype, M, E, top_k);
}

int moe_gate(const void* logits_dev, int dtype, long long ld, int M, int E, int top_k, int scoring,
             const float* bias_dev, int n_group, int topk_group, int renormalize, float scale,
             int32_t* topk_ids_dev, float* topk_weights_dev, void* stream) {
  int rc = check_gate(dtype, ld, M, E, top_k, scoring, scale);
  if (rc != QMOE_OK) return rc;
  if (n_group < 1 || n_group > 32 || E % n_group || topk_group < 1 || topk_group > n_group ||
      top_k > E / n_group * topk_group)
    return QMOE_ERR_SHAPE;
  if (bias_dev && scoring != QMOE_GATE_SIGMOID) return QMOE_ERR_ARG;
  if (M == 0) return QMOE_OK;
  if (!logits_dev || !topk_ids_dev || !topk_weights_dev) return QMOE_ERR_ARG;
  if (misaligned(logits_dev, elem_size(dtype)) || misaligned(bias_dev, 4) ||
      misaligned(topk_ids_dev, 4) || misaligned(topk_weights_dev, 4))
    return QMOE_ERR_ARG;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != QMOE_OK) return rc;
  GateArgs p = {};
  p.logits = logits_dev;
  p.ld = ld;
  p.M = M;
  p.E = E;
  p.top_k = top_k;
  p.scoring = scoring;
  p.bias = bias_dev;
  p.n_group = n_group;
  p.topk_group = topk_group;
  p.renormalize = renormalize != 0;
  p.scale = scale;
  p.ids = topk_ids_dev;
  p.weights = topk_weights_dev;
  return cuda_rc(launch_gate(p, dtype, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int moe_gate_backward(const float* dweights_dev, const void* logits_dev, int dtype, long long ld,
                      const int32_t* topk_ids_dev, int M, int E, int top_k, int scoring,
                      int renormalize, float scale, void* dlogits_dev, void* stream) {
  int rc = check_gate(dtype, ld, M, E, top_k, scoring, scale);
  if (rc != QMOE_OK) return rc;
  if (M == 0) return QMOE_OK;
  if (!dweights_dev || !logits_dev || !topk_ids_dev || !dlogits_dev) return QMOE_ERR_ARG;
  const int es = elem_size(dtype);
  if (misaligned(logits_dev, es) || misaligned(dlogits_dev, es) || misaligned(topk_ids_dev, 4) ||
      misaligned(dweights_dev, 4))
    return QMOE_ERR_ARG;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != QMOE_OK) return rc;
  GateArgs p = {};
  p.logits = logits_dev;
  p.ld = ld;
  p.M = M;
  p.E = E;
  p.top_k = top_k;
  p.scoring = scoring;
  p.renormalize = renormalize != 0;
  p.scale = scale;
  p.dweights = dweights_dev;
  p.ids_in = topk_ids_dev;
  p.dlogits = dlogits_dev;
  return cuda_rc(launch_gate_backward(p, dtype, chunked(dlogits_dev, E, E, es, 16), sms,
                                      reinterpret_cast<cudaStream_t>(stream)));
}

size_t qmoe_sort_workspace_size(int M, int top_k, int E) {
  if (M < 0 || top_k < 1 || top_k > 64 || E < 1 || E > 2048) return 0;
  if ((long long)M * top_k >= (1LL << 31) / 16) return 0;
  return kWsHeaderBytes + sort_scratch_bytes((long long)M * top_k, E);
}

int moe_sort_tokens(const void* x_dev, int dtype, long long ldx, const int32_t* topk_ids_dev, int M,
                    int H, int top_k, int E, void* xs_dev, int32_t* offsets_dev,
                    int32_t* sorted_pair_dev, int32_t* pair_pos_dev, void* workspace_dev,
                    size_t ws_bytes, void* stream) {
  int rc = check_tokens(dtype, M, H, top_k);
  if (rc != QMOE_OK) return rc;
  if (E < 1 || E > 2048 || bad_ld(ldx, H)) return QMOE_ERR_SHAPE;
  if (M == 0) return QMOE_OK;
  if (!x_dev || !topk_ids_dev || !xs_dev || !offsets_dev || !sorted_pair_dev || !pair_pos_dev ||
      !workspace_dev)
    return QMOE_ERR_ARG;
  const int es = elem_size(dtype);
  if (misaligned(workspace_dev, 256) || misaligned(x_dev, es) || misaligned(xs_dev, es) ||
      misaligned(topk_ids_dev, 4) || misaligned(offsets_dev, 4) || misaligned(sorted_pair_dev, 4) ||
      misaligned(pair_pos_dev, 4))
    return QMOE_ERR_ARG;
  if (ws_bytes < qmoe_sort_workspace_size(M, top_k, E)) return QMOE_ERR_WORKSPACE;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != QMOE_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  unsigned int* err = reinterpret_cast<unsigned int*>(workspace_dev);
  const int P = M * top_k;
  Chunk chunk;
  chunk.rows(x_dev, ldx, H, es);
  chunk.rows(xs_dev, H, H, es);
  if (P <= kSortSmallPairs)
    return cuda_rc(launch_sort_small(x_dev, ldx * es, topk_ids_dev, M, top_k, E, (long long)H * es,
                                     chunk.bytes, xs_dev, offsets_dev, sorted_pair_dev,
                                     pair_pos_dev, err, s));
  cudaError_t e = launch_sort_route(topk_ids_dev, P, E, offsets_dev, sorted_pair_dev, pair_pos_dev,
                                    err, reinterpret_cast<uint8_t*>(workspace_dev) + kWsHeaderBytes,
                                    s);
  if (e != cudaSuccess) return QMOE_ERR_CUDA;
  return cuda_rc(launch_sort_copy(x_dev, ldx * es, pair_pos_dev, offsets_dev + E, M, top_k,
                                  (long long)H * es, chunk.bytes, xs_dev, s));
}

static int unsort_call(const void* y_dev, int dtype, long long ldy, const int32_t* pair_pos_dev,
                       const float* weights_dev, int M, int H, int top_k, void* out_dev,
                       void* stream) {
  int rc = check_tokens(dtype, M, H, top_k);
  if (rc != QMOE_OK) return rc;
  if (bad_ld(ldy, H)) return QMOE_ERR_SHAPE;
  if (M == 0) return QMOE_OK;
  if (!y_dev || !pair_pos_dev || !out_dev) return QMOE_ERR_ARG;
  const int es = elem_size(dtype);
  if (misaligned(y_dev, es) || misaligned(out_dev, es) || misaligned(pair_pos_dev, 4) ||
      misaligned(weights_dev, 4))
    return QMOE_ERR_ARG;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != QMOE_OK) return rc;
  TokenArgs a = {};
  a.y = y_dev;
  a.ldy = ldy;
  a.pair_pos = pair_pos_dev;
  a.weights = weights_dev;
  a.M = M;
  a.H = H;
  a.top_k = top_k;
  a.out = out_dev;
  Chunk chunk;
  chunk.rows(y_dev, ldy, H, es);
  chunk.rows(out_dev, H, H, es);
  return cuda_rc(launch_unsort(a, dtype, chunk.bytes / es, reinterpret_cast<cudaStream_t>(stream)));
}

int moe_sort_tokens_backward(const void* dxs_dev, int dtype, long long ld,
                             const int32_t* pair_pos_dev, int M, int H, int top_k, void* dx_dev,
                             void* stream) {
  return unsort_call(dxs_dev, dtype, ld, pair_pos_dev, nullptr, M, H, top_k, dx_dev, stream);
}

int moe_unsort_tokens(const void* y_dev, int dtype, long long ldy, const int32_t* pair_pos_dev,
                      const float* topk_weights_dev, int M, int H, int top_k, void* out_dev,
                      void* stream) {
  if (M > 0 && !topk_weights_dev) return QMOE_ERR_ARG;
  return unsort_call(y_dev, dtype, ldy, pair_pos_dev, topk_weights_dev, M, H, top_k, out_dev,
                     stream);
}

int moe_unsort_tokens_backward(const void* dout_dev, long long ldd, const void* y_dev,
                               long long ldy, int dtype, const int32_t* sorted_pair_dev,
                               const int32_t* pair_pos_dev, const float* topk_weights_dev, int M,
                               int H, int top_k, void* dy_dev, float* dweights_dev, void* stream) {
  int rc = check_tokens(dtype, M, H, top_k);
  if (rc != QMOE_OK) return rc;
  if (bad_ld(ldd, H) || bad_ld(ldy, H)) return QMOE_ERR_SHAPE;
  if (M == 0) return QMOE_OK;
  if (!dout_dev || !y_dev || !sorted_pair_dev || !pair_pos_dev || !topk_weights_dev || !dy_dev ||
      !dweights_dev)
    return QMOE_ERR_ARG;
  const int es = elem_size(dtype);
  if (misaligned(dout_dev, es) || misaligned(y_dev, es) || misaligned(dy_dev, es) ||
      misaligned(sorted_pair_dev, 4) || misaligned(pair_pos_dev, 4) ||
      misaligned(topk_weights_dev, 4) || misaligned(dweights_dev, 4))
    return QMOE_ERR_ARG;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != QMOE_OK) return rc;
  TokenArgs a = {};
  a.y = y_dev;
  a.ldy = ldy;
  a.dout = dout_dev;
  a.ldd = ldd;
  a.sorted_pair = sorted_pair_dev;
  a.pair_pos = pair_pos_dev;
  a.weights = topk_weights_dev;
  a.M = M;
  a.H = H;
  a.top_k = top_k;
  a.out = dy_dev;
  a.dweights = dweights_dev;
  Chunk chunk;
  chunk.rows(y_dev, ldy, H, es);
  chunk.rows(dout_dev, ldd, H, es);
  chunk.rows(dy_dev, H, H, es);
  return cuda_rc(launch_unsort_backward(a, dtype, chunk.bytes / es, sms,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

static int check_lora(int M, int K, int N, int R, int L) {
  if (M < 0 || K < 8 || K > 65536 || K % 8 || N < 1 || N > 131072 || R < 8 || R > 128 || R % 8 ||
      L < 1 || L > 65536 || (long long)M * R >= (1LL << 31))
    return QMOE_ERR_SHAPE;
  return QMOE_OK;
}

// Workspace of qmoe_lora_linear: the error word's block, the tiles' adapter lists, the
// low-rank activations.  Each part is as large as any batch of up to M tokens needs (fewer
// tokens can have more segments of t), so that a workspace made for some batch serves every
// smaller one.
struct LoraLayout {
  size_t count, bad, list, place, left, any_left, t, tleft, total;
};

static LoraLayout lora_layout(int M, int K, int R) {
  LoraLayout L;
  const size_t tiles = (size_t)M / kLoraLeastTile + 1, tokens = (size_t)M + kLoraMostTile;
  L.count = kWsHeaderBytes;
  L.bad = align_up(L.count + 4 * tiles, 256);
  L.list = align_up(L.bad + 4 * tiles, 256);
  L.place = align_up(L.list + 4 * tokens, 256);
  L.left = align_up(L.place + 4 * tokens, 256);
  L.any_left = align_up(L.left + 4 * tokens, 256);
  L.t = align_up(L.any_left + 4 * tiles, 256);
  L.tleft = align_up(L.t + 4 * (size_t)R * lora_segment_rows(M, K, R), 256);
  L.total = align_up(L.tleft + 4 * (size_t)M * R, 256);
  return L;
}

size_t qmoe_lora_workspace_size(int M, int K, int N, int R, int L) {
  if (check_lora(M, K, N, R, L) != QMOE_OK) return 0;
  return M == 0 ? kWsHeaderBytes : lora_layout(M, K, R).total;
}

int qmoe_lora_linear(const void* x_dev, int dtype, long long ldx, const void* w_dev,
                     const void* a_dev, const void* b_dev, const int32_t* adapter_ids_dev,
                     const float* scales_dev, const void* base_dev, long long ldbase,
                     void* out_dev, int M, int K, int N, int R, int L, void* workspace_dev,
                     size_t ws_bytes, void* stream) {
  if (dtype != QMOE_DTYPE_BF16 && dtype != QMOE_DTYPE_FP16) return QMOE_ERR_ARG;
  int rc = check_lora(M, K, N, R, L);
  if (rc != QMOE_OK) return rc;
  if (ldx < K || ldx % 8 || (base_dev && bad_ld(ldbase, N))) return QMOE_ERR_SHAPE;
  if (M == 0) return QMOE_OK;
  if (!x_dev || !a_dev || !b_dev || !adapter_ids_dev || !scales_dev || !out_dev || !workspace_dev)
    return QMOE_ERR_ARG;
  if (misaligned(x_dev, 16) || misaligned(w_dev, 16) || misaligned(a_dev, 16) ||
      misaligned(b_dev, 16) || misaligned(adapter_ids_dev, 4) || misaligned(scales_dev, 4) ||
      misaligned(base_dev, 2) || misaligned(out_dev, 2) || misaligned(workspace_dev, 256))
    return QMOE_ERR_ARG;
  if (ws_bytes < qmoe_lora_workspace_size(M, K, N, R, L)) return QMOE_ERR_WORKSPACE;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != QMOE_OK) return rc;
  LoraArgs p = {};
  static_cast<LoraPlan&>(p) = lora_plan(M, K, N, R, w_dev != nullptr);
  const LoraLayout W = lora_layout(M, K, R);
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace_dev);
  p.dtype = dtype;
  p.x = x_dev;
  p.ldx = ldx;
  p.w = w_dev;
  p.a = a_dev;
  p.b = b_dev;
  p.ids = adapter_ids_dev;
  p.scales = scales_dev;
  p.base = base_dev;
  p.ldbase = ldbase;
  p.out = out_dev;
  p.M = M;
  p.K = K;
  p.N = N;
  p.R = R;
  p.L = L;
  p.err = reinterpret_cast<unsigned int*>(ws);
  p.count = reinterpret_cast<int*>(ws + W.count);
  p.bad = reinterpret_cast<int*>(ws + W.bad);
  p.list = reinterpret_cast<int*>(ws + W.list);
  p.place = reinterpret_cast<int*>(ws + W.place);
  p.t = reinterpret_cast<float*>(ws + W.t);
  p.left = reinterpret_cast<unsigned int*>(ws + W.left);
  p.any_left = reinterpret_cast<unsigned int*>(ws + W.any_left);
  p.tleft = reinterpret_cast<float*>(ws + W.tleft);
  p.wide = chunked(out_dev, N, N, 2, 16);
  return cuda_rc(launch_lora(p, sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
