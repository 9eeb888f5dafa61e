// The expert gate: each token's top_k experts and their routing weights from the router's
// logits, and the gradient of the logits.
//
// A row of logits l[0..E) gives every expert a choice value: l itself (softmax scoring) or
// sigmoid(l) + bias (sigmoid scoring).  An expert whose logit or choice value is -infinity
// or NaN is masked.  With groups, only the topk_group best of n_group equal runs of experts
// stay, a group counting by its largest choice value (softmax) or by the sum of its two
// largest (sigmoid).  The top_k unmasked experts are taken by choice value, ties to the
// lowest index; a slot without an expert gets id -1 and weight 0.  Weights:
//   softmax, renormalized  w = scale exp(l_e) / sum over the chosen of exp(l)
//   softmax                w = scale exp(l_e) / sum over all unmasked of exp(l)
//   sigmoid, renormalized  w = scale s_e / (sum over the chosen of s + 1e-20)
//   sigmoid                w = scale s_e
// The choice value is computed with the same fp32 operations as its definition (one
// expf, one addition, one division, one addition), so which experts are chosen does not
// depend on how a kernel is arranged; only the weights' sums have an order of their own.
#include <math.h>

#include "common.cuh"
#include "launch.h"
#include "pack.cuh"

namespace qmoe {
namespace {

constexpr int kGateWarps = 4;

// An unsigned key in the order of the float (both zeros equal); 0 is kept for masked.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);  // a negative's bits all turn
}

// ... of a group's score: the sum of an infinite choice value and a masked one is NaN, which
// comes before all (compared as floats it came before none and none before it, so that one
// group more than topk_group stayed).
__device__ __forceinline__ uint32_t group_key(float v) {
  return v == v ? order_key(v) : 0xffffffffu;
}

// The reciprocal is correctly rounded, so this is 1 / (1 + exp(-l)) to the bit.
__device__ __forceinline__ float sigmoid_f32(float l) { return __frcp_rn(1.0f + expf(-l)); }

// Elements e0 .. e0 + VPT - 1 of a row of E as fp32, -infinity past its end; VEC: in wide
// loads (the row's start, E and e0 are multiples of their length).
template <class T, int VPT>
__host__ __device__ constexpr int run_chunk() {
  return VPT * sizeof(T) <= 16 ? VPT : 16 / (int)sizeof(T);
}
template <class T, int VPT, bool VEC>
__device__ __forceinline__ void load_run(const T* __restrict__ l, int e0, int E, float (&v)[VPT]) {
  if constexpr (VEC) {
    constexpr int N = run_chunk<T, VPT>();
    using P_ = Pack<T, N>;
#pragma unroll
    for (int c = 0; c < VPT / N; ++c) {
      P_ x;
      const bool in = e0 + c * N < E;
      if (in) x.raw = *reinterpret_cast<const typename P_::raw_t*>(l + e0 + c * N);
#pragma unroll
      for (int i = 0; i < N; ++i) v[c * N + i] = in ? to_f32(x.v[i]) : -INFINITY;
    }
  } else {
#pragma unroll
    for (int j = 0; j < VPT; ++j) v[j] = e0 + j < E ? to_f32(l[e0 + j]) : -INFINITY;
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Which groups stay, as a bit mask: the warp's choice values are in row[E] (shared).  The
// lanes of a warp are dealt to the groups (a power of two of them each); a group's rank is
// the count of groups before it by (score, index).
__device__ __forceinline__ uint32_t best_groups(const float* row, int E, int n_group,
                                                int topk_group, bool top2, int lane) {
  const int size = E / n_group;
  int per = 32;  // lanes per group
  while (per * n_group > 32) per >>= 1;
  const int g = lane / per, sub = lane % per;
  float a = -INFINITY, b = -INFINITY;  // the two largest
  if (g < n_group) {
    const int n = (size + per - 1) / per;
    int i = g % n;  // start apart, so that the groups' reads fall on different banks
    for (int t = 0; t < n; ++t) {
      const int e = i * per + sub;
      const float v = e < size ? row[g * size + e] : -INFINITY;
      if (v > a) {
        b = a;
        a = v;
      } else if (v > b) {
        b = v;
      }
      if (++i == n) i = 0;
    }
  }
  for (int o = 1; o < per; o <<= 1) {
    const float a2 = __shfl_xor_sync(0xffffffffu, a, o);
    const float b2 = __shfl_xor_sync(0xffffffffu, b, o);
    const float lo = fminf(a, a2);
    a = fmaxf(a, a2);
    b = fmaxf(lo, fmaxf(b, b2));
  }
  // a group of one expert has no second: it counts by that expert alone
  const uint32_t score = group_key(top2 && size > 1 ? a + b : a);
  int rank = 0;
  for (int h = 0; h < n_group; ++h) {
    const uint32_t s = __shfl_sync(0xffffffffu, score, h * per);
    rank += s > score || (s == score && h < g);
  }
  const uint32_t lanes = __ballot_sync(0xffffffffu, g < n_group && sub == 0 && rank < topk_group);
  uint32_t keep = 0;
  for (int h = 0; h < n_group; ++h) keep |= ((lanes >> (h * per)) & 1u) << h;
  return keep;
}

// A warp per row; lane holds the VPT experts from lane * VPT on, so that the lowest index
// among equal keys is the lowest lane's lowest j, and a group of a power of two of lanes is
// reduced by shuffles.
//
// The top_k are found in three steps, without a round per slot over all keys (which was
// half of the kernel's instructions): the top_k-th largest of the lanes' largest keys bounds
// the top_k-th largest key from below; the keys that reach the bound (a few more than
// top_k) are compacted to one per lane; and each of those counts the candidates before it,
// which is its slot.  More than 32 candidates (many equal keys, or top_k near 32 or above)
// take a round per slot instead.
// A candidate is one 64-bit number, its key above the complement of its expert, so that the
// larger number comes first.
struct GateScratch {
  unsigned long long cand[32];
};

template <class T, int VPT, bool VEC>
__global__ void __launch_bounds__(kGateWarps * 32) gate_kernel(const GateArgs p) {
  extern __shared__ float rows[];  // [kGateWarps][E], with groups that lanes do not align with
  __shared__ GateScratch scratch[kGateWarps];
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned below = (1u << lane) - 1u;
  const bool sigmoid = p.scoring == QMOE_GATE_SIGMOID;
  const int e0 = lane * VPT;
  unsigned long long* cand = scratch[warp].cand;
  grid_dep_wait();
  grid_dep_launch();
  for (long long m = (long long)blockIdx.x * kGateWarps + warp; m < p.M;
       m += (long long)gridDim.x * kGateWarps) {
    const T* l = reinterpret_cast<const T*>(p.logits) + m * p.ld;
    float v[VPT];
    load_run<T, VPT, VEC>(l, e0, p.E, v);
    float top = 0.f, total = 0.f;  // over all unmasked experts
    if (!sigmoid && !p.renormalize) {
      top = -INFINITY;
#pragma unroll
      for (int j = 0; j < VPT; ++j) top = fmaxf(top, v[j]);  // fmaxf ignores NaN
      top = warp_max(top);
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        if (v[j] > -INFINITY) total += expf(v[j] - top);
      total = warp_sum(total);
    }
    if (sigmoid) {
      float bias[VPT];
      if (p.bias) load_run<float, VPT, VEC>(p.bias, e0, p.E, bias);
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const float s = sigmoid_f32(v[j]);
        v[j] = v[j] > -INFINITY ? (p.bias ? s + bias[j] : s) : -INFINITY;
      }
    }
    uint32_t key[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const bool in = v[j] > -INFINITY;  // not so for NaN
      key[j] = in ? order_key(v[j]) : 0u;
      if (!in) v[j] = -INFINITY;
    }
    if (p.group_lanes > 0) {
      // groups of group_lanes whole lanes (a power of two)
      float a = -INFINITY, b = -INFINITY;  // the two largest
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        b = fmaxf(b, fminf(a, v[j]));
        a = fmaxf(a, v[j]);
      }
      for (int o = 1; o < p.group_lanes; o <<= 1) {
        const float a2 = __shfl_xor_sync(kAll, a, o), b2 = __shfl_xor_sync(kAll, b, o);
        b = fmaxf(fminf(a, a2), fmaxf(b, b2));
        a = fmaxf(a, a2);
      }
      const uint32_t score = group_key(sigmoid && p.E > p.n_group ? a + b : a);
      const int g = lane / p.group_lanes;
      int rank = 0;
      for (int h = 0; h < p.n_group; ++h) {
        const uint32_t s = __shfl_sync(kAll, score, h * p.group_lanes);
        rank += s > score || (s == score && h < g);
      }
      if (rank >= p.topk_group) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) key[j] = 0u;
      }
    } else if (p.n_group > 1) {
      float* row = rows + warp * p.E;
      __syncwarp();
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        if (e0 + j < p.E) row[e0 + j] = v[j];
      __syncwarp();
      const uint32_t keep = best_groups(row, p.E, p.n_group, p.topk_group, sigmoid, lane);
      const int size = p.E / p.n_group;
      int g = e0 / size, left = (g + 1) * size - e0;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        if (!((keep >> (g & 31)) & 1u)) key[j] = 0u;
        if (--left == 0) {
          ++g;
          left = size;
        }
      }
    }
    uint32_t best = 0;
#pragma unroll
    for (int j = 0; j < VPT; ++j) best = max(best, key[j]);
    // a bound from below of the top_k-th key
    uint32_t bound = 0, mx = best;
#pragma unroll 1
    for (int r = 0; r < p.top_k; ++r) {
      bound = __reduce_max_sync(kAll, mx);
      if (mx == bound) mx = 0u;
    }
    bound = max(bound, 1u);  // no lane left: every unmasked key
    // each lane's candidates, at a place after those of the lanes before it
    int mine_n = 0;
#pragma unroll
    for (int j = 0; j < VPT; ++j) mine_n += key[j] >= bound;
    int at = 0, n = 0;
#pragma unroll
    for (int bit = 1; bit <= VPT; bit <<= 1) {
      const unsigned who = __ballot_sync(kAll, mine_n & bit);
      at += bit * __popc(who & below);
      n += bit * __popc(who);
    }
    if (n <= 32) {
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        if (key[j] >= bound) cand[at++] = (unsigned long long)key[j] << 32 | (uint32_t)~(e0 + j);
    }
    __syncwarp();
    // slot `slot` of the row belongs to this lane, with this expert (and a second one above 32)
    const int nslot = p.top_k > 32 ? 2 : 1;
    int slot[2] = {-1, -1}, expert[2] = {-1, -1};
    if (n <= 32) {
      // the lanes past the candidates take the slots that are left over, as empty ones
      if (lane >= n) cand[lane] = 0u;
      __syncwarp();
      const unsigned long long mine = cand[lane];
      int rank = 0;
#pragma unroll 1
      for (int i = 0; i < n; i += 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) rank += cand[i + k] > mine;
      }
      slot[0] = lane < n ? rank : lane;
      if (lane < n) expert[0] = (int)~(uint32_t)mine;
      slot[1] = lane + 32;
    } else {
      for (int r = 0; r < p.top_k; ++r) {
        const uint32_t w = __reduce_max_sync(kAll, best);
        if (w == 0u) break;
        const int winner = __ffs(__ballot_sync(kAll, best == w)) - 1;
        int j_won = 0;
        if (lane == winner) {
          best = 0u;
          bool gone = false;
#pragma unroll
          for (int j = 0; j < VPT; ++j) {
            if (!gone && key[j] == w) {
              key[j] = 0u;
              j_won = j;
              gone = true;
            }
            best = max(best, key[j]);
          }
        }
        const int e = __shfl_sync(kAll, e0 + j_won, winner);
        if (lane == (r & 31)) expert[r >> 5] = e;
      }
      slot[0] = lane;
      slot[1] = lane + 32;
    }
    __syncwarp();  // the candidates have been read
    float s[2] = {0.f, 0.f}, lv[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (i >= nslot) break;
      if (slot[i] >= p.top_k) slot[i] = expert[i] = -1;
      if (expert[i] >= 0) lv[i] = to_f32(l[expert[i]]);
    }
    float divide = 1.f;
    if (sigmoid) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (i < nslot && expert[i] >= 0) s[i] = sigmoid_f32(lv[i]);
      if (p.renormalize) divide = warp_sum(s[0] + s[1]) + 1e-20f;
    } else {
      if (p.renormalize) top = warp_max(fmaxf(lv[0], lv[1]));
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (i < nslot && expert[i] >= 0) s[i] = expf(lv[i] - top);
      divide = p.renormalize ? warp_sum(s[0] + s[1]) : total;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (i >= nslot) break;
      if (slot[i] >= 0) {
        p.ids[m * p.top_k + slot[i]] = expert[i];
        p.weights[m * p.top_k + slot[i]] = expert[i] >= 0 ? s[i] / divide * p.scale : 0.f;
      }
    }
  }
}

// Gradient of the logits, a warp per row (p = the chosen experts' scores, c = scale):
//   softmax, renormalized  dl_e = c p_e (dw_e - sum p dw) on the chosen, 0 elsewhere
//   softmax                dl_e = c p_e (dw_e [chosen] - sum over the chosen of p dw)
//   sigmoid, renormalized  dl_e = c / S (dw_e - sum (s / S) dw) s_e (1 - s_e), S = sum s + 1e-20
//   sigmoid                dl_e = c dw_e s_e (1 - s_e)
// The chosen experts' gradients go through a shared row, so that the (mostly zero) output
// row leaves in wide stores.
template <class T, int N>
__global__ void __launch_bounds__(kGateWarps * 32) gate_backward_kernel(const GateArgs p) {
  extern __shared__ float rows[];  // [kGateWarps][E]
  using P_ = Pack<T, N>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* row = rows + warp * p.E;
  for (int e = lane; e < p.E; e += 32) row[e] = 0.f;
  __syncwarp();
  grid_dep_wait();
  grid_dep_launch();
  const bool sigmoid = p.scoring == QMOE_GATE_SIGMOID;
  const int nslot = p.top_k > 32 ? 2 : 1;  // slots a lane
  for (long long m = (long long)blockIdx.x * kGateWarps + warp; m < p.M;
       m += (long long)gridDim.x * kGateWarps) {
    const T* l = reinterpret_cast<const T*>(p.logits) + m * p.ld;
    int e[2] = {-1, -1};
    float s[2] = {0.f, 0.f}, dw[2] = {0.f, 0.f}, lv[2] = {-INFINITY, -INFINITY}, d[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (i >= nslot) break;
      const int r = lane + 32 * i;
      e[i] = r < p.top_k ? p.ids_in[m * p.top_k + r] : -1;
      if ((unsigned)e[i] >= (unsigned)p.E) e[i] = -1;
      dw[i] = e[i] >= 0 ? p.dweights[m * p.top_k + r] : 0.f;
      lv[i] = e[i] >= 0 ? to_f32(l[e[i]]) : -INFINITY;
    }
    float top = 0.f, dense = 0.f;  // dense: what every expert's exp(l - top) is multiplied by
    if (sigmoid) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (i < nslot && e[i] >= 0) s[i] = sigmoid_f32(lv[i]);
      // 1 - s as the score of -l: from the rounded s it keeps no bits where s is next to 1
      // (at l = 10 it was off by 0.1 %, from 17 on it was 0)
      float rest[2], inner = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) rest[i] = i < nslot && e[i] >= 0 ? sigmoid_f32(-lv[i]) : 0.f;
      if (p.renormalize) {
        // the weights first, as the softmax below: a single expert's is 1 and its gradient 0
        // (with sum s dw / S something of dw's last bit remained)
        const float total = warp_sum(s[0] + s[1]) + 1e-20f;
        s[0] /= total;
        s[1] /= total;
        inner = warp_sum(s[0] * dw[0] + s[1] * dw[1]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) d[i] = p.scale * s[i] * rest[i] * (dw[i] - inner);
    } else {
      float total = 0.f;
      if (p.renormalize) {
        top = warp_max(fmaxf(lv[0], lv[1]));
      } else {
        top = -INFINITY;
        for (int i = lane; i < p.E; i += 32) top = fmaxf(top, to_f32(l[i]));
        top = warp_max(top);
        for (int i = lane; i < p.E; i += 32) {
          const float li = to_f32(l[i]);
          if (li > -INFINITY) total += expf(li - top);
        }
        total = warp_sum(total);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (i < nslot && e[i] >= 0) s[i] = expf(lv[i] - top);
      if (p.renormalize) total = warp_sum(s[0] + s[1]);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (i < nslot && e[i] >= 0) s[i] /= total;
      const float inner = warp_sum(s[0] * dw[0] + s[1] * dw[1]);
      if (!p.renormalize && __any_sync(0xffffffffu, e[0] >= 0 || e[1] >= 0))
        dense = -p.scale * inner / total;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        d[i] = p.scale * s[i] * (dw[i] - (p.renormalize ? inner : 0.f));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (e[i] >= 0) row[e[i]] = d[i];
    __syncwarp();
    T* out = reinterpret_cast<T*>(p.dlogits) + (size_t)m * p.E;
    for (int c = lane; c < p.E / N; c += 32) {
      P_ o;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float g = row[c * N + i];
        if (dense != 0.f) {
          const float li = to_f32(l[c * N + i]);
          if (li > -INFINITY) g += dense * expf(li - top);
        }
        o.v[i] = from_f32<T>(g);
      }
      *reinterpret_cast<typename P_::raw_t*>(out + (size_t)c * N) = o.raw;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (e[i] >= 0) row[e[i]] = 0.f;
    __syncwarp();
  }
}

template <class K>
cudaError_t launch(K* kernel, const GateArgs& p, size_t smem, int num_sms, cudaStream_t stream) {
  // E <= 2048: at most 32 KB of shared memory, within what needs no opt-in
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  long long blocks = ((long long)p.M + kGateWarps - 1) / kGateWarps;
  if (blocks > num_sms * 32LL) blocks = num_sms * 32LL;
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kGateWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <class T, int VPT>
cudaError_t gate_vpt(GateArgs p, int num_sms, cudaStream_t stream) {
  // groups made of whole lanes, a power of two of them
  const int size = p.E / p.n_group, lanes = size / VPT;
  p.group_lanes = p.n_group > 1 && size % VPT == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
  const size_t smem =
      p.n_group > 1 && p.group_lanes == 0 ? (size_t)kGateWarps * p.E * sizeof(float) : 0;
  constexpr int N = run_chunk<T, VPT>();
  const bool vec = reinterpret_cast<uintptr_t>(p.logits) % (N * sizeof(T)) == 0 && p.ld % N == 0 &&
                   reinterpret_cast<uintptr_t>(p.bias) % (run_chunk<float, VPT>() * 4) == 0 &&
                   p.E % N == 0;
  return vec ? launch(gate_kernel<T, VPT, true>, p, smem, num_sms, stream)
             : launch(gate_kernel<T, VPT, false>, p, smem, num_sms, stream);
}

template <class T>
cudaError_t gate(const GateArgs& p, int num_sms, cudaStream_t stream) {
  if (p.E <= 32) return gate_vpt<T, 1>(p, num_sms, stream);
  if (p.E <= 64) return gate_vpt<T, 2>(p, num_sms, stream);
  if (p.E <= 128) return gate_vpt<T, 4>(p, num_sms, stream);
  if (p.E <= 256) return gate_vpt<T, 8>(p, num_sms, stream);
  if (p.E <= 512) return gate_vpt<T, 16>(p, num_sms, stream);
  if (p.E <= 1024) return gate_vpt<T, 32>(p, num_sms, stream);
  return gate_vpt<T, 64>(p, num_sms, stream);
}

}  // namespace

cudaError_t launch_gate(const GateArgs& p, int dtype, int num_sms, cudaStream_t stream) {
  if (dtype == QMOE_DTYPE_BF16) return gate<__nv_bfloat16>(p, num_sms, stream);
  if (dtype == QMOE_DTYPE_FP16) return gate<__half>(p, num_sms, stream);
  return gate<float>(p, num_sms, stream);
}

cudaError_t launch_gate_backward(const GateArgs& p, int dtype, bool vec, int num_sms,
                                 cudaStream_t stream) {
  const size_t smem = (size_t)kGateWarps * p.E * sizeof(float);
  if (dtype == QMOE_DTYPE_BF16)
    return vec ? launch(gate_backward_kernel<__nv_bfloat16, 8>, p, smem, num_sms, stream)
               : launch(gate_backward_kernel<__nv_bfloat16, 1>, p, smem, num_sms, stream);
  if (dtype == QMOE_DTYPE_FP16)
    return vec ? launch(gate_backward_kernel<__half, 8>, p, smem, num_sms, stream)
               : launch(gate_backward_kernel<__half, 1>, p, smem, num_sms, stream);
  return vec ? launch(gate_backward_kernel<float, 4>, p, smem, num_sms, stream)
             : launch(gate_backward_kernel<float, 1>, p, smem, num_sms, stream);
}

}  // namespace qmoe
