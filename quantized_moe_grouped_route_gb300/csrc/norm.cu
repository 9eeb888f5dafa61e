// The norms after and before a block, with the block's gate and the residual between them:
//   v = y * post_rstd * (offset + post_weight)        post_rstd = 1 / sqrt(mean(y^2) + eps)
//   out = residual_scale * residual + gate * v
//   normed = out * pre_rstd * (offset + pre_weight)    pre_rstd likewise from out
// in one pass: a row of y and of the residual is read once into registers, and what the row's two
// sums wait for never leaves them.  out is rounded once, when it is written; normed is made from
// the sums before that rounding.  Bound by memory: four rows a token where all parts are there.
#include "norm.cuh"

namespace qmoe {
namespace {

template <class T, int VEC, int NCH>
__global__ void __launch_bounds__(VEC* NCH > 32 ? 1024 : VEC * NCH > 8 ? 512 : 1024)
    norm_forward_kernel(const NormArgs a) {
  __shared__ float sums[64];
  const int threads = a.threads;  // of a row
  const int rows = norm_rows(threads);
  const int tid = rows == 1 ? threadIdx.x : threadIdx.x & 31;
  const int row = blockIdx.x * rows + (rows == 1 ? 0 : threadIdx.x >> 5);
  if (row >= a.M) return;  // (a warp with a row of its own)
  RowSum row_sum{sums, threads / 32};
  using raw_t = typename Pack<T, VEC>::raw_t;
  int col[NCH];
  bool in[NCH];
  Pack<T, VEC> y[NCH], r[NCH], g[NCH];
  const bool full = a.gate && a.gate_form == QMOE_GATE_FULL && !a.gate_fp32;
  grid_dep_wait();
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
    col[k] = (tid + k * threads) * VEC;
    in[k] = col[k] < a.H;
    const long long at = in[k] ? col[k] : 0;
    y[k].raw = load_if(reinterpret_cast<const raw_t*>(reinterpret_cast<const T*>(a.y) +
                                                      row * a.ldy + at), in[k]);
    if (a.residual)
      r[k].raw = load_if(reinterpret_cast<const raw_t*>(reinterpret_cast<const T*>(a.residual) +
                                                        row * a.ldr + at), in[k]);
    if (full)
      g[k].raw = load_if(reinterpret_cast<const raw_t*>(reinterpret_cast<const T*>(a.gate) +
                                                        row * a.ldgate + at), in[k]);
  }
  float v[NCH][VEC];
#pragma unroll
  for (int k = 0; k < NCH; ++k)
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[k][e] = to_f32(y[k].v[e]);
  float scale = 1.f;
  if (a.gate && a.gate_form == QMOE_GATE_TOKEN) {
    float one[1];
    load_either<T, 1>(a.gate, a.gate_fp32, row * a.ldgate, one);
    scale = gate_value(a, one[0]);
  }
  if (a.post_weight) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < NCH; ++k)
#pragma unroll
      for (int e = 0; e < VEC; ++e) s = fmaf(v[k][e], v[k][e], s);
    const float rstd = rsqrtf(row_sum(s) / (float)a.H + a.eps);
    if (tid == 0 && a.post_rstd) a.post_rstd[row] = rstd;
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      float w[VEC];
      if (!in[k]) continue;
      load_either<T, VEC>(a.post_weight, a.weight_fp32, col[k], w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[k][e] *= rstd * (a.weight_offset + w[e]);
    }
  }
  if (a.gate) {
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      float f[VEC];
      if (!in[k]) continue;
      if (a.gate_form == QMOE_GATE_TOKEN) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[k][e] *= scale;
        continue;
      }
      if (full) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = to_f32(g[k].v[e]);
      } else {
        const long long at = a.gate_form == QMOE_GATE_FULL ? row * a.ldgate : 0;
        load_either<T, VEC>(a.gate, a.gate_fp32, at + col[k], f);
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[k][e] *= gate_value(a, f[e]);
    }
  }
  if (a.residual) {
#pragma unroll
    for (int k = 0; k < NCH; ++k)
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[k][e] = fmaf(a.residual_scale, to_f32(r[k].v[e]), v[k][e]);
  }
  const size_t start = (size_t)row * a.H;
  if (a.out) {
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      Pack<T, VEC> o;
#pragma unroll
      for (int e = 0; e < VEC; ++e) o.v[e] = from_f32<T>(v[k][e]);
      if (in[k]) *reinterpret_cast<raw_t*>(reinterpret_cast<T*>(a.out) + start + col[k]) = o.raw;
    }
  }
  if (!a.pre_weight) return;
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < NCH; ++k)
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (in[k]) s = fmaf(v[k][e], v[k][e], s);
  const float rstd = rsqrtf(row_sum(s) / (float)a.H + a.eps);
  if (tid == 0 && a.pre_rstd) a.pre_rstd[row] = rstd;
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
    float w[VEC];
    if (!in[k]) continue;
    load_either<T, VEC>(a.pre_weight, a.weight_fp32, col[k], w);
    Pack<T, VEC> o;
#pragma unroll
    for (int e = 0; e < VEC; ++e) o.v[e] = from_f32<T>(v[k][e] * (rstd * (a.weight_offset + w[e])));
    *reinterpret_cast<raw_t*>(reinterpret_cast<T*>(a.normed) + start + col[k]) = o.raw;
  }
}

template <class T, int VEC, int ELEMS>
cudaError_t run(NormArgs a, cudaStream_t stream) {
  a.threads = norm_threads(a.H, VEC, ELEMS);
  const int rows = norm_rows(a.threads);
  norm_forward_kernel<T, VEC, ELEMS / VEC>
      <<<(a.M + rows - 1) / rows, a.threads * rows, 0, stream>>>(a);
  return cudaGetLastError();
}

// Elements of a row a thread holds: few where there are few rows, for the shortest way through
// one; 32 otherwise, so that fewer threads wait for a row's sums; 64 for the longest rows.
template <class T, int VEC>
cudaError_t of_elements(const NormArgs& a, int sms, cudaStream_t stream) {
  if (a.H <= 8192 && a.M <= 2 * sms) return run<T, VEC, 8>(a, stream);
  if (a.H <= 16384) return run<T, VEC, 32>(a, stream);
  return run<T, VEC, 64>(a, stream);
}

template <class T>
cudaError_t of_chunk(const NormArgs& a, int chunk, int sms, cudaStream_t stream) {
  constexpr int kWide = 16 / (int)sizeof(T);
  if (chunk == kWide) return of_elements<T, kWide>(a, sms, stream);
  if (sizeof(T) == 2 && chunk >= 2) return of_elements<T, 2>(a, sms, stream);
  return of_elements<T, 1>(a, sms, stream);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, int dtype, int chunk, int sms, cudaStream_t stream) {
  if (dtype == QMOE_DTYPE_BF16) return of_chunk<__nv_bfloat16>(a, chunk, sms, stream);
  if (dtype == QMOE_DTYPE_FP16) return of_chunk<__half>(a, chunk, sms, stream);
  return of_chunk<float>(a, chunk, sms, stream);
}

}  // namespace qmoe
