// Gradients of the norms after and before a block (norm.cu).  With x^ = out * pre_rstd and
// y^ = y * post_rstd, w the weights with their offset, <a, b> the mean over a row's elements:
//   g = dout + pre_rstd * (dnormed w_pre - x^ <dnormed w_pre, x^>)       dpre = sum_m dnormed x^
//   dresidual = residual_scale * g,   dgate = g v (summed over what shares a gate),  v = y^ w_post
//   d = gate * g,   dy = post_rstd * (d w_post - y^ <d w_post, y^>)       dpost = sum_m d y^
// One pass over the rows: four are read and two written a token.  The sums over the tokens stay in
// the registers of the threads that own the columns; each CTA (or warp) goes through many rows
// and leaves one row of sums, and a second kernel adds those up in a fixed order.
#include "norm.cuh"

namespace qmoe {
namespace {

// Sums over tokens, by their place in a unit's rows of them.
enum { kPost, kPre, kGate };

// ACC: the sums over the tokens are kept in registers (rows of up to 8192 elements); otherwise in
// the unit's own rows in memory, which its threads alone touch.
template <class T, int VEC, int NCH, bool ACC>
__global__ void __launch_bounds__(1024) norm_backward_kernel(const NormArgs a) {
  __shared__ float sums[64];
  const int threads = a.threads;
  const int rows = norm_rows(threads);
  const int tid = rows == 1 ? threadIdx.x : threadIdx.x & 31;
  const int unit = blockIdx.x * rows + (rows == 1 ? 0 : threadIdx.x >> 5);
  if (unit >= a.units) return;
  RowSum row_sum{sums, threads / 32};
  using raw_t = typename Pack<T, VEC>::raw_t;
  const float per = 1.f / (float)a.H;
  const bool post = a.post_weight != nullptr, pre = a.pre_weight != nullptr;
  const int form = a.gate ? a.gate_form : -1;
  const bool per_channel = form == QMOE_GATE_CHANNEL;
  const bool need_y = post || (a.gate && a.dgate) || (pre && !a.out_in);
  float* acc_rows = a.partial + (size_t)unit * 3 * a.H;
  float acc[ACC ? 3 : 1][NCH][VEC] = {};
  int col[NCH];
  bool in[NCH];
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
    col[k] = (tid + k * threads) * VEC;
    in[k] = col[k] < a.H;
  }
  bool first = true;
  auto add = [&](int which, int k, int e, float v) {
    if constexpr (ACC) {
      acc[which][k][e] += v;
    } else if (in[k]) {
      float* at = acc_rows + (size_t)which * a.H + col[k] + e;
      *at = first ? v : *at + v;
    }
  };
  auto fetch = [&](const void* base, long long ld, int row, int k) {
    Pack<T, VEC> p;
    p.raw = load_if(reinterpret_cast<const raw_t*>(reinterpret_cast<const T*>(base) + row * ld +
                                                   (in[k] ? col[k] : 0)), in[k]);
    return p;
  };
  auto put = [&](void* base, int row, int k, const float (&f)[VEC]) {
    Pack<T, VEC> o;
#pragma unroll
    for (int e = 0; e < VEC; ++e) o.v[e] = from_f32<T>(f[e]);
    if (in[k])
      *reinterpret_cast<raw_t*>(reinterpret_cast<T*>(base) + (size_t)row * a.H + col[k]) = o.raw;
  };
  grid_dep_wait();
  for (int row = unit; row < a.M; row += a.units) {
    Pack<T, VEC> pd[NCH], pn[NCH], py[NCH], po[NCH], pg[NCH];
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      if (a.dout) pd[k] = fetch(a.dout, a.lddout, row, k);
      if (pre) pn[k] = fetch(a.dnormed, a.lddnormed, row, k);
      if (pre && a.out_in) po[k] = fetch(a.out_in, a.ldout, row, k);
      if (need_y) py[k] = fetch(a.y, a.ldy, row, k);
      if (form == QMOE_GATE_FULL && !a.gate_fp32) pg[k] = fetch(a.gate, a.ldgate, row, k);
    }
    float g[NCH][VEC];
#pragma unroll
    for (int k = 0; k < NCH; ++k)
#pragma unroll
      for (int e = 0; e < VEC; ++e) g[k][e] = a.dout ? to_f32(pd[k].v[e]) : 0.f;
    if (pre) {
      const float rstd = a.pre_rstd[row];
      float s = 0.f, x[NCH][VEC], d[NCH][VEC];
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        float w[VEC] = {};
        if (in[k]) load_either<T, VEC>(a.pre_weight, a.weight_fp32, col[k], w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          x[k][e] = to_f32(a.out_in ? po[k].v[e] : py[k].v[e]) * rstd;
          const float dn = to_f32(pn[k].v[e]);
          if (a.dpre_weight) add(kPre, k, e, dn * x[k][e]);
          d[k][e] = in[k] ? dn * (a.weight_offset + w[e]) : 0.f;
          s = fmaf(d[k][e], x[k][e], s);
        }
      }
      const float along = row_sum(s) * per;
#pragma unroll
      for (int k = 0; k < NCH; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) g[k][e] += rstd * (d[k][e] - x[k][e] * along);
    }
    if (a.dresidual) {
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        float f[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = a.residual_scale * g[k][e];
        put(a.dresidual, row, k, f);
      }
    }
    // a token's gate, or 1
    float gate1 = 1.f;
    if (form == QMOE_GATE_TOKEN) {
      float one[1];
      load_either<T, 1>(a.gate, a.gate_fp32, row * a.ldgate, one);
      gate1 = gate_value(a, one[0]);
    }
    const float rstd = post ? a.post_rstd[row] : 1.f;
    float s = 0.f;
    // from here on g holds d, where the gate is an element's own
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      float w[VEC], f[VEC], dg[VEC];
      const bool own = form == QMOE_GATE_FULL || per_channel;
#pragma unroll
      for (int e = 0; e < VEC; ++e) w[e] = 1.f;
      if (post && in[k]) {
        load_either<T, VEC>(a.post_weight, a.weight_fp32, col[k], w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[e] += a.weight_offset;
      }
      if (own && in[k]) {
        if (form == QMOE_GATE_FULL && !a.gate_fp32) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) f[e] = to_f32(pg[k].v[e]);
        } else {
          load_either<T, VEC>(a.gate, a.gate_fp32,
                              (form == QMOE_GATE_FULL ? row * a.ldgate : 0) + col[k], f);
        }
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float unit_y = need_y && in[k] ? to_f32(py[k].v[e]) * rstd : 0.f;
        dg[e] = g[k][e] * unit_y * w[e];
        if (own) {
          const float value = in[k] ? gate_value(a, f[e]) : 0.f;
          g[k][e] *= value;
          s = fmaf(g[k][e], unit_y * w[e], s);
          dg[e] *= gate_slope(a, value);
          if (per_channel && a.dgate) add(kGate, k, e, dg[e]);
        } else {
          s += dg[e];
        }
        if (post && a.dpost_weight) add(kPost, k, e, g[k][e] * gate1 * unit_y);
      }
      if (form == QMOE_GATE_FULL && a.dgate) put(a.dgate, row, k, dg);
    }
    float along = 0.f;
    if (post || (form == QMOE_GATE_TOKEN && a.dgate)) along = row_sum(s);
    if (form == QMOE_GATE_TOKEN && a.dgate && tid == 0)
      reinterpret_cast<float*>(a.dgate)[row] = along * gate_slope(a, gate1);
    along *= gate1 * per;
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      float w[VEC], f[VEC];
      if (!in[k]) continue;
      if (post) load_either<T, VEC>(a.post_weight, a.weight_fp32, col[k], w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        f[e] = g[k][e] * gate1;
        if (post)
          f[e] = rstd * (f[e] * (a.weight_offset + w[e]) - to_f32(py[k].v[e]) * rstd * along);
      }
      put(a.dy, row, k, f);
    }
    first = false;
  }
  if constexpr (ACC) {
    const bool want[3] = {post && a.dpost_weight != nullptr, pre && a.dpre_weight != nullptr,
                          per_channel && a.dgate != nullptr};
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
      for (int k = 0; k < NCH; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (want[i] && in[k]) acc_rows[(size_t)i * a.H + col[k] + e] = acc[i][k][e];
  }
}

// dst[h] = sum over the units of their sum number `which`, 32 columns a CTA.
__global__ void __launch_bounds__(1024) norm_sums_kernel(const float* partial, int units, int H,
                                                         float* post, float* pre, float* gate) {
  __shared__ float part[32][33];
  float* dst = blockIdx.y == kPost ? post : blockIdx.y == kPre ? pre : gate;
  grid_dep_wait();
  if (!dst) return;
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int h = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (h < H) {
    const float* src = partial + (size_t)blockIdx.y * H + h;
#pragma unroll 4
    for (int u = slice; u < units; u += 32) s += src[(size_t)u * 3 * H];
  }
  part[slice][lane] = s;
  __syncthreads();
  if (slice != 0 || h >= H) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) s += part[i][lane];
  dst[h] = s;
}

template <class T, int VEC, int ELEMS, bool ACC>
cudaError_t run(NormArgs a, cudaStream_t stream) {
  a.threads = norm_threads(a.H, VEC, ELEMS);
  const int rows = norm_rows(a.threads);
  norm_backward_kernel<T, VEC, ELEMS / VEC, ACC>
      <<<(a.units + rows - 1) / rows, a.threads * rows, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  float* gate = a.gate && a.gate_form == QMOE_GATE_CHANNEL ? reinterpret_cast<float*>(a.dgate)
                                                           : nullptr;
  float* post = a.post_weight ? a.dpost_weight : nullptr;
  float* pre = a.pre_weight ? a.dpre_weight : nullptr;
  if (!gate && !post && !pre) return cudaSuccess;
  norm_sums_kernel<<<dim3((a.H + 31) / 32, 3), 1024, 0, stream>>>(a.partial, a.units, a.H, post,
                                                                  pre, gate);
  return cudaGetLastError();
}

template <class T, int VEC>
cudaError_t of_elements(const NormArgs& a, cudaStream_t stream) {
  if (a.H <= kNormRegisterColumns) return run<T, VEC, 8, true>(a, stream);
  return run<T, VEC, 64, false>(a, stream);
}

template <class T>
cudaError_t of_chunk(const NormArgs& a, int chunk, cudaStream_t stream) {
  constexpr int kWide = 16 / (int)sizeof(T);
  if (chunk == kWide) return of_elements<T, kWide>(a, stream);
  if (sizeof(T) == 2 && chunk >= 2) return of_elements<T, 2>(a, stream);
  return of_elements<T, 1>(a, stream);
}

}  // namespace

int norm_units(int M, int H) {
  // as many rows in the making as CTAs of 1024 threads' registers hold, a thread eight elements
  const int threads = norm_threads(H < kNormRegisterColumns ? H : kNormRegisterColumns, 8, 8);
  const int most = 152 * (1024 / threads);
  return M < most ? M : most;
}

cudaError_t launch_norm_backward(const NormArgs& a, int dtype, int chunk, cudaStream_t stream) {
  if (dtype == QMOE_DTYPE_BF16) return of_chunk<__nv_bfloat16>(a, chunk, stream);
  if (dtype == QMOE_DTYPE_FP16) return of_chunk<__half>(a, chunk, stream);
  return of_chunk<float>(a, chunk, stream);
}

}  // namespace qmoe
