// The norms after and before a block, with the block's gate and the residual between them:
//   v = y * post_rstd * (offset + post_weight)        post_rstd = 1 / sqrt(mean(y^2) + eps)
//   out = residual_scale * residual + gate * v
//   normed = out * pre_rstd * (offset + pre_weight)    pre_rstd likewise from out
// in one pass: a row of y and of the residual is read once into registers, and what the row's two
// sums wait for never leaves them.  out is rounded once, when it is written; normed is made from
// the sums before that rounding.  Bound by memory: four rows a token where all parts are there. Of
// many rows each CTA takes one after the other, and copies the next ones to shared memory while a
// row waits for its sums (norm.cuh), as many CTAs an SM as 1024 threads are: where two rows and the
// vectors fit a CTA's share, in 16 bits with both norms and a residual at 7168 columns, with less
// beside them at more widths.  Elsewhere, and of few rows, a row has a CTA and comes straight from
// memory.  8192 rows of 7168 bf16: 81.6 us in a graph, 5.8 TB/s, with a token's gate 87.5 (straight
// 137); 58.7 million elements straight at 1024 to 5120 and 8192 columns: 81 to 94 us, with a
// channel's or full gate 95 to 120 (full: five matrices), in fp32 half as many 73 to 78 (gated 77
// to 124); 16 rows: 3.0 us.
#include "norm.cuh"

namespace qmoe {
namespace {

// CTAs an SM that 1024 threads of 64 registers are, and each one's share of shared memory (less
// what the system and the sums' buffers take).
int norm_ctas(int threads) { return 1024 / threads; }
int norm_cta_bytes(int threads) {
  const int share = 233472 / norm_ctas(threads) - 1280;
  return share < kNormRingBytes ? share : kNormRingBytes;
}

enum { kPost, kPre, kGate };  // vectors over the columns

template <class T, int VEC, int NCH, In HOW, bool GATED>
__global__ void __launch_bounds__(HOW == In::kDirect ? 1024 : 512, HOW == In::kDirect ? 1 : 2)
    norm_forward_kernel(const NormArgs a) {
  __shared__ float sums[64];
  extern __shared__ __align__(16) uint8_t ring_raw[];
  const int threads = a.threads;  // of a row
  const int rows = norm_rows(threads);
  const int tid = rows == 1 ? threadIdx.x : threadIdx.x & 31;
  const int unit = blockIdx.x * rows + (rows == 1 ? 0 : threadIdx.x >> 5);
  RowSum row_sum{sums, threads / 32};
  using raw_t = typename Pack<T, VEC>::raw_t;
  constexpr int kMats = GATED ? 3 : 2, kElems = VEC * NCH;
  const float per = 1.f / (float)a.H;
  const int form = GATED ? a.gate_form : -1;
  const bool full_t = form == QMOE_GATE_FULL && !a.gate_fp32;
  int col[NCH];
  bool in[NCH];
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
    col[k] = (tid + k * threads) * VEC;
    in[k] = col[k] < a.H;
  }
  // the weights with their offset, and a channel's gate
  const Vectors<VEC, NCH> vectors{
      ring_raw + threadIdx.x * sizeof(float) * Vectors<VEC, NCH>::kPart,
      (int)(blockDim.x * sizeof(float)) * Vectors<VEC, NCH>::kPart};
  auto slot = [&](int which) {  // the vectors that are there, one after the other
    return which == kPost ? 0
                          : (a.post_weight != nullptr) +
                                (which == kGate && a.pre_weight != nullptr ? 1 : 0);
  };
  auto load_vector = [&](int which, int k, float (&f)[VEC]) {
    const void* p = which == kGate ? a.gate : which == kPost ? a.post_weight : a.pre_weight;
    load_either<T, VEC>(p, which == kGate ? a.gate_fp32 : a.weight_fp32, col[k], f);
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      f[e] = which == kGate ? gate_value(a, f[e]) : a.weight_offset + f[e];
  };
  auto vector = [&](int which, int k, float (&f)[VEC]) {
    if constexpr (HOW != In::kDirect) {
      vectors.get(slot(which), k, f);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[e] = 0.f;
      if (in[k]) load_vector(which, k, f);
    }
  };
  // f's elements times a vector's
  auto times = [&](int which, float by, float (&f)[kElems]) {
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      float w[VEC];
      vector(which, k, w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[k * VEC + e] *= by * w[e];
    }
  };
  auto put = [&](void* base, int row, const float (&f)[kElems]) {
    T* to = reinterpret_cast<T*>(base) + (size_t)row * a.H;
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      Pack<T, VEC> o;
#pragma unroll
      for (int e = 0; e < VEC; ++e) o.v[e] = from_f32<T>(f[k * VEC + e]);
      if (in[k]) *reinterpret_cast<raw_t*>(to + col[k]) = o.raw;
    }
  };
  // the matrices that a row is read from
  const int own_row = rows == 1 ? 0 : threadIdx.x >> 5;
  RowsIn<T, VEC, NCH, HOW, kMats> in_rows;
  in_rows.source[0] = a.y, in_rows.apart[0] = a.ldy;
  in_rows.source[1] = a.residual, in_rows.apart[1] = a.ldr;
  if constexpr (GATED) in_rows.source[2] = full_t ? a.gate : nullptr, in_rows.apart[2] = a.ldgate;
  in_rows.M = a.M, in_rows.H = a.H, in_rows.units = a.units, in_rows.depth = a.depth;
  in_rows.mats = a.mats, in_rows.tid = tid, in_rows.threads = threads;
  in_rows.one_warp = threads == 32;
  in_rows.stride = HOW == In::kOwn ? (int)(blockDim.x * sizeof(raw_t))
                                   : (a.H * (int)sizeof(T) + 30) / 16 * 16;
  in_rows.base = smem_u32(ring_raw) + vector_bytes(a.vectors, VEC * NCH) * blockDim.x +
                 (HOW == In::kOwn ? (uint32_t)threadIdx.x * (uint32_t)sizeof(raw_t)
                                  : (uint32_t)(own_row * a.depth * a.mats * in_rows.stride));
  grid_dep_wait();
  grid_dep_launch();
  in_rows.begin(unit, col, in);
  if constexpr (HOW != In::kDirect) {
    const bool there[3] = {a.post_weight != nullptr, a.pre_weight != nullptr,
                           form == QMOE_GATE_CHANNEL};
#pragma unroll
    for (int k = 0; k < NCH; ++k)
#pragma unroll
      for (int i = 0; i < (GATED ? 3 : 2); ++i) {
        float f[VEC] = {};
        if (!there[i]) continue;
        if (in[k]) load_vector(i, k, f);
        vectors.put(slot(i), k, f);
      }
  }
  for (int row = unit; row < a.M; row += a.units) {
    in_rows.next(row, col, in);
    float v[kElems];
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      float f[VEC];
      in_rows.chunk(0, k, in, f);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[k * VEC + e] = f[e];
    }
    float scale = 1.f;  // a token's gate
    if (form == QMOE_GATE_TOKEN) {
      float one[1];
      load_either<T, 1>(a.gate, a.gate_fp32, row * a.ldgate, one);
      scale = gate_value(a, one[0]);
    }
    if (a.post_weight) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kElems; ++i) s = fmaf(v[i], v[i], s);
      const float rstd = rsqrtf(row_sum(s) * per + a.eps);
      if (tid == 0 && a.post_rstd) a.post_rstd[row] = rstd;
      times(kPost, rstd, v);
    }
    if (form == QMOE_GATE_CHANNEL) {
      times(kGate, 1.f, v);
    } else if (form == QMOE_GATE_TOKEN) {
#pragma unroll
      for (int i = 0; i < kElems; ++i) v[i] *= scale;
    } else if (form == QMOE_GATE_FULL) {
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        float f[VEC] = {};
        if (full_t)
          in_rows.chunk(GATED ? 2 : 0, k, in, f);
        else if (in[k])
          load_either<T, VEC>(a.gate, true, row * a.ldgate + col[k], f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[k * VEC + e] *= gate_value(a, f[e]);
      }
    }
    if (a.residual) {
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        float f[VEC];
        in_rows.chunk(1, k, in, f);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          v[k * VEC + e] = fmaf(a.residual_scale, f[e], v[k * VEC + e]);
      }
    }
    if (a.out) put(a.out, row, v);
    if (!a.pre_weight) continue;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kElems; ++i) s = fmaf(v[i], v[i], s);
    const float rstd = rsqrtf(row_sum(s) * per + a.eps);
    if (tid == 0 && a.pre_rstd) a.pre_rstd[row] = rstd;
    times(kPre, rstd, v);
    put(a.normed, row, v);
  }
}

template <class T, int VEC, int ELEMS, In HOW, bool GATED>
cudaError_t run(NormArgs a, int sms, cudaStream_t stream) {
  a.threads = norm_threads(a.H, VEC, ELEMS);
  const int rows = norm_rows(a.threads), threads = a.threads * rows;
  auto* k = norm_forward_kernel<T, VEC, ELEMS / VEC, HOW, GATED>;
  int ctas = (a.M + rows - 1) / rows;
  size_t smem = 0;
  if (HOW != In::kDirect) {
    smem = (size_t)vector_bytes(a.vectors, ELEMS) * threads +
           (size_t)a.depth * stage_bytes<T, VEC, HOW>(a.mats, a.threads, rows, ELEMS, a.H);
    const cudaError_t e = allow_smem(k, kNormRingBytes);
    if (e != cudaSuccess) return e;
    const int most = norm_ctas(threads) * sms;
    if (ctas > most) ctas = most;
  }
  a.units = ctas * rows;
  return launch_pdl(k, dim3(ctas), threads, smem, stream, a);
}

// Elements of a row a thread holds: eight where there are few rows, for the shortest way through
// one; else sixteen, and more in the longest rows.
template <class T, int VEC, bool GATED>
cudaError_t of_length(NormArgs a, int sms, cudaStream_t stream) {
  if (a.H <= 8192 && a.M <= 2 * sms) return run<T, VEC, 8, In::kDirect, GATED>(a, sms, stream);
  constexpr In kHow = VEC * sizeof(T) >= 4 ? In::kOwn : In::kShared;
  const int row_threads = norm_threads(a.H, VEC, 16), rows = norm_rows(row_threads);
  if (row_threads <= 512) {
    const int left = norm_cta_bytes(row_threads * rows) -
                     vector_bytes(a.vectors, 16) * row_threads * rows;
    a.depth = left / stage_bytes<T, VEC, kHow>(a.mats, row_threads, rows, 16, a.H);
    if (a.depth > 4) a.depth = 4;
    if (a.depth >= 2) return run<T, VEC, 16, kHow, GATED>(a, sms, stream);
  }
  if (a.H <= 16384) return run<T, VEC, 16, In::kDirect, GATED>(a, sms, stream);
  return run<T, VEC, 64, In::kDirect, GATED>(a, sms, stream);
}

template <class T, int VEC>
cudaError_t of_gate(const NormArgs& a, int sms, cudaStream_t stream) {
  return a.gate ? of_length<T, VEC, true>(a, sms, stream) : of_length<T, VEC, false>(a, sms, stream);
}

template <class T>
cudaError_t of_chunk(const NormArgs& a, int chunk, int sms, cudaStream_t stream) {
  constexpr int kWide = 16 / (int)sizeof(T);
  if (chunk == kWide) return of_gate<T, kWide>(a, sms, stream);
  if constexpr (sizeof(T) == 2)
    if (chunk >= 2) return of_gate<T, 2>(a, sms, stream);
  return of_gate<T, 1>(a, sms, stream);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& args, int dtype, int chunk, int sms, cudaStream_t stream) {
  NormArgs a = args;
  a.mats = 1 + (a.residual != nullptr) +
           (a.gate && a.gate_form == QMOE_GATE_FULL && !a.gate_fp32);
  a.vectors = (a.post_weight != nullptr) + (a.pre_weight != nullptr) +
              (a.gate && a.gate_form == QMOE_GATE_CHANNEL);
  if (dtype == QMOE_DTYPE_BF16) return of_chunk<__nv_bfloat16>(a, chunk, sms, stream);
  if (dtype == QMOE_DTYPE_FP16) return of_chunk<__half>(a, chunk, sms, stream);
  return of_chunk<float>(a, chunk, sms, stream);
}

}  // namespace qmoe
