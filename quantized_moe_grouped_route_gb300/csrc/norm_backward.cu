// Gradients of the norms after and before a block (norm.cu).  With x^ = out * pre_rstd and
// y^ = y * post_rstd, w the weights with their offset, <a, b> the mean over a row's elements:
//   g = dout + pre_rstd * (dnormed w_pre - x^ <dnormed w_pre, x^>)       dpre = sum_m dnormed x^
//   dresidual = residual_scale * g,   dgate = slope * sum of g v over what shares a gate,  v = y^ w_post
//   d = gate * g,   dy = post_rstd * (d w_post - y^ <d w_post, y^>)       dpost = sum_m d y^
// One pass over the rows: four are read and two written a token.  The sums over the tokens stay in
// the registers of the threads that own the columns; each CTA (or warp) goes through many rows and
// leaves one row of sums, and a second kernel adds those up in a fixed order.  A CTA that has an SM
// to itself waits for its own sums, so the next rows are copied meanwhile (norm.cuh).  8192 rows of
// 7168 bf16: 139 us, 5.1 TB/s, and 4 for the second kernel (straight loads 452; with the weights
// read from memory for each row, which the copies leave no L1 for, 244; rows held in registers
// beside the sums, 211).  Other widths, 58.7 million elements each (bytes: 105): 4096 columns 171
// us, 2048 158, 1024 162, where a CTA's up to four rows of shared memory leave no room for all the
// CTAs that the grid has an SM; gated 170 to 310.  Rows that come straight (past 8192 columns, 660
// us and more; half as many elements of fp32 past 5632 columns with both norms and a residual, 650
// to 670) spill the registers of 1024 threads.
#include "norm.cuh"

namespace qmoe {
namespace {

// Sums over tokens, by their place in a unit's rows of them.
enum { kPost, kPre, kGate };

// ACC: the sums over the tokens are kept in registers (rows of up to 8192 elements); otherwise in
// the unit's own rows in memory, which its threads alone touch.  HOW: how rows come in.
template <class T, int VEC, int NCH, bool ACC, In HOW, bool GATED>
__global__ void __launch_bounds__(ACC && VEC > 1 ? 512 : 1024) norm_backward_kernel(const NormArgs a) {
  __shared__ float sums[64];
  extern __shared__ __align__(16) uint8_t ring_raw[];
  const int threads = a.threads;
  const int rows = norm_rows(threads);
  const int tid = rows == 1 ? threadIdx.x : threadIdx.x & 31;
  const int unit = blockIdx.x * rows + (rows == 1 ? 0 : threadIdx.x >> 5);
  if (unit >= a.units) return;
  RowSum row_sum{sums, threads / 32};
  using raw_t = typename Pack<T, VEC>::raw_t;
  constexpr int kMats = GATED ? 5 : 4, kElems = VEC * NCH;
  const float per = 1.f / (float)a.H;
  const bool post = a.post_weight != nullptr, pre = a.pre_weight != nullptr;
  const int form = GATED && a.gate ? a.gate_form : -1;
  const bool per_channel = form == QMOE_GATE_CHANNEL;
  const bool full_t = form == QMOE_GATE_FULL && !a.gate_fp32;
  const int norm_of = a.out_in ? 2 : 3;  // the matrix that the norm before the next block is of
  const bool need_y = post || (GATED && a.dgate) || (pre && !a.out_in);
  float* acc_rows = a.partial + (size_t)unit * 3 * a.H;
  float acc[ACC ? (GATED ? 3 : 2) : 1][kElems] = {};
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
    return which == kPost ? 0 : (post ? 1 : 0) + (which == kGate && pre ? 1 : 0);
  };
  auto load_vector = [&](int which, int k, float (&f)[VEC]) {
    const void* p = which == kGate ? a.gate : which == kPost ? a.post_weight : a.pre_weight;
    load_either<T, VEC>(p, which == kGate ? a.gate_fp32 : a.weight_fp32, col[k], f);
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      f[e] = which == kGate ? gate_value(a, f[e]) : a.weight_offset + f[e];
  };
  auto vector = [&](int which, int k, float (&f)[VEC]) {
    if constexpr (ACC) {
      vectors.get(slot(which), k, f);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[e] = 0.f;
      if (in[k]) load_vector(which, k, f);
    }
  };
  bool first = true;
  // chunk k's f to a unit's sums
  auto add = [&](int which, int k, const float (&f)[VEC]) {
    if constexpr (ACC) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[which][k * VEC + e] += f[e];
    } else if (in[k]) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float* at = acc_rows + (size_t)which * a.H + col[k] + e;
        *at = first ? f[e] : *at + f[e];
      }
    }
  };
  auto put = [&](void* base, int row, const float (&f)[kElems], bool fp32 = false) {
    if (sizeof(T) == 2 && fp32) {  // (a gate's gradient beside 16-bit rows)
      constexpr int kPart = VEC < 4 ? VEC : 4;
      float* to = reinterpret_cast<float*>(base) + (size_t)row * a.H + tid * VEC;
#pragma unroll
      for (int k = 0; k < NCH; ++k)
#pragma unroll
        for (int i = 0; i < VEC; i += kPart) {
          Pack<float, kPart> o;
#pragma unroll
          for (int e = 0; e < kPart; ++e) o.v[e] = f[k * VEC + i + e];
          if (in[k])
            *reinterpret_cast<typename Pack<float, kPart>::raw_t*>(to + k * threads * VEC + i) = o.raw;
        }
      return;
    }
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
  in_rows.source[0] = a.dout, in_rows.apart[0] = a.lddout;
  in_rows.source[1] = pre ? a.dnormed : nullptr, in_rows.apart[1] = a.lddnormed;
  in_rows.source[2] = pre ? a.out_in : nullptr, in_rows.apart[2] = a.ldout;
  in_rows.source[3] = need_y ? a.y : nullptr, in_rows.apart[3] = a.ldy;
  if constexpr (GATED) in_rows.source[4] = full_t ? a.gate : nullptr, in_rows.apart[4] = a.ldgate;
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
  if constexpr (ACC) {
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const bool there[3] = {post, pre, per_channel};
#pragma unroll
      for (int i = 0; i < (GATED ? 3 : 2); ++i) {
        float f[VEC] = {};
        if (!there[i]) continue;
        if (in[k]) load_vector(i, k, f);
        vectors.put(slot(i), k, f);
      }
    }
  }
  in_rows.begin_zero();
  // the norms' scales of a row come with the row before it
  float next_pre = pre ? a.pre_rstd[unit] : 0.f, next_post = post ? a.post_rstd[unit] : 1.f;
  for (int row = unit; row < a.M; row += a.units) {
    const float pre_rstd = next_pre, rstd = next_post;
    if (row + a.units < a.M) {
      if (pre) next_pre = a.pre_rstd[row + a.units];
      if (post) next_post = a.post_rstd[row + a.units];
    }
    in_rows.next(row, col, in);
    auto chunk = [&](int mat, int k, float (&f)[VEC]) { in_rows.chunk(mat, k, in, f); };
    float g[kElems];
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      float f[VEC];
      chunk(0, k, f);
#pragma unroll
      for (int e = 0; e < VEC; ++e) g[k * VEC + e] = f[e];
    }
    if (pre) {
      float s = 0.f, d[kElems];
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        float x[VEC], dn[VEC], w[VEC], p[VEC];
        chunk(norm_of, k, x);
        chunk(1, k, dn);
        vector(kPre, k, w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          p[e] = dn[e] * (x[e] * pre_rstd);
          s = fmaf(p[e], w[e], s);
          d[k * VEC + e] = dn[e] * w[e];
        }
        add(kPre, k, p);
      }
      const float along = row_sum(s) * per * pre_rstd;
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        float x[VEC];
        chunk(norm_of, k, x);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int i = k * VEC + e;
          g[i] = fmaf(pre_rstd, fmaf(-x[e], along, d[i]), g[i]);
        }
      }
    }
    if (a.dresidual) {
      float f[kElems];
#pragma unroll
      for (int i = 0; i < kElems; ++i) f[i] = a.residual_scale * g[i];
      put(a.dresidual, row, f);
    }
    // a token's gate, or 1
    float gate1 = 1.f, slope1 = 1.f;
    if (form == QMOE_GATE_TOKEN) {
      float one[1];
      load_either<T, 1>(a.gate, a.gate_fp32, row * a.ldgate, one);
      gate1 = gate_parts(a, one[0], &slope1);
    }
    const bool summed = post || (form == QMOE_GATE_TOKEN && a.dgate);
    float s = 0.f;
    // from here on g holds d, but for a token's gate
    if (per_channel || form == QMOE_GATE_FULL) {
      float dg[kElems];
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        float f[VEC], w[VEC], y[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[e] = 1.f;
        if (post) vector(kPost, k, w);
        if (per_channel) {  // (its slope is one for all tokens: norm_sums_kernel multiplies by it)
          vector(kGate, k, f);
        } else {
          if (full_t) {
            chunk(GATED ? 4 : 0, k, f);
          } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[e] = 0.f;
            if (in[k]) load_either<T, VEC>(a.gate, true, row * a.ldgate + col[k], f);
          }
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            float slope;
            f[e] = gate_parts(a, f[e], &slope);
            w[e] *= slope;
          }
        }
        chunk(3, k, y);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int i = k * VEC + e;
          dg[i] = g[i] * (y[e] * rstd) * w[e];
          g[i] *= f[e];
        }
        if (per_channel) {
          float p[VEC];
#pragma unroll
          for (int e = 0; e < VEC; ++e) p[e] = dg[k * VEC + e];
          add(GATED ? kGate : 0, k, p);
        }
      }
      if (form == QMOE_GATE_FULL && a.dgate) put(a.dgate, row, dg, a.dgate_fp32 != 0);
    }
    if (summed) {
      const float by = GATED ? gate1 : 1.f;
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        float y[VEC], w[VEC], p[VEC];
        chunk(3, k, y);
#pragma unroll
        for (int e = 0; e < VEC; ++e) p[e] = g[k * VEC + e] * (y[e] * rstd);
        if (post) {
          vector(kPost, k, w);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            s = fmaf(p[e], w[e], s);
            p[e] *= by;
          }
          add(kPost, k, p);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) s += p[e];
        }
      }
      s = row_sum(s);
    }
    if (form == QMOE_GATE_TOKEN && a.dgate && tid == 0)
      reinterpret_cast<float*>(a.dgate)[row] = s * slope1;
    if (GATED) {
#pragma unroll
      for (int i = 0; i < kElems; ++i) g[i] *= gate1;
    }
    if (post) {
      const float along = rstd * s * gate1 * per;
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        float w[VEC], y[VEC];
        vector(kPost, k, w);
        chunk(3, k, y);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int i = k * VEC + e;
          g[i] = rstd * fmaf(g[i], w[e], -(y[e] * along));
        }
      }
    }
    put(a.dy, row, g);
    first = false;
  }
  if constexpr (ACC) {
    const bool want[3] = {post && a.dpost_weight != nullptr, pre && a.dpre_weight != nullptr,
                          per_channel && a.dgate != nullptr};
#pragma unroll
    for (int w = 0; w < (GATED ? 3 : 2); ++w) {
      if (!want[w]) continue;
#pragma unroll
      for (int i = 0; i < kElems; ++i)
        if (in[i / VEC]) acc_rows[(size_t)w * a.H + col[i / VEC] + i % VEC] = acc[w][i];
    }
  }
}

// dst[h] = sum over the units of their sum number `which`, 32 columns a CTA, a warp every kSumWarps
// units (few columns have few CTAs, so many units have many warps).  A channel's gate: times its
// slope.
template <class T, int kSumWarps>
__global__ void __launch_bounds__(kSumWarps * 32) norm_sums_kernel(const NormArgs a) {
  __shared__ float part[kSumWarps][32];
  const int which = blockIdx.y, H = a.H;
  const bool channel = a.gate && a.gate_form == QMOE_GATE_CHANNEL;
  float* dst = which == kPost  ? (a.post_weight ? a.dpost_weight : nullptr)
               : which == kPre ? (a.pre_weight ? a.dpre_weight : nullptr)
                               : (channel ? reinterpret_cast<float*>(a.dgate) : nullptr);
  grid_dep_wait();
  if (!dst) return;
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int h = blockIdx.x * 32 + lane;
  float s = 0.f, gate[1] = {0.f}, slope = 1.f;
  if (h < H) {
    if (which == kGate && slice == 0) load_either<T, 1>(a.gate, a.gate_fp32, h, gate);
    const float* src = a.partial + (size_t)which * H + h;
#pragma unroll 8
    for (int u = slice; u < a.units; u += kSumWarps) s += src[(size_t)u * 3 * H];
  }
  part[slice][lane] = s;
  __syncthreads();
  if (slice != 0 || h >= H) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < kSumWarps; ++i) s += part[i][lane];
  if (which == kGate) gate_parts(a, gate[0], &slope);
  dst[h] = s * slope;
}

template <class T>
cudaError_t sums(const NormArgs& a, cudaStream_t stream) {
  const bool wide = a.units > 256;
  return launch_pdl(wide ? norm_sums_kernel<T, 32> : norm_sums_kernel<T, 8>, dim3((a.H + 31) / 32, 3),
                    wide ? 1024 : 256, 0, stream, a);
}

template <class T, int VEC, int ELEMS, bool ACC, In HOW, bool GATED>
cudaError_t run(NormArgs a, cudaStream_t stream) {
  a.threads = norm_threads(a.H, VEC, ELEMS);
  const int rows = norm_rows(a.threads), threads = a.threads * rows;
  auto* k = norm_backward_kernel<T, VEC, ELEMS / VEC, ACC, HOW, GATED>;
  size_t smem = 0;
  if (ACC) {
    smem = (size_t)vector_bytes(a.vectors, ELEMS) * threads;
    if (HOW != In::kDirect)
      smem += (size_t)a.depth * stage_bytes<T, VEC, HOW>(a.mats, a.threads, rows, ELEMS, a.H);
    const cudaError_t e = allow_smem(k, kNormRingBytes);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(k, dim3((a.units + rows - 1) / rows), threads, smem, stream, a);
}

template <class T, int VEC, bool GATED>
cudaError_t of_length(NormArgs a, cudaStream_t stream) {
  constexpr int kWide = 16 / (int)sizeof(T);
  if (a.H > kNormRegisterColumns) {
    constexpr int V = VEC == kWide ? VEC : 1;
    return a.H <= 16384 ? run<T, V, 16, false, In::kDirect, true>(a, stream)
                        : run<T, V, 64, false, In::kDirect, true>(a, stream);
  }
  // (single elements cost so many more instructions that eight a thread are enough)
  constexpr int kElems = VEC == 1 ? 8 : 16;
  constexpr In kHow = VEC * sizeof(T) >= 4 ? In::kOwn : In::kShared;
  const int row_threads = norm_threads(a.H, VEC, kElems), rows = norm_rows(row_threads);
  const int left = kNormRingBytes - vector_bytes(a.vectors, kElems) * row_threads * rows;
  a.depth = left / stage_bytes<T, VEC, kHow>(a.mats, row_threads, rows, kElems, a.H);
  if (a.depth > 4) a.depth = 4;
  if (a.depth >= 2) return run<T, VEC, kElems, true, kHow, GATED>(a, stream);
  // (the longest rows of fp32)
  if constexpr (sizeof(T) == 4) return run<T, VEC, kElems, true, In::kDirect, GATED>(a, stream);
  return cudaErrorInvalidValue;
}

template <class T, int VEC>
cudaError_t of_gate(const NormArgs& a, cudaStream_t stream) {
  return a.gate ? of_length<T, VEC, true>(a, stream) : of_length<T, VEC, false>(a, stream);
}

template <class T>
cudaError_t of_chunk(const NormArgs& a, int chunk, cudaStream_t stream) {
  constexpr int kWide = 16 / (int)sizeof(T);
  if (chunk == kWide) return of_gate<T, kWide>(a, stream);
  if constexpr (sizeof(T) == 2)
    if (chunk >= 2) return of_gate<T, 2>(a, stream);
  return of_gate<T, 1>(a, stream);
}

}  // namespace

int norm_units(int M, int H) {
  // as many rows in the making as 512 threads an SM have, a thread sixteen elements; and two rows a
  // unit or more, whose sums are written and read again, where that leaves every SM one (of the
  // shortest rows fewer: there the sums of the units are what takes time)
  const int threads = norm_threads(H < kNormRegisterColumns ? H : kNormRegisterColumns, 8, 16);
  const int most = 152 * (threads >= 512 ? 1 : threads >= 64 ? 512 / threads : 8);
  const int two = (M + 1) / 2, least = M < 152 ? M : 152;
  const int n = two > least ? two : least;
  return n < most ? n : most;
}

cudaError_t launch_norm_backward(const NormArgs& args, int dtype, int chunk, cudaStream_t stream) {
  NormArgs a = args;
  const bool full = a.gate && a.gate_form == QMOE_GATE_FULL && !a.gate_fp32;
  const bool need_y = a.post_weight || (a.gate && a.dgate) || (a.pre_weight && !a.out_in);
  a.mats = (a.dout != nullptr) + (a.pre_weight != nullptr) +
           (a.pre_weight != nullptr && a.out_in != nullptr) + need_y + full;
  a.vectors = (a.post_weight != nullptr) + (a.pre_weight != nullptr) +
              (a.gate && a.gate_form == QMOE_GATE_CHANNEL);
  cudaError_t e = dtype == QMOE_DTYPE_BF16   ? of_chunk<__nv_bfloat16>(a, chunk, stream)
                  : dtype == QMOE_DTYPE_FP16 ? of_chunk<__half>(a, chunk, stream)
                                             : of_chunk<float>(a, chunk, stream);
  if (e != cudaSuccess) return e;
  const bool gate = a.gate && a.gate_form == QMOE_GATE_CHANNEL && a.dgate;
  if (!gate && !(a.post_weight && a.dpost_weight) && !(a.pre_weight && a.dpre_weight))
    return cudaSuccess;
  return dtype == QMOE_DTYPE_BF16   ? sums<__nv_bfloat16>(a, stream)
         : dtype == QMOE_DTYPE_FP16 ? sums<__half>(a, stream)
                                    : sums<float>(a, stream);
}

}  // namespace qmoe
