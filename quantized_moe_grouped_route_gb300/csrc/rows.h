// Checks of matrices of rows that the operators' C-ABI calls share.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "qmoe.h"

namespace qmoe {

inline int elem_size(int dtype) { return dtype == QMOE_DTYPE_FP32 ? 4 : 2; }

inline bool known_dtype(int dtype) { return dtype >= QMOE_DTYPE_BF16 && dtype <= QMOE_DTYPE_FP32; }

inline bool misaligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) % bytes) != 0; }

// A stride of 0 stands for the same row throughout.
inline bool bad_ld(long long ld, int width) { return ld < width && ld != 0; }

// Whether every row of `rows` (stride ld elements, length H) can move in chunks of `bytes`.
inline bool chunked(const void* rows, long long ld, int H, int es, int bytes) {
  return !misaligned(rows, bytes) && ld * es % bytes == 0 && (long long)H * es % bytes == 0;
}

inline int cuda_rc(cudaError_t e) { return e == cudaSuccess ? QMOE_OK : QMOE_ERR_CUDA; }

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// Bytes of the widest chunk (at most 16) in which every one of some matrices' rows moves.
struct Chunk {
  int bytes = 16;
  void rows(const void* p, long long ld, int H, int es) {
    while (bytes > es && !chunked(p, ld, H, es, bytes)) bytes >>= 1;
  }
};

}  // namespace qmoe
