// What the two SMs of a pair copy of the operands of a tile of a product (ffn_gemm.cu), in plain
// C++ for host and device.
#pragma once

#ifdef __CUDACC__
#define QMOE_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define QMOE_HOST_DEVICE inline
#endif

namespace qmoe {

// A matrix's last block of `box` rows is copied in a box of its own number of rows: rows that a copy
// has to fill in cost it several times what rows of the matrix do (1 token by boxes of 128 rows: 182 us
// a call where 512 tokens took 43).  What is left in shared memory beyond reaches rows and columns of
// the accumulator that are not written; along K zeros are filled in up to the 16 of an MMA.
QMOE_HOST_DEVICE constexpr int last_rows(int rows, int box) { return (rows + box - 1) % box + 1; }
QMOE_HOST_DEVICE constexpr int last_deep(int depth) {
  return (last_rows(depth, 64) + 15) / 16 * 16;
}

// An SM's rows of A and columns of B in every step of a tile of 256 rows x tile_n columns: where they
// begin and how many there are.  Never none of both: the leader's MMAs wait for the copies of a step
// and for nothing else, so they could go round the ring twice before a producer that copies nothing
// has seen its first stage emptied, which a wait on a parity then misses for good.  The second SM
// of a tile whose rows and columns the first has alone copies the first one's rows again (its part of
// the result is not written).
struct Share {
  int row, rows, col, cols;
};
QMOE_HOST_DEVICE int share_clamp(int left, int most) { return left < 0 ? 0 : left < most ? left : most; }
// `both`: both SMs take the same columns (of u and of g).
QMOE_HOST_DEVICE Share share_of(int M, int N, int tile_n, bool both, int tm, int tn, int rank) {
  const int half = tile_n / 2;
  Share s;
  s.row = tm * 256 + rank * 128;
  s.rows = share_clamp(M - s.row, 128);
  s.col = both ? tn * half : tn * tile_n + rank * half;
  s.cols = share_clamp(N - s.col, half);
  if (s.rows == 0 && s.cols == 0) {
    s.row = tm * 256;
    s.rows = share_clamp(M - s.row, 128);
  }
  return s;
}

}  // namespace qmoe
