// The shares of a pair's SMs of a tile (ffn_tiles.h): over many sizes they cover the operands, fit
// their boxes, and are never both empty.
#include <cstdio>
#include <initializer_list>

#include "ffn_tiles.h"

using qmoe::Share;

int main() {
  int bad = 0;
  auto check = [&](bool ok, const char* what, int M, int N, int tile_n, int tm, int tn) {
    if (ok) return;
    if (++bad <= 20) std::printf("%s: M %d N %d tile_n %d tile %d %d\n", what, M, N, tile_n, tm, tn);
  };
  const int rows[] = {1, 8, 17, 127, 128, 129, 136, 255, 256, 257, 300, 384, 385, 512, 513, 1000, 2310};
  const int columns[] = {8, 16, 64, 72, 120, 128, 136, 192, 200, 256, 264, 320, 328, 392, 1032, 2056};
  for (int M : rows)
    for (int N : columns)
      for (int tile_n : {128, 256})
        for (bool both : {false, true}) {
          const int half = tile_n / 2, cols = both ? half : tile_n;
          for (int tm = 0; tm < (M + 255) / 256; ++tm)
            for (int tn = 0; tn < (N + cols - 1) / cols; ++tn) {
              int covered_rows = 0, covered_cols = 0;
              for (int r = 0; r < 2; ++r) {
                const Share s = qmoe::share_of(M, N, tile_n, both, tm, tn, r);
                auto is = [&](bool ok, const char* what) { check(ok, what, M, N, tile_n, tm, tn); };
                // an SM that copies nothing is no part of the handshake of a step
                is(s.rows > 0 || s.cols > 0, "an SM copies nothing");
                // in whole boxes or the edge's
                is(s.rows == 0 || s.rows == 128 || s.rows == qmoe::last_rows(M, 128), "rows of a box");
                is(s.cols == 0 || s.cols == half || s.cols == qmoe::last_rows(N, half), "columns of a box");
                is(s.rows == 0 || (s.row >= 0 && s.row % 128 == 0 && s.row + s.rows <= M), "rows");
                is(s.cols == 0 || (s.col >= 0 && s.col % half == 0 && s.col + s.cols <= N), "columns");
                // each SM has the rows and columns that its part of the result needs
                const int row = tm * 256 + r * 128, col = both ? tn * half : tn * tile_n + r * half;
                if (row < M) {
                  is(s.row == row && s.rows == (M - row < 128 ? M - row : 128), "the rows needed");
                  covered_rows += s.rows;
                }
                if (col < N) {
                  is(s.col == col && s.cols == (N - col < half ? N - col : half), "the columns needed");
                  covered_cols += s.cols;
                }
              }
              const int left_rows = M - tm * 256, left_cols = N - tn * cols;
              check(covered_rows == (left_rows < 256 ? left_rows : 256), "all rows", M, N, tile_n, tm, tn);
              check(covered_cols == (both ? 2 : 1) * (left_cols < cols ? left_cols : cols),
                    "all columns", M, N, tile_n, tm, tn);
            }
        }
  std::printf("%d failure(s)\n", bad);
  return bad != 0;
}
