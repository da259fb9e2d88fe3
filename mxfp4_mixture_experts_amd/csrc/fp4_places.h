// Where a wave of the tile kernel of fp4_matmul.hip finds its weights' codes.  Plain
// arithmetic, so that a host program can go over every lane's offsets.
#pragma once

namespace mxfp4 {

// A wave's weight rows from n on, of N: the first (past N: the last row, whose products
// are not stored) and how many of `most` there are from it on.
constexpr int fp4_wave_first(int n, int N) { return n < N ? n : N - 1; }
constexpr int fp4_wave_rows(int n, int N, int most) {
  return N - fp4_wave_first(n, N) < most ? N - fp4_wave_first(n, N) : most;
}

// Byte offset in the wave's rows (of KB blocks of 16 bytes) of the row that lane `lane` loads of
// piece (sub-tile, upper): rows 16 upper .. + 15 of the sub-tile's 32; past the last: the last.
constexpr int fp4_row_at(int sub_tile, int upper, int lane, int rows, int KB) {
  const int r = 32 * sub_tile + 16 * upper + (lane & 15);
  return (r < rows ? r : rows - 1) * (KB * 16);
}

// Byte offset in its row of a lane's block of stage s (eight blocks), half v (four of them); past
// the row's end (the last stage's tail, and stages asked for ahead that do not exist) the last block.
constexpr int fp4_block_at(int s, int v, int lane, int KB) {
  const int last = (KB - 1) >> 3;
  const int b = 8 * (s < last ? s : last) + 4 * v + (lane >> 4);
  return (b < KB ? b : KB - 1) * 16;
}

}  // namespace mxfp4
