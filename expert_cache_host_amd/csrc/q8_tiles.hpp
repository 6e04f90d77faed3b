// Tiles of the 8-bit product: which one a product takes, and where in an operand a
// tile's loads start.  Plain C++, so that the offsets are checked without a GPU too.
#pragma once
#include <cstdint>

namespace moe {

// Tiles (rows x tokens, waves along each, steps under way), how many fit a CU, and what a
// step of 128 columns takes on a CU, in microseconds: alone, and with as many workgroups
// as fit; `tile` is a tile's start and end.  Fitted to 48 products of 65 to 4096 tokens,
// 200 to 12288 columns and 64 to 32768 rows (matrices out of the cache), of which the
// estimate's choice took 1.03 of the best tile's time in the mean and 1.17 at most; one
// tile of 256 x 256 for all took 1.9 and 4.8.  The sizes are those that a sweep of these
// products kept: each is the best in 3 to 11 of them (160 x 128 in 11: without it they
// take 1.5 % more, one 18 %; 192 x 128 in the same waves is slower in 10 of the 11, up
// to 1.4 times).
struct Q8Tile {
  int rows, tokens, row_waves, token_waves, ahead, fit;
  float tile, alone, shared;
};
constexpr Q8Tile kQ8Tiles[] = {
    {256, 256, 2, 4, 2, 1, 9.6f, 1.11f, 1.11f}, {160, 128, 1, 4, 2, 2, 6.0f, 0.49f, 1.32f},
    {128, 128, 2, 2, 2, 2, 5.5f, 0.43f, 1.08f}, {96, 128, 1, 4, 4, 1, 4.0f, 0.39f, 0.39f},
    {64, 64, 2, 2, 4, 2, 2.0f, 0.21f, 0.44f},   {32, 64, 1, 2, 6, 2, 1.8f, 0.19f, 0.28f},
    {64, 32, 2, 1, 4, 3, 1.1f, 0.17f, 0.49f},
};
constexpr int kQ8TileCount = (int)(sizeof kQ8Tiles / sizeof *kQ8Tiles);

// Few tokens and rows: too few tiles of 64 or 32 rows to keep the CUs' loads under way,
// so that 8 waves share a tile's columns.  One token, 2816 and 6144 columns, 4096 rows:
// 6.8 and 8.4 us (tiles of 64 x 32 take 8.5 and 12.8); 8192 rows: 6.9 and 12.1 (8.2 and
// 13.4); 16384 rows: 11.7 and 22.0 (10.9 and 19.8).
constexpr bool q8_few(int T, int rows) { return T <= (rows <= 4096 ? 32 : 16) && rows < 10240; }

constexpr int q8_steps(int cols) { return (cols + 127) / 128; }

inline int q8_best_tile(int T, int rows, int cols) {
  int best = 0;
  double least = 1e30;
  for (int i = 0; i < kQ8TileCount; ++i) {
    const Q8Tile &c = kQ8Tiles[i];
    const int64_t tiles = (int64_t)((rows + c.rows - 1) / c.rows) * ((T + c.tokens - 1) / c.tokens);
    if (tiles >= 1 << 22) continue;  // a grid holds fewer than 2^32 threads
    const int64_t n = (tiles + 255) / 256, steps = q8_steps(cols);  // tiles a CU
    const double t = (double)((n + c.fit - 1) / c.fit) * c.tile +
                     (double)steps * ((double)(n / c.fit) * c.shared + (double)(n % c.fit) * c.alone);
    if (t < least) least = t, best = i;
  }
  return best;
}

// A tile's operand is a buffer from its first row to the end of its last: `rows` rows
// (those the matrix has left, or the tile's) ld bytes apart, of `bytes` bytes.
constexpr int q8_buffer_bytes(int rows, int ld, int bytes) { return (rows - 1) * ld + bytes; }

// A load's address in it is the sum of a lane's part, a load's and a step's.  The last
// two go to the instruction as its scalar offset, which alone never leaves the buffer:
// loads behind the last row repeat the last ones, steps past the last column the last
// step (neither is used).  So only the lane's part can, for which the buffer reads 0.
//
// A wave's load takes 8 rows of 128 bytes; the 16-byte pieces of row r lie at place
// piece ^ r / 2 % 8: sixteen lanes that read the same piece of sixteen rows then
// touch each of the 64 banks once (with r % 8 half of the LDS time was conflicts).
constexpr int q8_lane_at(int lane, int wave, int ld) {
  return ((lane >> 3) + 8 * wave) * ld + ((lane & 7) ^ ((wave & 1) * 4 + (lane >> 4))) * 16;
}
// The jth load of each of the workgroup's waves.
constexpr int q8_load_at(int j, int waves, int rows, int ld) {
  const int row = 8 * waves * j, last = (rows - 1) / (8 * waves) * (8 * waves);
  return (row < last ? row : last) * ld;
}
constexpr int q8_step_at(int step, int cols) {
  return 128 * (step < q8_steps(cols) ? step : q8_steps(cols) - 1);
}

}  // namespace moe
