// The 8-bit product's tiles without a GPU.
//   no arguments: every address a tile's loads make, for every number of rows a tile
//     can have left: the scalar part lies in the buffer, and a lane reads the element it
//     stands for, or (its row or column being none) reads nothing that is used: a
//     repeated row or step, or bytes behind the buffer's end.
//   T rows cols ...: prints for each three the kernel's choice, -1 for the one of few
//     tokens, else the tile's index, and its steps under way.
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "../../expert_cache_host_amd/csrc/q8_tiles.hpp"

static long long checked = 0;

static void require(bool ok, const char *what, const int (&at)[7]) {
  if (ok) return;
  std::printf("%s: waves %d loads %d rows %d ld %d cols %d step %d load %d\n", what, at[0], at[1], at[2], at[3], at[4],
              at[5], at[6]);
  std::exit(1);
}

// An operand of which a tile has `span` rows, loaded by `waves` waves; `bytes` of a row are there.
static void operand(int span, int waves, int ahead, int rows, int ld, int cols, int bytes) {
  const int loads = span / 8 / waves, steps = moe::q8_steps(cols), end = moe::q8_buffer_bytes(rows, ld, bytes);
  const int last = steps > ahead ? steps : ahead;
  for (int step = 0; step < last; ++step) {
    if (step > 2 * ahead && step < steps - 3) continue;
    for (int j = 0; j < loads; ++j) {
      const int at[7] = {waves, loads, rows, ld, cols, step, j};
      const int scalar = moe::q8_load_at(j, waves, rows, ld) + moe::q8_step_at(step, cols);
      require(scalar >= 0 && scalar < end, "the scalar offset leaves the buffer", at);
      for (int wave = 0; wave < waves; ++wave)
        for (int lane = 0; lane < 64; ++lane) {
          const int part = moe::q8_lane_at(lane, wave, ld), from = part + scalar;
          require(part >= 0 && from % 16 == 0, "a lane's part", at);
          require(from + 16 <= end || from >= end, "a load cut by the buffer's end", at);
          const int row = 8 * waves * j + 8 * wave + lane / 8;
          if (row >= rows || step >= steps) continue;
          const int piece = (lane % 8) ^ (row / 2 % 8), col = 128 * step + 16 * piece;
          require(from == row * ld + col, "another element's address", at);
          ++checked;
        }
    }
  }
}

int main(int argc, char **argv) {
  if (argc > 1) {
    for (int i = 1; i + 2 < argc; i += 3) {
      const int T = std::atoi(argv[i]), rows = std::atoi(argv[i + 1]), cols = std::atoi(argv[i + 2]);
      const int t = moe::q8_few(T, rows) ? -1 : moe::q8_best_tile(T, rows, cols);
      std::printf("%d %d\n", t, t < 0 ? 0 : moe::kQ8Tiles[t].ahead);
    }
    return 0;
  }
  const int cols_of[] = {1, 16, 100, 127, 128, 129, 256, 384, 500, 640, 769, 1300, 131072};
  for (const moe::Q8Tile &c : moe::kQ8Tiles) {
    const int waves = c.row_waves * c.token_waves;
    for (int cols : cols_of) {
      const int b16 = (cols + 15) / 16 * 16, b128 = moe::q8_steps(cols) * 128;
      for (int span : {c.rows, c.tokens})
        for (int rows = 1; rows <= span; rows += (rows < 70 || rows > span - 3 ? 1 : 7))
          for (int bytes : {b16, b128})
            for (int ld : {bytes, bytes + 48, 1 << 22}) operand(span, waves, c.ahead, rows, ld, cols, bytes);
    }
  }
  std::printf("%lld loads\nok\n", checked);
}
