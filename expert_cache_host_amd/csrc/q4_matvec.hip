// A few tokens times a matrix held in 4 bits:
//
//   out[t][r] = sum_g s[r][g] * sum_{c in group g} (q[r][c] - 8) * x[t][c]
//
// Bound by reading the weights (0.56 bytes each at group 32).  On the vector
// units a weight would cost one fused multiply-add per token beside its
// decoding, more than the memory rate leaves room for; so the products go to
// the matrix cores: B = 16 rows' codes of a block (exact binary16 integers), A =
// the tokens as binary16 rows.  A float32 token takes two rows (hi and lo part,
// 22 bits), a half-width one takes one; the power of two that brings a token's
// largest element of a wave's K slice to [2^13, 2^14) keeps the precision
// independent of the input's magnitude.  Each group's sum is exact to float32
// and its scale is applied in float32.
//
// A workgroup owns all of K: wave w holds the tokens' slice of KT chunks of 128
// columns in registers for the whole launch and streams its slice of 16 rows
// after 16 rows, the next tile's loads in flight while the present one is
// multiplied; the waves' sums meet in LDS, a barrier per tile.  K beyond 6144
// columns takes passes, the tokens laid out again for each.
//
// Measured (GPU time, inputs past the last-level cache): one float32 token, 131072 x
// 2048: 34 us, 4.45 TB/s (a large copy reaches 5.1); 8192 x 2816: 6.5 us, of which
// the weights need 2.6; four bfloat16 tokens, 10240 x 6144: 15.5 us, where twelve
// waves a CU wait for loads half of their time.
#include <algorithm>

#include "device_types.hpp"
#include "q4_tile.hpp"

namespace moe {

namespace {

constexpr int kMaxWaves = 16;

// Row of A that token part u = t * PL + p takes: parts 0..3 in the first C
// register of the four lane rows, 4..7 in the second, and so on, so that few
// tokens need few scaled adds.
__device__ __forceinline__ int part_of_row(int m) { return 4 * (m & 3) + (m >> 2); }

// Binary16 parts of a token.
constexpr int parts_of(int type) { return type == kF32 ? 2 : 1; }

// TY: element type; KT: chunks of 4 blocks per wave and pass; FI: C registers in
// use (4 FI parts).
template <int TY, int KT, int FI>
struct Matvec {
  static constexpr int PL = parts_of(TY);
  const Q4MatvecArgs &a;
  const int lane, n, g, wave, waves, nb, t0, parts;
  half8_t X[KT * 4];  // the lane's part, 8 K slots of every block
  float xs[FI];       // 2^e of the parts in this lane's C registers

  __device__ Matvec(const Q4MatvecArgs &args, int first_token)
      : a(args), lane(threadIdx.x & 63), n(lane & 15), g(lane >> 4), wave(threadIdx.x >> 6),
        waves(blockDim.x >> 6), nb(args.cols / 32), t0(first_token),
        parts(min(args.T - first_token, 4 * FI / PL) * PL) {}

  // Word gg of a block of token t, in the codes' order; zeros unless `live`.  The
  // load is from a valid place either way: a branch around it would make the
  // loads wait for each other.
  __device__ __forceinline__ void load_unit(bool live, int t, int block, int gg, float (&v)[8]) const {
    const long long i = (long long)min(t, a.T - 1) * a.ldx + min(block, nb - 1) * 32 + 4 * gg;
    const float4 p = load4(a.x, TY, i), q = load4(a.x, TY, i + 16);
    unit_order(p, q, v);
    live = live && block < nb;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = live ? v[j] : 0.f;
  }

  // The wave's K slice of every token into X and xs; `first` is its first block.
  // Many parts: every lane converts the units of its own row of A.  The slice is
  // read twice (its largest element, then the parts), which holds no more
  // registers than X.  Binary16 tokens are taken as they are.
  __device__ __forceinline__ void stage_many(int first) {
    const int u = part_of_row(n), t = t0 + u / PL, p = u % PL;
    const bool mine = u < parts;
    if constexpr (TY == kF16) {
#pragma unroll
      for (int b = 0; b < KT * 4; ++b) {
        float v[8];
        load_unit(mine, t, first + b, g, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) X[b][j] = (_Float16)v[j];
      }
#pragma unroll
      for (int i = 0; i < FI; ++i) xs[i] = 1.f;
      return;
    }
    uint32_t top = 0;
#pragma unroll
    for (int b = 0; b < KT * 4; ++b) {
      float v[8];
      load_unit(mine, t, first + b, g, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, __builtin_bit_cast(uint32_t, v[j]) & 0x7fffffffu);
    }
    const int e = scale_exp(rows_max_u32(top));
    const float f = exp2_int(-e);
#pragma unroll
    for (int b = 0; b < KT * 4; ++b) {
      float v[8];
      load_unit(mine, t, first + b, g, v);
      _Float16 hi[8], lo[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) split_half(v[j] * f, hi[j], lo[j]);
#pragma unroll
      for (int j = 0; j < 8; ++j) X[b][j] = PL == 2 && p == 1 ? lo[j] : hi[j];
    }
    // part 4 i + g stands in row 4 g + i of A, so lane n = 4 g + i knows its exponent
#pragma unroll
    for (int i = 0; i < FI; ++i) xs[i] = exp2_int(__shfl(e, 4 * g + i));
  }

  // Up to four parts: a lane converts one unit (word g' of block b') of each
  // token, and the wave shares them through its own LDS, where a lane then reads
  // the units of its row of A.
  // (All tokens' loads go out together, and ahead of the weights': loads return in
  // order.)
  __device__ __forceinline__ void load_few(int first, float (&x)[4 / PL][8]) const {
#pragma unroll
    for (int t = 0; t < 4 / PL; ++t)
      load_unit(lane < KT * 16, t0 + t, first + (lane >> 2), lane & 3, x[t]);
  }
  __device__ __forceinline__ void stage_few(const float (&xt)[4 / PL][8], uint4 (*buf)[KT * 16 + 4]) {
    const int b = lane >> 2, u = part_of_row(n);
    xs[0] = 1.f;
#pragma unroll
    for (int t = 0; t < 4 / PL; ++t) {
      if (t * PL >= parts) break;
      const float(&v)[8] = xt[t];
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, __builtin_bit_cast(uint32_t, v[j]) & 0x7fffffffu);
      const int e = TY == kF16 ? 0 : scale_exp(wave_max_u32(top));
      const float f = exp2_int(-e);
      half8_t hi, lo;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        _Float16 x, y;
        split_half(v[j] * f, x, y);
        hi[j] = x, lo[j] = y;
      }
      if (b < KT * 4) {
        buf[t * PL][lane] = __builtin_bit_cast(uint4, hi);
        if constexpr (PL == 2) buf[t * PL + 1][lane] = __builtin_bit_cast(uint4, lo);
      }
      if (g / PL == t) xs[0] = exp2_int(e);  // C's one register in row g: part g
    }
    wave_lds_order();  // the units are read by the wave that wrote them
#pragma unroll
    for (int k = 0; k < KT * 4; ++k) {
      uint4 r = make_uint4(0, 0, 0, 0);
      if (u < parts) r = buf[u][4 * k + g];
      X[k] = __builtin_bit_cast(half8_t, r);
    }
    wave_lds_order();  // the next pass's are written over them
  }
};

// GB: blocks per scale; RB: 0 when one pass takes all of K, else row tiles per
// visit.
template <int TY, int KT, int FI, int GB, int RB>
__global__ __launch_bounds__(KT == 4 ? 768 : 1024) void q4_matvec_kernel(Q4MatvecArgs a, int passes) {
  constexpr int PL = parts_of(TY);
  __shared__ float red[2][kMaxWaves][FI * 64];
  // FI == 1: the waves' units of x on their way to X
  __shared__ uint4 units[FI == 1 ? (KT == 4 ? 12 : kMaxWaves) : 1][4][KT * 16 + 4];
  Matvec<TY, KT, FI> m(a, (int)blockIdx.y * (4 * FI / PL));
  const int tiles = (a.rows + 15) / 16, nb = m.nb, per_pass = m.waves * KT * 4;
  uint4 w[RB > 0 ? 1 : 2][KT];
  uint32_t s[RB > 0 ? 1 : 2][KT];
  const CodeBits bits;
  // the wave's KT chunks of tile `tile`; blocks and rows past the end re-read a
  // valid place (their scale, or their row's output, is dropped)
  auto load = [&](int tile, int first, uint4 (&ww)[KT], uint32_t (&ss)[KT]) {
    const long long row = min(tile * 16 + m.n, a.rows - 1);
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const int b = first + 4 * k + m.g, bb = min(b, nb - 1);
      ww[k] = *(const uint4 *)(a.q + (row * nb + bb) * 16);
      const uint32_t sc = a.scales[row * (nb / GB) + bb / GB];
      ss[k] = b < nb ? sc : 0u;
    }
  };
  auto multiply = [&](const uint4 (&ww)[KT], const uint32_t (&ss)[KT], float (&acc)[FI]) {
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const uint4 t = transpose_rows(ww[k]);
      const uint4 sg = gather_rows(ss[k]);
      const uint32_t tw[4] = {t.x, t.y, t.z, t.w}, sw[4] = {sg.x, sg.y, sg.z, sg.w};
#pragma unroll
      for (int b = 0; b < 4; b += GB) {
        floatx4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < GB; ++j)
          c = __builtin_amdgcn_mfma_f32_16x16x32_f16(m.X[4 * k + b + j], decode_word(bits, tw[b + j]), c,
                                                     0, 0, 0);
        const float d = f16_to_f32((uint16_t)sw[b]);
#pragma unroll
        for (int i = 0; i < FI; ++i) acc[i] = fmaf(d, c[i], acc[i]);
      }
    }
  };
  // the waves' sums of a tile to out
  auto finish = [&](int tile, int buf, const float (&acc)[FI]) {
#pragma unroll
    for (int i = 0; i < FI; ++i) red[buf][m.wave][i * 64 + m.lane] = acc[i];
    __syncthreads();
    const int tokens = m.parts / PL;
    for (int j = threadIdx.x; j < 16 * tokens; j += blockDim.x) {
      const int t = j >> 4, row = tile * 16 + (j & 15);
      float v = 0.f;
#pragma unroll 4
      for (int x = 0; x < m.waves; ++x)
#pragma unroll
        for (int p = 0; p < PL; ++p) {
          const int u = t * PL + p;
          v += red[buf][x][(u >> 2) * 64 + (u & 3) * 16 + (j & 15)];
        }
      if (row < a.rows) store1(a.out, TY, (long long)(m.t0 + t) * a.ldo + row, v);
    }
  };
  if constexpr (RB == 0) {
    const int first = m.wave * KT * 4;
    int tile = blockIdx.x, it = 0;
    if constexpr (FI == 1) {
      float x[4 / PL][8];
      m.load_few(first, x);
      load(tile, first, w[0], s[0]);
      m.stage_few(x, units[m.wave]);
    } else {
      load(tile, first, w[0], s[0]);
      m.stage_many(first);
    }
    for (; tile < tiles; tile += gridDim.x, ++it) {
      load(min(tile + (int)gridDim.x, tiles - 1), first, w[1], s[1]);
      float acc[FI] = {};
      multiply(w[0], s[0], acc);
#pragma unroll
      for (int i = 0; i < FI; ++i) acc[i] *= m.xs[i];
      finish(tile, it & 1, acc);
#pragma unroll
      for (int k = 0; k < KT; ++k) w[0][k] = w[1][k], s[0][k] = s[1][k];
    }
  } else {
    // more columns than one pass holds: the tokens' slices are staged again for
    // every pass and RB tiles
    int it = 0;
    for (int tile = blockIdx.x * RB; tile < tiles; tile += gridDim.x * RB) {
      float acc[RB][FI] = {};
      for (int p = 0; p < passes; ++p) {
        const int first = p * per_pass + m.wave * KT * 4;
        if constexpr (FI == 1) {
          float x[4 / PL][8];
          m.load_few(first, x);
          load(tile, first, w[0], s[0]);
          m.stage_few(x, units[m.wave]);
        } else {
          load(tile, first, w[0], s[0]);
          m.stage_many(first);
        }
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          if (r) load(min(tile + r, tiles - 1), first, w[0], s[0]);
          float part[FI] = {};
          multiply(w[0], s[0], part);
#pragma unroll
          for (int i = 0; i < FI; ++i) acc[r][i] = fmaf(part[i], m.xs[i], acc[r][i]);
        }
      }
#pragma unroll
      for (int r = 0; r < RB; ++r)
        if (tile + r < tiles) finish(tile + r, it++ & 1, acc[r]);
    }
  }
}

// Chunks of K that one pass can take: 12 waves of 4.
constexpr int kPassChunks = 48;

template <int TY, int KT, int FI, int GB>
hipError_t launch_one(const Q4MatvecArgs &a, int chunks, hipStream_t s) {
  const int tiles = (a.rows + 15) / 16, tokens = 4 * FI / parts_of(TY);
  const int gy = (a.T + tokens - 1) / tokens;
  // Each workgroup with the same number of visits, and no more of them than 12, 16
  // or 32 waves a CU make (by the chunks a wave holds; the instantiations of few
  // tokens would fit more), so that the tokens are laid out no more often than that
  // (45 x 2144 x 5003 f16: 10.8 us; with a workgroup per tile 24.5)
  auto grid = [&](int waves, int visits) {
    const int fit = std::max(1, (KT == 4 ? 12 : KT == 2 ? 16 : 32) / waves);
    const int most = std::max(1, 256 * fit / gy), each = (visits + most - 1) / most;
    return dim3((unsigned)((visits + each - 1) / each), (unsigned)gy);
  };
  if constexpr (KT == 4)
    if (chunks > kPassChunks) {
      const int passes = (chunks + kPassChunks - 1) / kPassChunks;
      const int waves = (chunks + 4 * passes - 1) / (4 * passes);
      // Four tiles a visit share the laying out of many tokens, one spreads the tiles
      // over the chip (one token, 8192 x 12288: 31 us with four, 23 with one; 16
      // float32 tokens, 8192 x 8192: 54 with four, 105 with one, though the four
      // tiles' kernels spill 22 to 40 registers); below 128 visits of four the chip
      // stands too empty for it.
      if constexpr (FI > 1)
        if ((long long)(tiles / 4) * gy >= 128)
          return launch(q4_matvec_kernel<TY, 4, FI, GB, 4>, grid(waves, (tiles + 3) / 4), waves * 64, s, a, passes);
      return launch(q4_matvec_kernel<TY, 4, FI, GB, 1>, grid(waves, tiles), waves * 64, s, a, passes);
    }
  const int waves = (chunks + KT - 1) / KT;
  return launch(q4_matvec_kernel<TY, KT, FI, GB, 0>, grid(waves, tiles), waves * 64, s, a, 1);
}

template <int TY, int KT, int FI>
hipError_t launch_group(const Q4MatvecArgs &a, int chunks, hipStream_t s) {
  if (a.group == 32) return launch_one<TY, KT, FI, 1>(a, chunks, s);
  if (a.group == 64) return launch_one<TY, KT, FI, 2>(a, chunks, s);
  return launch_one<TY, KT, FI, 4>(a, chunks, s);
}

template <int TY, int KT>
hipError_t launch_parts(const Q4MatvecArgs &a, int chunks, hipStream_t s) {
  const int parts = a.T * parts_of(TY);
  if (parts <= 4) return launch_group<TY, KT, 1>(a, chunks, s);
  if (parts <= 8) return launch_group<TY, KT, 2>(a, chunks, s);
  return launch_group<TY, KT, 4>(a, chunks, s);
}

// Chunks of K per wave: 2 up to 32 chunks (one float32 token, 131072 x 2048: 36 us
// with 2, 39 with 1, 48 with 4), 4 above.
template <int TY>
hipError_t launch_cols(const Q4MatvecArgs &a, hipStream_t s) {
  const int chunks = (a.cols / 32 + 3) / 4;
  if (chunks <= 4) return launch_parts<TY, 1>(a, chunks, s);
  if (chunks <= 32) return launch_parts<TY, 2>(a, chunks, s);
  return launch_parts<TY, 4>(a, chunks, s);
}

}  // namespace

hipError_t launch_q4_matvec(const Q4MatvecArgs &a, hipStream_t s) {
  if (a.type == kF32) return launch_cols<kF32>(a, s);
  return a.type == kBf16 ? launch_cols<kBf16>(a, s) : launch_cols<kF16>(a, s);
}

}  // namespace moe
