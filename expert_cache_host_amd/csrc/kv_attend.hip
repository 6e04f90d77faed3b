// Attention of the new tokens over the paged 4-bit cache:
//
//   out = softmax(scale * q K^T) V over the keys a row may see: positions up to
//   its own, within `window` positions when window > 0, on valid pages; a row
//   that sees no key gets 0.
//
// One pass over the cached codes with the running maximum and sum of the
// softmax.  The rows of a tile are (new token, query head) pairs of one
// sequence and one KV head, so that a group's heads share one reading of the
// cache.  At decode the kernel is bound by reading the codes; decoding them and
// two multiply-adds per element on the vector units would take longer than the
// reading, so both products run on the matrix cores with the codes as exact
// binary16 integers:
//
//  - S^T = K q^T, 16 keys by 16 columns a block of 32 elements; a key's block
//    scale is applied to the block's sum in float32.
//  - S^T leaves a lane one column and the keys 4 g + i of a tile, which is the
//    layout the second product wants its probabilities in when its K slots are
//    those keys of two tiles: nothing is moved between lanes.
//  - O^T = V^T P^T: a value's block scale belongs to the summed index, so it is
//    multiplied into the probability (a product per key and block) before that
//    is rounded to binary16.
//
// A float32 row takes two columns of 16 (hi and lo binary16 parts of q and of
// the scaled probabilities, 22 bits), a half-width row one (11 bits).  Powers of
// two keep binary16 in range whatever the magnitudes are: the columns' for q, and
// for the scaled probabilities that of the largest value scale a wave has met so
// far, of any block.  So a product of probability and value scale is held to 2^-35
// of the largest value scale, beside its relative rounding: values whose scales
// lie more than 2^13 (float32; half-width types 2^24) below the largest of their
// KV head lose digits, which no cache of real values comes near.  (A power per
// block of 32, applied on the scales' way through LDS, was built: its registers
// spill, and it took 135 us for 104 at decode and 161 for 77 for chunks.)  The
// running maximum is raised only when a score passes it by 2^4 (the sums' common
// factor cancels).
//
// Keys are split over the waves of a workgroup and over workgroups; the parts
// are joined in LDS, and by a second kernel when there is more than one
// workgroup to a tile.
//
// Measured (GPU time): 32 sequences of 6000 to 16000 keys, 64 heads on 8 KV heads
// of 128, bfloat16: 94 us and 7 us of joining, 3.9 TB/s (a large copy reaches 5.1;
// the vector units are busy half of the time, loads are waited for a third of it);
// 3 chunks of 490 tokens, 16 heads on 8 of 256, window 1024, binary16: 77 us (80 on
// inputs past the last-level cache); 4 sequences of up to 500 keys: 7.2 us.
#include <algorithm>

#include "device_types.hpp"
#include "q4_tile.hpp"

namespace moe {

namespace {

constexpr int kWaves = 4;
constexpr float kLog2e = 1.4426950408889634f;
// Probabilities stand at 2^kHead over the running maximum's, and may rise by
// 2^kSlack before the maximum is raised: with scales below 2 a product stays
// under 2^15.
constexpr int kHead = 10;
constexpr float kSlack = 4.f;

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Columns a row takes, and rows of a tile.
constexpr int parts_of(int type) { return type == kF32 ? 2 : 1; }
constexpr int rows_of(int type) { return 16 / parts_of(type); }

// Rows of a tile of sequence s, and the 32-key steps that some row of it sees.  Of
// a sequence that begins before the tensors' first row or ends past their last,
// the rows in them are the ones counted.
struct Tile {
  int s, first, rows;  // sequence, first row of the tile in it, rows of the sequence
  int t0;              // packed row of the sequence's first token in the tensors
  long long past;      // that token's position, -1 in a hole
  int step0, steps;
};

// First packed row of sequence s in the tensors.
__device__ __forceinline__ int row_start(const KvBatch &b, int s) {
  return min(max(b.start[s], 0), b.T);
}

// First tile of sequence s when tiles of RT rows never span sequences: an upper
// bound of the tiles before it that needs no running count.
__device__ __forceinline__ long long tile_base(int start_s, int start_0, int s, int G, int RT) {
  return ((long long)start_s - start_0) * G / RT + s;
}

__device__ __forceinline__ long long position_cap(const KvAttendArgs &a) {
  return min((long long)a.b.max_pages * a.c.page_tokens, (long long)kMaxPos);
}

// Fills in a tile of sequence o.s from the sequence's rows start .. end in the
// tensors; false when the tile has no row.
__device__ __forceinline__ bool fill_tile(const KvAttendArgs &a, int G, int RT, long long tile,
                                          int start_0, int start, int end, Tile &o) {
  o.t0 = start;
  o.rows = max(end - start, 0) * G;
  o.steps = 0;
  const long long first = (tile - tile_base(start, start_0, o.s, G, RT)) * RT;
  if (first < 0 || first >= o.rows) return false;
  o.first = (int)first;
  if (o.past < 0) return true;
  const int tok0 = o.first / G, tok1 = (min(o.first + RT, o.rows) - 1) / G;
  const long long cap = position_cap(a);
  const int hi = (int)min(o.past + tok1 + 1, cap);
  const int lo = a.window > 0 ? (int)min(max(o.past + tok0 + 1 - a.window, 0ll), cap) : 0;
  o.step0 = lo / 32;
  o.steps = max(0, (hi + 31) / 32 - o.step0);
  return true;
}

// The tile with this number: a search over the batch's sequences, 64 of them a
// probe (one load's latency for up to 64 sequences, two up to 4096).
__device__ __forceinline__ bool find_tile(const KvAttendArgs &a, int G, int RT, long long tile,
                                          Tile &o) {
  const int lane = threadIdx.x & 63, start_0 = row_start(a.b, 0);
  int lo = 0, hi = a.b.n_seqs;  // the last s in [lo, hi) whose first tile is at most `tile`
  while (hi - lo > 1) {
    const int each = (hi - lo + 63) / 64, s = lo + lane * each;
    const bool before = s < hi && tile_base(row_start(a.b, min(s, hi - 1)), start_0, s, G, RT) <= tile;
    lo += (max(__popcll(__ballot(before)), 1) - 1) * each;
    hi = min(hi, lo + each);
  }
  o.s = uniform(lo);
  const int past = uniform(a.b.past[o.s]), start = uniform(row_start(a.b, o.s));
  o.past = past < 0 ? -1 : (long long)past + start - uniform(a.b.start[o.s]);
  return fill_tile(a, G, RT, tile, uniform(start_0), start, uniform(row_start(a.b, o.s + 1)), o);
}

// How tiles are cut into parts, a workgroup each.
struct Split {
  int most;  // parts of a tile at most
  int want;  // parts that would give the chip 4 workgroups to a CU
};
// Equal parts of a tile of `steps` steps, by its own length and not the page
// table's: as many as are wanted, if they leave every wave two steps, and none of
// more than 64 steps.  (A part's start and end cost about two steps, the last one
// to end sets the time: 32 sequences of 6000 to 16000 keys take 106 us with parts
// of 48, 105 with 64, 110 with 96.)
__host__ __device__ __forceinline__ long long parts_of_steps(const Split &sp, long long steps) {
  const long long by_size = (steps + 63) / 64, by_waves = (steps + 2 * kWaves - 1) / (2 * kWaves);
  const long long few = by_waves < sp.want ? by_waves : sp.want;
  const long long parts = by_size > few ? by_size : few;
  return parts < sp.most ? (parts > 1 ? parts : 1) : sp.most;
}

__device__ __forceinline__ float as_float(uint32_t v) { return __builtin_bit_cast(float, v); }
__device__ __forceinline__ uint32_t as_bits(float v) { return __builtin_bit_cast(uint32_t, v); }

// The largest and the sum of v over the four 16-lane rows, per lane n.  (The
// swaps' results are taken as integers first: a bit cast straight from an
// element of the returned pair yields element 0.)
__device__ __forceinline__ float rows_max(float v) {
  const auto a = __builtin_amdgcn_permlane32_swap(as_bits(v), as_bits(v), false, false);
  v = fmaxf(as_float(a[0]), as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane16_swap(as_bits(v), as_bits(v), false, false);
  return fmaxf(as_float(b[0]), as_float(b[1]));
}

__device__ __forceinline__ float rows_sum(float v) {
  const auto a = __builtin_amdgcn_permlane32_swap(as_bits(v), as_bits(v), false, false);
  v = as_float(a[0]) + as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane16_swap(as_bits(v), as_bits(v), false, false);
  return as_float(b[0]) + as_float(b[1]);
}

// v of the lane 8 columns away (within 16 lanes).
__device__ __forceinline__ float other_half(float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x128, 0xF, 0xF, true));
}

// Block scales of 4 keys.  Every one of a tile's 16 rows of A needs those of 4
// keys in 16 lanes each, so a lane loads its share of a step's scales once (NB
// bytes), the wave puts them into its LDS and the lanes read what they need: a
// sixteenth of the loads, and registers only while the scales are used.
template <int NB>
struct Scales {
  uint32_t w[2 * NB];
  __device__ __forceinline__ void read(const char *p) {
#pragma unroll
    for (int i = 0; i < NB / 2; ++i) {
      const uint4 v = *(const uint4 *)(p + 16 * i);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  }
  __device__ __forceinline__ float at(int key, int b) const {
    const half2_t h = __builtin_bit_cast(half2_t, w[(key * NB + b) / 2]);
    return (float)h[(key * NB + b) & 1];
  }
};

// A lane's share of a step's scales: NB / 2 of key (lane % 32) / 2 of tile lane / 32.
template <int NB>
struct Share {
  uint32_t w[NB == 8 ? 2 : 1];
  __device__ __forceinline__ void load(const uint16_t *scales, const long long (&row)[2], int lane) {
    const uint16_t *p = scales + (lane < 32 ? row[0] : row[1]) * NB + (lane & 31) * (NB / 2);
    if constexpr (NB == 2) {
      w[0] = *p;
    } else if constexpr (NB == 4) {
      w[0] = *(const uint32_t *)p;
    } else {
      const uint2 v = *(const uint2 *)p;
      w[0] = v.x, w[1] = v.y;
    }
  }
  __device__ __forceinline__ void write(char *lds, int lane) const {
    if constexpr (NB == 2)
      *(uint16_t *)(lds + lane * NB) = (uint16_t)w[0];
    else if constexpr (NB == 4)
      *(uint32_t *)(lds + lane * NB) = w[0];
    else
      *(uint2 *)(lds + lane * NB) = make_uint2(w[0], w[1]);
  }
  // Bits of the largest magnitude in it.
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = max(w[0] & 0x7fffu, (w[0] >> 16) & 0x7fffu);
    if constexpr (NB == 8) m = max(m, max(w[1] & 0x7fffu, (w[1] >> 16) & 0x7fffu));
    return m;
  }
};

template <int D, int PL>
struct Attend {
  static constexpr int NB = D / 32;
  // Half-width types take the codes as they are, with their offset of 8 summed
  // apart; float32 takes them minus 8: keys and values of either sign cancel in
  // the sums and the offset would not, which costs float32 more than a digit over a
  // few hundred keys (an error of 4.6e-6 against 1.3e-7).
  static constexpr bool kRaw = PL == 1;
  const CodeBits bits;
  __device__ __forceinline__ half8_t codes_of(uint32_t w) const {
    if constexpr (kRaw) return RawCodes::word(w);
    return decode_word(bits, w);
  }
  // What slot j of q and a score's unit are multiplied by.
  static __device__ __forceinline__ constexpr float slot(int j) { return kRaw ? RawCodes::slot(j) : 1.f; }
  static constexpr int kUnitBits = kRaw ? 24 : 0;
  static constexpr int KW = NB >= 4 ? NB / 2 : 1;  // 16-byte loads of 32 keys' codes per lane
  const KvAttendArgs &a;
  const int lane, n, g, tiles_per_page;
  const long long page_rows, head_row;  // cache rows of a page, and before the KV head's in it
  const int32_t *table;  // the sequence's pages
  int pi, off;  // the cursor: next step's first 16-key tile as page index and tile in the page
  // a step's codes and scales
  uint4 kc[KW];
  Share<NB> sk, sv;
  char *lds;  // the wave's room for a step's scales: keys', then values'
  uint32_t vc[8][NB == 8 ? 2 : 1];

  __device__ Attend(const KvAttendArgs &args, int kv_head, int s, char *room)
      : a(args), lane(threadIdx.x & 63), n(lane & 15), g(lane >> 4),
        tiles_per_page(args.c.page_tokens / 16),
        page_rows((long long)args.c.kv_heads * args.c.page_tokens),
        head_row((long long)kv_head * args.c.page_tokens), table(args.b.pages + (long long)s * args.b.max_pages), lds(room) {}

  __device__ __forceinline__ void seek(int step) {
    pi = 2 * step / tiles_per_page;
    off = 2 * step - pi * tiles_per_page;
  }
  // First cache rows of the step's two 16-key tiles (clamped to a valid place)
  // and whether the sequence has pages there; then to the next step.
  __device__ __forceinline__ void next(long long (&row)[2], bool (&ok)[2]) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int page = pi < a.b.max_pages ? uniform(table[pi]) : -1;
      ok[x] = page >= 0 && page < a.c.n_pages;
      row[x] = (ok[x] ? page : 0) * page_rows + head_row + off * 16;
      if (++off == tiles_per_page) off = 0, ++pi;
    }
  }

  // The loads take a uniform base (a tile's first row) and the lane's 32-bit
  // offset in the tile, which costs no vector instruction.
  __device__ __forceinline__ void load_k(const long long (&row)[2]) {
    if constexpr (NB == 2) {
      // a tile's codes are 512 bytes: half the lanes to a tile
      const uint8_t *p = a.c.k_q + (g < 2 ? row[0] : row[1]) * 32;
      kc[0] = *(const uint4 *)(p + (uint32_t)(n * 32 + (g & 1) * 16));
    } else {
      const uint32_t o = (uint32_t)(n * (D / 2) + g * 16);
#pragma unroll
      for (int j = 0; j < KW; ++j) {
        const uint8_t *p = a.c.k_q + row[j / (KW / 2)] * (D / 2);
        kc[j] = *(const uint4 *)(p + o + j % (KW / 2) * 64);
      }
    }
    // both scales with the keys: a step begins by sharing them, with the values'
    // codes still on their way (loads return in order)
    sk.load(a.c.k_s, row, lane);
    sv.load(a.c.v_s, row, lane);
  }

  __device__ __forceinline__ void load_v(const long long (&row)[2]) {
    const uint32_t o = (uint32_t)(g * 2 * D + n * NB);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint8_t *p = a.c.v_q + row[j >> 2] * (D / 2);
      if constexpr (NB == 2) {
        vc[j][0] = *(const uint16_t *)(p + o + (j & 3) * (D / 2));
      } else if constexpr (NB == 4) {
        vc[j][0] = *(const uint32_t *)(p + o + (j & 3) * (D / 2));
      } else {
        const uint2 v = *(const uint2 *)(p + o + (j & 3) * (D / 2));
        vc[j][0] = v.x, vc[j][1] = v.y;
      }
    }
  }

  // Scores of the step's keys less `base`, in units of `unit`, as the matrix cores
  // leave them: s[x][i] is key 4 g + i of tile x against the lane's column.
  __device__ __forceinline__ void scores(const half8_t (&Q)[NB], float base, float (&s)[2][4]) const {
    const floatx4 z = {0.f, 0.f, 0.f, 0.f};
    uint4 both = make_uint4(0, 0, 0, 0);
    if constexpr (NB == 2) both = transpose_rows(kc[0]);  // both tiles' two blocks
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      Scales<NB> ks;
      ks.read(lds + (16 * x + 4 * g) * NB * 2);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[x][i] = PL == 2 ? -0.5f * base : -base;
#pragma unroll
      for (int h = 0; h < (NB + 3) / 4; ++h) {
        uint4 t = both;
        if constexpr (NB == 2) {
          if (x) t.x = both.z, t.y = both.w;
        } else {
          t = transpose_rows(kc[x * (KW / 2) + h]);
        }
        const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
        for (int k = 0; k < (NB == 2 ? 2 : 4); ++k) {
          const int b = h * 4 + k;
          // raw: -8 times the block's sum of q, which the codes' offset takes away
          floatx4 c = z;
          if constexpr (kRaw)
            c = __builtin_amdgcn_mfma_f32_16x16x32_f16(RawCodes::minus_eight(), Q[b], z, 0, 0, 0);
          c = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes_of(w[k]), Q[b], c, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[x][i] = fmaf(ks.at(i, b), c[i], s[x][i]);
        }
      }
    }
    if constexpr (PL == 2) {
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[x][i] += other_half(s[x][i]);
    }
  }

  // Binary16 products p0 s0 and p1 s1, each rounded once: a mixed multiply-add
  // per product takes the scale as binary16.  (The first half is made opaque,
  // else the compiler converts scales and products one by one: 5 instructions
  // a pair in place of 2.)
  static __device__ __forceinline__ half2_t scaled(float p0, float s0, float p1, float s1) {
    _Float16 x = (_Float16)fmaf(p0, s0, 0.f);
    asm("" : "+v"(x));
    return half2_t{x, (_Float16)fmaf(p1, s1, 0.f)};
  }

  // O += V^T P^T for the step's probabilities p (key j of K slot j); with raw codes
  // off[b] sums what their offset of 8 multiplies.
  // Half-width types take one binary16 part of p times the scale.  Relative error
  // against binary64 (root mean square), where float32 products rounded at the end
  // have 1.66e-3 (bfloat16, 32 sequences of ~12000 keys) and 2.08e-4 (binary16, 3
  // chunks of 490): 1.67e-3 and 2.55e-4, less than the output's own half step.  A
  // pair of parts was measured: as float32 products, but 118 us for 104 and 92 for 77.
  __device__ __forceinline__ void weigh(const float (&p)[8], floatx4 (&O)[2 * NB],
                                        float (&off)[NB]) const {
    const uint32_t lo_part = PL == 2 && n >= 8 ? 0xffffffffu : 0u;
    Scales<NB> vs[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) vs[x].read(lds + 64 * NB + (16 * x + 4 * g) * NB * 2);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      half2_t P[4];
      uint32_t A[2][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const Scales<NB> &sc = vs[j >> 1];
        const int k = 2 * (j & 1);
        const float s0 = sc.at(k, b), s1 = sc.at(k + 1, b);
        half2_t h = scaled(p[2 * j], s0, p[2 * j + 1], s1);
        if constexpr (PL == 2) {
          // the second part's columns hold what the first part's rounding left.
          // The compiler may round the product in two ways for two uses (once
          // or twice), which would lose a whole step: the register is fixed first.
          uint32_t bits = __builtin_bit_cast(uint32_t, h);
          asm("" : "+v"(bits));
          h = __builtin_bit_cast(half2_t, bits);
          const half2_t l = {(_Float16)fmaf(p[2 * j], s0, -(float)h[0]),
                             (_Float16)fmaf(p[2 * j + 1], s1, -(float)h[1])};
          h = __builtin_bit_cast(half2_t, (__builtin_bit_cast(uint32_t, l) & lo_part) |
                                              (__builtin_bit_cast(uint32_t, h) & ~lo_part));
        }
        P[j] = h;
        // keys 2 j and 2 j + 1: the half of their words that holds block b
        const uint32_t w0 = vc[2 * j][b / 4], w1 = vc[2 * j + 1][b / 4];
        const uint32_t w = __builtin_amdgcn_perm(w1, w0, (b & 2) ? 0x07060302u : 0x05040100u);
        if constexpr (kRaw) {
          A[0][j] = RawCodes::low(b & 1 ? w >> 8 : w);
          A[1][j] = RawCodes::high(b & 1 ? w >> 8 : w);
          off[b] = __builtin_amdgcn_fdot2(h, half2_t{(_Float16)1.f, (_Float16)1.f}, off[b], false);
        } else {
          A[0][j] = __builtin_bit_cast(uint32_t, bits.low(b & 1 ? w >> 8 : w));
          A[1][j] = __builtin_bit_cast(uint32_t, bits.high(b & 1 ? w >> 8 : w));
        }
      }
      const half8_t B = join8(P[0], P[1], P[2], P[3]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        O[2 * b + h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
            RawCodes::join(A[h][0], A[h][1], A[h][2], A[h][3]), B, O[2 * b + h], 0, 0, 0);
    }
  }
};

template <int D, int TY>
struct Shared {
  static constexpr int RT = rows_of(TY);
  float o[kWaves][RT][D + 4];
  float ref[kWaves][RT], sum[kWaves][RT], unit[RT];
  __attribute__((aligned(16))) char scales[kWaves][128 * (D / 32)];
};

// Steps c0 .. c1 - 1 of a tile and KV head by one workgroup: to `out` when they
// are all of its steps, else as a part: RT rows of D sums in part_o; their
// references, sums of probabilities and units in part_l.
template <int D, int TY>
__device__ __forceinline__ void attend_part(const KvAttendArgs &a, int G, int kvh, const Tile &tile,
                                            int c0, int c1, float *part_o,
                                            float *part_l, Shared<D, TY> &sh) {
  constexpr int NB = D / 32, PL = parts_of(TY), RT = rows_of(TY);
  const int wave = uniform(threadIdx.x >> 6);
  Attend<D, PL> w(a, kvh, tile.s, sh.scales[wave]);
  const int n = w.n, g = w.g;

  // the lane's column: row n % RT of the tile, part n / RT of it
  const int row = tile.first + n % RT, tok = row / G, head = kvh * G + row % G;
  const long long t = (long long)tile.t0 + tok, past = tile.past;
  const bool live = row < tile.rows;
  const long long cap = position_cap(a);
  const int hi = live ? (int)min(past + tok + 1, cap) : 0;
  const int lo_key = a.window > 0 ? (int)min(max(past + tok + 1 - a.window, 0ll), cap) : 0;
  // keys that every row sees, and the range of the keys that some row sees
  const int tok0 = tile.first / G, tok1 = (min(tile.first + RT, tile.rows) - 1) / G;
  const int hi_max = (int)min(past + tok1 + 1, cap), hi_min = (int)min(past + tok0 + 1, cap);
  const int lo_max = a.window > 0 ? (int)min(max(past + tok1 + 1 - a.window, 0ll), cap) : 0;
  const int lo_min = a.window > 0 ? (int)min(max(past + tok0 + 1 - a.window, 0ll), cap) : 0;
  const int per = (c1 - c0 + kWaves - 1) / kWaves;
  const int i0 = min(c0 + wave * per, c1), i1 = min(i0 + per, c1);

  floatx4 O[2 * NB];
#pragma unroll
  for (int b = 0; b < 2 * NB; ++b) O[b] = floatx4{0.f, 0.f, 0.f, 0.f};
  float off[NB] = {};
  // The probabilities' reference score (in units of `unit`), what a score may pass
  // it by before it is raised (-inf before the first key), and the running sum.
  // Scores come with the reference taken off, so that an exponent is as exact as
  // their difference however large they are.
  float base = 0.f, room = -INFINITY, sum = 0.f;
  float unit = 1.f;
  int vexp = -14;                    // value scales met so far lie below 2^(vexp + 1)

  if (i0 < i1) {
    long long at[2];
    bool ok[2];
    w.seek(tile.step0 + i0);
    w.next(at, ok);
    w.load_k(at);
    w.load_v(at);

    // q: the column's elements in the codes' order, at the row's power of two
    half8_t Q[NB];
    uint32_t big = 0;
    float v[NB][8];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      if (live) {
        const long long i = t * a.ldq + head * D + b * 32 + 4 * g;
        x = load4(a.q, TY, i), y = load4(a.q, TY, i + 16);
      }
      unit_order(x, y, v[b]);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        big = max(big, __builtin_bit_cast(uint32_t, v[b][j]) & 0x7fffffffu);
    }
    big = rows_max_u32(big);
    const int e = scale_exp(big);
    // a row with an infinity or a NaN has no finite score: NaN, and not the -inf that
    // stands for unseen keys
    const float f = big >= 0x7f800000u ? __builtin_nanf("")
                    : a.scale == 0.f   ? 0.f
                    : a.scale < 0.f    ? -exp2_int(-e)
                                       : exp2_int(-e);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        _Float16 x, y;
        split_half(v[b][j] * (f * Attend<D, PL>::slot(j)), x, y);
        Q[b][j] = PL == 2 && n >= 8 ? y : x;
      }
    // a score's unit in log2: positive (a negative scale is q's sign), the raw
    // codes' 2^24 in it.  At the bounds: scores that all differ by nothing, and
    // scores of which any two that differ do so by more than an exponential tells
    // apart, with none beyond float32 (15 * 32 codes, q below 2^14, scales below
    // 2^16, NB blocks: below 2^42 units).
    unit = ldexpf(fabsf(a.scale) * kLog2e, e + Attend<D, PL>::kUnitBits);
    unit = fminf(fmaxf(unit, 1e-37f), Attend<D, PL>::kRaw ? 0x1p108f : 0x1p84f);

    for (int i = i0; i < i1; ++i) {
      const int key0 = (tile.step0 + i) * 32;
      const bool whole = ok[0] && ok[1] && key0 >= lo_max && key0 + 32 <= hi_min;
      const bool ok_now[2] = {ok[0], ok[1]};
      w.next(at, ok);  // past the last step: loaded from a valid place and not used

      if (!whole) {
        // places that no row sees, whose scales may be anything
        const int key = key0 + (w.lane >> 1);
        if (!((w.lane < 32 ? ok_now[0] : ok_now[1]) && key >= lo_min && key < hi_max)) {
          w.sv.w[0] = 0;
          if constexpr (NB == 8) w.sv.w[1] = 0;
        }
      }
      wave_lds_order();  // the last step's scales have been read
      w.sk.write(w.lds, w.lane);
      w.sv.write(w.lds + 64 * NB, w.lane);
      wave_lds_order();  // and these are read by other lanes
      const uint32_t sb = w.sv.top();
      float s[2][4];
      w.scores(Q, base, s);
      w.load_k(at);
      if (!whole) {
        // keys the row does not see
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int key = key0 + 16 * x + 4 * g + j;
            if (!(ok_now[x] && key >= lo_key && key < hi)) s[x][j] = -INFINITY;
          }
      }
      float m = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                      fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
      if (__any(m > room)) {
        const float up = rows_max(m);
        const bool first = room == -INFINITY;
        // rounded down, so that the largest score does not end below its reference
        float to = up == -INFINITY ? base : base + (first ? up : fmaxf(up, 0.f));
        if (to - base > up && to != base) to = nextafterf(to, -INFINITY);
        const float d = to - base;
        const float f = first ? 1.f : exp2f(-d * unit);
        base = to;
        if (up != -INFINITY) room = kSlack / unit;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[x][j] -= d;
            // where even the sum's rounding is more than the room, scores that
            // float32 does not tell apart count the same
            s[x][j] = s[x][j] > room ? room : s[x][j];
          }
        sum *= f;
#pragma unroll
        for (int b = 0; b < NB; ++b) off[b] *= f;
#pragma unroll
        for (int b = 0; b < 2 * NB; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) O[b][j] *= f;
      }
      if (__any((int)(sb >> 10) - 15 > vexp)) {
        const int to = max(vexp, (int)(wave_max_u32(sb) >> 10) - 15);
        const float f = exp2_int(vexp - to);
        vexp = uniform(to);
        sum *= f;
#pragma unroll
        for (int b = 0; b < NB; ++b) off[b] *= f;
#pragma unroll
        for (int b = 0; b < 2 * NB; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) O[b][j] *= f;
      }
      const float head = (float)(kHead - vexp);
      float p[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p[j] = __builtin_amdgcn_exp2f(fmaf(s[j >> 2][j & 3], unit, head));
        sum += p[j];
      }
      w.weigh(p, O, off);
      w.load_v(at);
    }
  }

  // Join the waves.  Their sums go there without the value scales' power of two, so
  // that they differ by their references alone, and those stay what they are: a
  // score beside the unit it counts in (-inf where no key was seen).  The
  // difference of two references is taken before it is multiplied by the unit: as
  // one number in log2 a reference past 2^24 would hold neither the power of two
  // nor the difference of two close scores.
  const float back = exp2_int(vexp);
  sum = rows_sum(sum) * back;
  __syncthreads();  // an earlier part's sums have been read
  if (g == 0 && n < RT) {
    sh.ref[wave][n] = sum == 0.f ? -INFINITY : base;
    sh.sum[wave][n] = sum;
    if (wave == 0) sh.unit[n] = unit;  // the same for every wave with a step, and wave 0 has one
  }
#pragma unroll
  for (int b = 0; b < 2 * NB; ++b) {
    // the sums of the raw codes (units of 2^-24, of 2^-20 for the second nibbles)
    // without their offset of 8
    if constexpr (Attend<D, PL>::kRaw) {
      const float eight = 8.f * back * rows_sum(off[b / 2]);
#pragma unroll
      for (int j = 0; j < 4; ++j) O[b][j] = fmaf(O[b][j], (b & 1 ? 0x1p20f : 0x1p24f) * back, -eight);
    }
    if constexpr (PL == 2) {
#pragma unroll
      for (int j = 0; j < 4; ++j) O[b][j] = (O[b][j] + other_half(O[b][j])) * back;
    }
    if (n < RT) *(floatx4 *)&sh.o[wave][n][b * 16 + 4 * g] = O[b];
  }
  __syncthreads();
  const bool all = c0 == 0 && c1 == tile.steps;
  for (int j = threadIdx.x; j < RT * D / 4; j += kWaves * 64) {
    const int r = j / (D / 4), d = j % (D / 4) * 4;
    const int rr = tile.first + r, tk = rr / G;
    const long long tt = (long long)tile.t0 + tk;
    if (rr >= tile.rows) continue;
    const float unit_r = sh.unit[r];
    float best = -INFINITY;
#pragma unroll
    for (int x = 0; x < kWaves; ++x) best = fmaxf(best, sh.ref[x][r]);
    float l = 0.f;
    floatx4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int x = 0; x < kWaves; ++x) {
      const float f = sh.ref[x][r] == -INFINITY ? 0.f : exp2f((sh.ref[x][r] - best) * unit_r);
      l = fmaf(f, sh.sum[x][r], l);
      const floatx4 v = *(const floatx4 *)&sh.o[x][r][d];
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = fmaf(f, v[k], o[k]);
    }
    if (all) {
      const long long to = tt * a.ldo + (kvh * G + rr % G) * D + d;
#pragma unroll
      for (int k = 0; k < 4; ++k) store1(a.out, TY, to + k, l == 0.f ? 0.f : o[k] / l);
    } else {
      *(floatx4 *)(part_o + r * D + d) = o;
      if (d == 0) part_l[r] = best, part_l[RT + r] = l, part_l[2 * RT + r] = unit_r;
    }
  }
}

// What the registers allow without spilling (at D = 128 four waves spill eight
// registers and take 121 us where three take 103: 32 sequences of ~12000 keys).
template <int D>
constexpr int waves_per_simd() { return D == 64 ? 4 : D == 128 ? 3 : 2; }

// A workgroup per tile, KV head and part.  The workspace holds RT rows of D sums
// per part, then the parts' references, sums of probabilities and units.
template <int D, int TY>
__global__ __launch_bounds__(kWaves * 64, waves_per_simd<D>()) void kv_attend_kernel(
    KvAttendArgs a, Split sp) {
  constexpr int RT = rows_of(TY);
  __shared__ Shared<D, TY> sh;
  const int G = a.q_heads / a.c.kv_heads, kvh = blockIdx.y % a.c.kv_heads, part = blockIdx.y / a.c.kv_heads;
  Tile tile;
  if (!find_tile(a, G, RT, blockIdx.x, tile)) return;
  const int parts = (int)parts_of_steps(sp, tile.steps);
  if (part >= parts) return;
  const int c0 = (int)((long long)tile.steps * part / parts);
  const int c1 = (int)((long long)tile.steps * (part + 1) / parts);
  const size_t slot = ((size_t)blockIdx.x * a.c.kv_heads + kvh) * sp.most + part;
  const size_t slots = (size_t)gridDim.x * a.c.kv_heads * sp.most;
  float *ws = (float *)a.ws;
  attend_part<D, TY>(a, G, kvh, tile, c0, c1, ws + slot * RT * D,
                     ws + slots * RT * D + slot * RT * 3, sh);
}

// Joins a tile's parts where there are several.
template <int D, int TY>
__global__ __launch_bounds__(256) void kv_join_kernel(KvAttendArgs a, Split sp) {
  constexpr int RT = rows_of(TY);
  const int G = a.q_heads / a.c.kv_heads, kvh = blockIdx.y;
  Tile tile;
  if (!find_tile(a, G, RT, blockIdx.x, tile)) return;
  const int parts = (int)parts_of_steps(sp, tile.steps);
  if (parts < 2) return;
  const size_t slot = ((size_t)blockIdx.x * a.c.kv_heads + kvh) * sp.most;
  const size_t slots = (size_t)gridDim.x * a.c.kv_heads * sp.most;
  const float *o_parts = (const float *)a.ws + slot * RT * D;
  const float *l_parts = (const float *)a.ws + slots * RT * D + slot * RT * 3;
  for (int j = threadIdx.x; j < RT * D / 4; j += 256) {
    const int r = j / (D / 4), d = j % (D / 4) * 4;
    const int rr = tile.first + r;
    const long long tt = (long long)tile.t0 + rr / G;
    if (rr >= tile.rows) continue;
    const float unit = l_parts[2 * RT + r];  // the same in every part
    float best = -INFINITY;
#pragma unroll 8
    for (int x = 0; x < parts; ++x) best = fmaxf(best, l_parts[x * RT * 3 + r]);
    float l = 0.f;
    floatx4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int x = 0; x < parts; ++x) {
      const float ref = l_parts[x * RT * 3 + r];
      const float f = ref == -INFINITY ? 0.f : exp2f((ref - best) * unit);
      l = fmaf(f, l_parts[x * RT * 3 + RT + r], l);
      const floatx4 v = *(const floatx4 *)(o_parts + ((size_t)x * RT + r) * D + d);
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = fmaf(f, v[k], o[k]);
    }
    const long long to = tt * a.ldo + (kvh * G + rr % G) * D + d;
#pragma unroll
    for (int k = 0; k < 4; ++k) store1(a.out, TY, to + k, l == 0.f ? 0.f : o[k] / l);
  }
}

long long tiles_bound(const KvCache &c, const KvBatch &b, int type, int q_heads) {
  return (long long)b.T * (q_heads / c.kv_heads) / rows_of(type) + b.n_seqs;
}

// The lengths are on the device; here the page table bounds them.  At most 64
// parts a tile and 8192 in all: that bounds the workspace (68 MB at D = 128) where
// a long prompt's tiles fill the chip many times over by themselves, and the
// workgroups that find no part to do where the table is much longer than the
// sequences.
Split split_of(const KvCache &c, const KvBatch &b, int type, int q_heads, int window) {
  const long long groups = tiles_bound(c, b, type, q_heads) * c.kv_heads;
  long long len = (long long)b.max_pages * c.page_tokens;
  // a tile of RT rows spans at most RT tokens beside the window
  if (window > 0 && window + 16ll < len) len = window + 16ll;
  Split sp;
  sp.want = (int)((1024 + groups - 1) / groups);
  sp.most = (int)std::min(64ll, std::max(1ll, 8192 / groups));
  sp.most = (int)parts_of_steps(sp, len / 32 + 2);
  return sp;
}

template <int D, int TY>
hipError_t launch_one(const KvAttendArgs &a, hipStream_t s) {
  const Split sp = split_of(a.c, a.b, a.type, a.q_heads, a.window);
  const unsigned tiles = (unsigned)tiles_bound(a.c, a.b, a.type, a.q_heads);
  const hipError_t e = launch(kv_attend_kernel<D, TY>, dim3(tiles, (unsigned)(a.c.kv_heads * sp.most)),
                              kWaves * 64, s, a, sp);
  if (e != hipSuccess || sp.most == 1) return e;
  return launch(kv_join_kernel<D, TY>, dim3(tiles, (unsigned)a.c.kv_heads), 256, s, a, sp);
}

template <int TY>
hipError_t launch_dim(const KvAttendArgs &a, hipStream_t s) {
  if (a.c.head_dim == 64) return launch_one<64, TY>(a, s);
  if (a.c.head_dim == 128) return launch_one<128, TY>(a, s);
  return launch_one<256, TY>(a, s);
}

}  // namespace

size_t kv_attend_ws_bytes(const KvCache &c, const KvBatch &b, int type, int q_heads, int window) {
  const int most = split_of(c, b, type, q_heads, window).most;
  if (most == 1) return 0;
  return (size_t)tiles_bound(c, b, type, q_heads) * c.kv_heads * most * rows_of(type) *
         (c.head_dim + 3) * sizeof(float);
}

hipError_t launch_kv_attend(const KvAttendArgs &a, hipStream_t s) {
  if (a.b.T == 0) return hipSuccess;
  if (a.type == kF32) return launch_dim<kF32>(a, s);
  return a.type == kBf16 ? launch_dim<kBf16>(a, s) : launch_dim<kF16>(a, s);
}

}  // namespace moe
