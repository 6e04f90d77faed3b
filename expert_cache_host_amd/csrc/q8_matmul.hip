// out[t][r] = sx[t] sw[r] sum_c x[t][c] w[r][c] over 8-bit integers, the sums in 32
// bits on the matrix cores (v_mfma_i32_32x32x32_i8; 16x16x64 for few tokens).
//
// Many tokens (q8_tile_kernel): a workgroup takes a tile of rows by tokens, 128
// columns a step, both operands loaded straight into LDS, S steps under way.  Large
// products are bound by the card's power (the clock falls to about 1.5 GHz while the
// matrix cores are busy, 0.85 of the CUs' cycles): 4096 x 6144 x 16384 in 345 us, 2390
// TOP/s (a library's product of these sizes without scales: 395 us); 8192^3 in 440 us,
// 2500 TOP/s (the library 440).  Middle ones keep no unit busy throughout: 512 x 6144 x
// 10240 takes 37 us, a tile of 160 x 128 and one wave a SIMD on each CU, matrix cores
// 0.46 of its cycles, LDS reads 0.28, its loads coming in at about 50 GB/s.
// What mattered: fragments read a step ahead of their products and loads a step and a
// quarter ahead of their fragments (8192^3: 567 -> 472 us); pieces laid out so that
// reads meet no bank conflict; a step's loads spread over it, since LDS takes their
// writes between the reads (491 -> 441 us, and 84 -> 67 us for 80 tiles of 6144
// columns, one each on 80 CUs).
// Few tokens: memory.  24 x 6144 x 10240 in 14 us (4.5 TB/s of weights), one token
// by 2816 x 8192, its codes made on the way, in 8.1.
#include "q8_code.hpp"
#include "q8_tiles.hpp"
#include "step_ops.hpp"

namespace moe {

namespace {

using i32x4 = __attribute__((ext_vector_type(4))) int;

// (sum sx) sw, both products rounded to float32.  The value is settled there:
// a conversion to binary16 taken together with the product would round once where
// the definition rounds twice.
__device__ __forceinline__ float scaled(int sum, float sx, float sw) {
  float v = (float)sum * sx * sw;
  asm volatile("" : "+v"(v));
  return v;
}

using i32x16 = __attribute__((ext_vector_type(16))) int;

// n rows of codes from row r0 on as a buffer.
__device__ __forceinline__ i32x4 rows_from(const int8_t *p, long long ld, int r0, int n, int bytes) {
  const uint64_t base = (uint64_t)(p + (long long)r0 * ld);
  i32x4 r;
  r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)base);
  r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(base >> 32) & 0xffff);
  r[2] = __builtin_amdgcn_readfirstlane(q8_buffer_bytes(n, (int)ld, bytes));
  r[3] = 0x00027000;
  return r;
}

// 16 bytes a lane from the buffer's byte lane_at + at into LDS, the wave's kilobyte
// at place `l`; `at` lies in the buffer, a lane's byte behind its end gives 0.  Written as assembly (it returns nothing in registers) because the
// compiler waits for every such load before any read of LDS (nothing else here uses
// m0); wait_loads says which
// of them a wave waits for.
__device__ __forceinline__ void load_lds(i32x4 rows, uint32_t l, int lane_at, int at) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(l), "v"(lane_at), "s"(rows), "s"(at)
               : "memory");
}

// The first n of eight elements of a row.
__device__ __forceinline__ void store8(void *p, int type, long long i, float4 x, float4 y, int n) {
  if (n >= 8) {
    if (type == kF32) {
      store4(p, type, i, x), store4(p, type, i + 4, y);
      return;
    }
    uint32_t b[4];
    store4(b, type, 0, x), store4(b, type, 4, y);
    __builtin_memcpy((uint16_t *)p + i, b, 16);
  } else if (n >= 4) {
    store4(p, type, i, x);
    if (n > 4) store_few(p, type, i + 4, y, n - 4);
  } else {
    store_few(p, type, i, x, n);
  }
}

// This wave's loads into LDS have landed but for the last N; then the workgroup's.
template <int N>
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
  __builtin_amdgcn_sched_barrier(0);
}
// Every wave's reads of LDS so far have returned.
__device__ __forceinline__ void reads_done() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// A tile of RT rows of w by TT tokens, WR x WT waves.
template <int TY, int RT, int TT, int WR, int WT, int S>
__global__ __launch_bounds__(64 * WR * WT) void q8_tile_kernel(Q8MatmulArgs a, int r_tiles, int t_tiles) {
  constexpr int NW = WR * WT, RI = RT / WR / 32, TI = TT / WT / 32;
  constexpr int LA = RT / 8 / NW, LB = TT / 8 / NW;
  static_assert(RT % (8 * NW) == 0 && TT % (8 * NW) == 0, "whole loads");
  constexpr int kStep = (RT + TT) * 128;
  __shared__ __attribute__((aligned(1024))) int8_t lds[S * kStep];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // workgroups are dealt to the 8 dies in turn: each die takes a run of tiles
  const int n = r_tiles * t_tiles, id = blockIdx.x;
  const int per = n / 8, rest = n % 8, die = id % 8;
  int at = die * per + min(die, rest) + id / 8;
  // groups of 8 row tiles, the token tiles of a group in turn
  const int group = at / (8 * t_tiles), in = at % (8 * t_tiles), high = min(8, r_tiles - 8 * group);
  const int r0 = (8 * group + in % high) * RT, t0 = in / high * TT;
  __shared__ __attribute__((aligned(16))) float sws[RT], sxs[TT];
  for (int i = threadIdx.x; i < RT; i += 64 * NW) sws[i] = r0 + i < a.rows ? a.w_scales[r0 + i] : 0.f;
  for (int i = threadIdx.x; i < TT; i += 64 * NW) sxs[i] = t0 + i < a.T ? a.x_scales[t0 + i] : 0.f;
  const int n_rows = min(a.rows - r0, RT), n_tokens = min(a.T - t0, TT);
  const auto wr = rows_from(a.w, a.ldw, r0, n_rows, (a.cols + 15) & ~15);
  const auto xr = rows_from(a.x, a.ldx, t0, n_tokens, (a.cols + 127) & ~127);
  static_assert(NW % 2 == 0, "a wave's loads all start at rows of the same r / 8 % 2");
  const int wo = q8_lane_at(lane, wave, (int)a.ldw), xo = q8_lane_at(lane, wave, (int)a.ldx);
  int wj[LA], xj[LB];
#pragma unroll
  for (int j = 0; j < LA; ++j) wj[j] = q8_load_at(j, NW, n_rows, (int)a.ldw);
#pragma unroll
  for (int j = 0; j < LB; ++j) xj[j] = q8_load_at(j, NW, n_tokens, (int)a.ldx);
  const uint32_t lds_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) int8_t *)lds + wave * 1024;
  const auto load_w = [&](int j, int to, int k) { load_lds(wr, lds_at + to + j * NW * 1024, wo, wj[j] + k); };
  const auto load_x = [&](int j, int to, int k) {
    load_lds(xr, lds_at + to + RT * 128 + j * NW * 1024, xo, xj[j] + k);
  };
  const auto load = [&](int to, int k) {
#pragma unroll
    for (int j = 0; j < LA; ++j) load_w(j, to, k);
#pragma unroll
    for (int j = 0; j < LB; ++j) load_x(j, to, k);
  };
  const int wi = wave % WR, ti = wave / WR;
  const int ra = (wi * (RT / WR) + (lane & 31)) * 128, rb = (RT + ti * (TT / WT) + (lane & 31)) * 128;
  i32x16 acc[RI][TI] = {};
  struct Frag {
    i32x4 w[RI], x[TI];
  };
  // fragment n of step s: the tokens' first, then the rows'
  const auto read1 = [&](const int8_t *l, int s, Frag &f, int n) {
    const int c = ((2 * s + (lane >> 5)) ^ (lane >> 1 & 7)) * 16;
    if (n < TI)
      f.x[n] = *(const i32x4 *)(l + rb + c + n * 4096);
    else
      f.w[n - TI] = *(const i32x4 *)(l + ra + c + (n - TI) * 4096);
  };
  constexpr int kFrags = RI + TI;
  // products of one step, with what `between(i)` issues after those of row block i
  const auto multiply = [&](const Frag &f, auto between) {
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      between(i);
#pragma unroll
      for (int j = 0; j < TI; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.w[i], f.x[j], acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  Frag f0, f1, f2, f3;
  int cur = 0;
  // S steps of 128 columns are under way
  const int steps = q8_steps(a.cols);
#pragma unroll
  for (int i = 0; i < S; ++i) load(i * kStep, q8_step_at(i, a.cols));
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the scales, before the workgroup meets
  wait_loads<(S - 1) * (LA + LB)>();
#pragma unroll
  for (int n = 0; n < kFrags; ++n) read1(lds, 0, f0, n);
  const auto first_half = [&](auto loads) {
    multiply(f0, [&](int i) {
#pragma unroll
      for (int n = i * 2 * kFrags / RI; n < (i + 1) * 2 * kFrags / RI; ++n)
        n < kFrags ? read1(lds + cur, 1, f1, n) : read1(lds + cur, 2, f2, n - kFrags);
      loads(i);
    });
    multiply(f1, [&](int i) {
#pragma unroll
      for (int n = i * 2 * kFrags / RI; n < (i + 1) * 2 * kFrags / RI && n < kFrags; ++n) read1(lds + cur, 3, f3, n);
    });
  };
  const auto turn = [&]() {
    cur = cur == (S - 1) * kStep ? 0 : cur + kStep;
    multiply(f3, [&](int i) {
#pragma unroll
      for (int n = i * kFrags / RI; n < (i + 1) * kFrags / RI; ++n) read1(lds + cur, 0, f0, n);
    });
  };
  const auto nothing = [](int) {};
  // the loads of a step are spread: the rows' pieces go out in its second half, the
  // tokens' in the first half of the next
  int i = 0, back = 0, k = 128 * S;
  const auto tokens = [&](int i) {
#pragma unroll
    for (int j = i * LB / RI; j < (i + 1) * LB / RI; ++j) load_x(j, back, k);
  };
  if (S < steps) {
    first_half(nothing);
    reads_done();
    multiply(f2, [&](int i) {
#pragma unroll
      for (int j = i * LA / RI; j < (i + 1) * LA / RI; ++j) load_w(j, cur, k);
    });
    back = cur;
    wait_loads<(S - 2) * (LA + LB) + LA>();
    turn();
    for (i = 1; i + S < steps; ++i) {
      first_half(tokens);
      // every wave has this step's fragments: its place takes the step S further on
      reads_done();
      k += 128;
      multiply(f2, [&](int i) {
#pragma unroll
        for (int j = i * LA / RI; j < (i + 1) * LA / RI; ++j) load_w(j, cur, k);
      });
      back = cur;
      wait_loads<(S - 2) * (LA + LB) + LA>();
      turn();
    }
    first_half(tokens);
    multiply(f2, nothing);
    wait_loads<0>();
    turn();
    ++i;
  }
  for (; i < steps - 1; ++i) {
    first_half(nothing);
    multiply(f2, nothing);
    wait_loads<0>();
    turn();
  }
  first_half(nothing);
  multiply(f2, nothing);
  multiply(f3, nothing);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // a single step's repeated loads
  // a lane holds, of token lane % 32, four rows in eight; the wave's halves swap, so
  // that it has eight in sixteen
  const int half = lane >> 5;
#pragma unroll
  for (int j = 0; j < TI; ++j) {
    const int tl = ti * (TT / WT) + j * 32 + (lane & 31), t = t0 + tl;
    const float sx = sxs[tl];
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
      for (int q = 0; q < 4; q += 2) {
        const int rl = wi * (RT / WR) + i * 32 + 8 * q;
        i32x4 lo, hi;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const auto p = __builtin_amdgcn_permlane32_swap(acc[i][j][4 * q + e], acc[i][j][4 * q + 4 + e], false, false);
          lo[e] = (int)p[0], hi[e] = (int)p[1];
        }
        const int rr = rl + 8 * half, r = r0 + rr;
        if (t >= a.T || r >= a.rows) continue;
        const float4 s0 = *(const float4 *)(sws + rr), s1 = *(const float4 *)(sws + rr + 4);
        const float4 v0 = make_float4(scaled(lo[0], sx, s0.x), scaled(lo[1], sx, s0.y), scaled(lo[2], sx, s0.z),
                                      scaled(lo[3], sx, s0.w));
        const float4 v1 = make_float4(scaled(hi[0], sx, s1.x), scaled(hi[1], sx, s1.y), scaled(hi[2], sx, s1.z),
                                      scaled(hi[3], sx, s1.w));
        store8(a.out, TY, t * a.ldo + r, v0, v1, a.rows - r);
      }
  }
}

// Few tokens: a workgroup takes 16 RB rows of w and up to 16 NT tokens, its 8 waves
// the pieces of 128 columns in turn; their sums meet in LDS.  The weights go from
// memory to registers, kAhead pieces of a wave at a time.  TX >= 0: x is of that type
// and the workgroup makes its codes itself (4 tokens at most), while its first weights
// are on the way.
constexpr int kFewWaves = 8, kAhead = 6;

template <int TY, int TX, int NT, int RB>
__global__ __launch_bounds__(64 * kFewWaves) void q8_few_kernel(Q8MatmulArgs a, const void *x, long long ldx) {
  extern __shared__ __attribute__((aligned(16))) int8_t lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r0 = blockIdx.x * 16 * RB, pieces = (a.cols + 127) / 128, padded = pieces * 128;
  i32x4 *sums = (i32x4 *)lds;                                  // [kFewWaves][NT * RB][64]
  int8_t *codes = lds + kFewWaves * NT * RB * 64 * 16;         // TX >= 0: [T][padded]
  const int at = (lane >> 4) * 16, wide = (a.cols + 15) & ~15;
  const int8_t *wp[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) wp[b] = a.w + (long long)min(r0 + 16 * b + (lane & 15), a.rows - 1) * a.ldw + at;
  i32x4 wv[kAhead][RB][2];
  const auto load = [&](int p0) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int c = (p0 + u * kFewWaves) * 128 + at;
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          // (columns past the last are multiplied by x's zeros)
          wv[u][b][h] = c + 64 * h < wide ? *(const i32x4 *)(wp[b] + c - at + 64 * h) : i32x4{0, 0, 0, 0};
    }
  };
  load(wave);
  __shared__ float scales[TX >= 0 ? 4 : 16 * NT];
  const int8_t *xp[NT];
  if constexpr (TX >= 0) {
    __shared__ uint32_t part[4][kFewWaves];
    for (int t = 0; t < a.T; ++t) {
      uint32_t m = 0;
      for (int c = 8 * threadIdx.x; c < a.cols; c += 8 * 64 * kFewWaves)
        m = largest(load8<TX>(x, t * ldx, c, a.cols), m);
      m = wave_largest(m);
      if (lane == 0) part[t][wave] = m;
    }
    __syncthreads();
    for (int t = 0; t < a.T; ++t) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kFewWaves; ++i) m = max(m, part[t][i]);
      const float s = q8_scale(m), inv = 1.f / s;
      if (threadIdx.x == 0) scales[t] = s;
      for (int c = 8 * threadIdx.x; c < padded; c += 8 * 64 * kFewWaves)
        *(uint2 *)(codes + t * padded + c) =
            c < a.cols ? q8_codes(load8<TX>(x, t * ldx, c, a.cols), s, inv) : make_uint2(0u, 0u);
    }
    __syncthreads();
    xp[0] = codes + min(lane & 15, a.T - 1) * padded + at;
  } else {
    if ((int)threadIdx.x < min(a.T, 16 * NT)) scales[threadIdx.x] = a.x_scales[threadIdx.x];
#pragma unroll
    for (int j = 0; j < NT; ++j) xp[j] = a.x + (long long)min(16 * j + (lane & 15), a.T - 1) * a.ldx + at;
  }
  i32x4 acc[RB][NT] = {};
  for (int p0 = wave; p0 < pieces; p0 += kAhead * kFewWaves) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int p = p0 + u * kFewWaves;
      if (p < pieces) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const i32x4 xv = *(const i32x4 *)(xp[j] + p * 128 + 64 * h);
#pragma unroll
            for (int b = 0; b < RB; ++b)
              acc[b][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[u][b][h], xv, acc[b][j], 0, 0, 0);
          }
      }
    }
    if (p0 + kAhead * kFewWaves < pieces) load(p0 + kAhead * kFewWaves);
  }
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int j = 0; j < NT; ++j) sums[(wave * NT * RB + b * NT + j) * 64 + lane] = acc[b][j];
  __syncthreads();
  // wave i takes tile i
  for (int i = wave; i < NT * RB; i += kFewWaves) {
    i32x4 v = sums[i * 64 + lane];
#pragma unroll
    for (int o = 1; o < kFewWaves; ++o) v += sums[(o * NT * RB + i) * 64 + lane];
    const int t = 16 * (i % NT) + (lane & 15), r = r0 + 16 * (i / NT) + 4 * (lane >> 4);
    if (t >= a.T || r >= a.rows) continue;
    const float sx = scales[t];
    float o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = scaled(v[e], sx, a.w_scales[min(r + e, a.rows - 1)]);
    const float4 f = make_float4(o[0], o[1], o[2], o[3]);
    if (r + 4 <= a.rows)
      store4(a.out, TY, t * a.ldo + r, f);
    else
      store_few(a.out, TY, t * a.ldo + r, f, a.rows - r);
  }
}

template <int TY, int I>
hipError_t launch_tile(const Q8MatmulArgs &a, hipStream_t s) {
  constexpr Q8Tile c = kQ8Tiles[I];
  const int r = (a.rows + c.rows - 1) / c.rows, t = (a.T + c.tokens - 1) / c.tokens;
  return launch(q8_tile_kernel<TY, c.rows, c.tokens, c.row_waves, c.token_waves, c.ahead>, dim3(r * t),
                dim3(64 * c.row_waves * c.token_waves), s, a, r, t);
}

template <int TY, int TX, int NT, int RB>
hipError_t launch_few(const Q8MatmulArgs &a, const Q8RowsArgs *q, hipStream_t s) {
  const size_t codes = q ? (size_t)a.T * q8_padded(a.cols) : 0;
  return launch_lds(q8_few_kernel<TY, TX, NT, RB>, dim3((a.rows + 16 * RB - 1) / (16 * RB)), dim3(64 * kFewWaves),
                    kFewWaves * NT * RB * 1024 + codes, s, a, q ? q->x : nullptr, q ? q->ldx : 0ll);
}

template <int TY>
hipError_t launch_type(const Q8MatmulArgs &a, hipStream_t s) {
  if (q8_few(a.T, a.rows)) {
    if (a.rows > 4096) return launch_few<TY, -1, 1, 2>(a, nullptr, s);
    return a.T <= 16 ? launch_few<TY, -1, 1, 1>(a, nullptr, s) : launch_few<TY, -1, 2, 1>(a, nullptr, s);
  }
  static_assert(kQ8TileCount == 7, "a case each");
  switch (q8_best_tile(a.T, a.rows, a.cols)) {
    case 0: return launch_tile<TY, 0>(a, s);
    case 1: return launch_tile<TY, 1>(a, s);
    case 2: return launch_tile<TY, 2>(a, s);
    case 3: return launch_tile<TY, 3>(a, s);
    case 4: return launch_tile<TY, 4>(a, s);
    case 5: return launch_tile<TY, 5>(a, s);
    default: return launch_tile<TY, 6>(a, s);
  }
}

// The tokens' codes made by the product's workgroups: saves a launch.
template <int TY>
hipError_t launch_few_linear(const Q8RowsArgs &q, const Q8MatmulArgs &a, hipStream_t s) {
  return a.rows > 4096 ? launch_few<TY, TY, 1, 2>(a, &q, s) : launch_few<TY, TY, 1, 1>(a, &q, s);
}

}  // namespace

hipError_t launch_q8_matmul(const Q8MatmulArgs &a, hipStream_t s) {
  return a.type == kF32 ? launch_type<kF32>(a, s) : a.type == kBf16 ? launch_type<kBf16>(a, s) : launch_type<kF16>(a, s);
}

hipError_t launch_q8_linear(const Q8RowsArgs &q, const Q8MatmulArgs &a, hipStream_t s) {
  // each workgroup makes all codes: worth it while they are few (and fit the LDS)
  if (q8_few(a.T, a.rows) && a.T <= 4 && a.T * q8_padded(a.cols) <= 32768 && q.type == a.type)
    return a.type == kF32    ? launch_few_linear<kF32>(q, a, s)
           : a.type == kBf16 ? launch_few_linear<kBf16>(q, a, s)
                             : launch_few_linear<kF16>(q, a, s);
  const hipError_t e = launch_q8_rows(q, s);
  return e == hipSuccess ? launch_q8_matmul(a, s) : e;
}

}  // namespace moe
