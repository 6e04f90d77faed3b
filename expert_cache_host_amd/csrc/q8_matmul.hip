// out[t][r] = sx[t] sw[r] sum_c x[t][c] w[r][c] over 8-bit integers.
#include "device_types.hpp"
#include "step_ops.hpp"

namespace moe {

namespace {

using i32x4 = __attribute__((ext_vector_type(4))) int;

constexpr int kThreads = 256;

// (sum sx) sw, both products rounded to float32.  The value is settled there:
// a conversion to binary16 taken together with the product would round once where
// the definition rounds twice.
__device__ __forceinline__ float scaled(int sum, float sx, float sw) {
  float v = (float)sum * sx * sw;
  asm volatile("" : "+v"(v));
  return v;
}

using i32x16 = __attribute__((ext_vector_type(16))) int;

// Rows of codes as a buffer that starts at row r0: what lies behind the last row reads 0.
__device__ __forceinline__ i32x4 rows_from(const int8_t *p, long long ld, int r0, int rows, int most, int bytes) {
  const uint64_t base = (uint64_t)(p + (long long)r0 * ld);
  i32x4 r;
  r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)base);
  r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(base >> 32) & 0xffff);
  r[2] = __builtin_amdgcn_readfirstlane((min(rows - r0, most) - 1) * (int)ld + bytes);
  r[3] = 0x00027000;
  return r;
}

// 16 bytes a lane from the buffer's byte lane_at + at into LDS, the wave's kilobyte
// at place `l`.  Written as assembly (it returns nothing in registers) because the
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
template <int TY, int RT, int TT, int WR, int WT>
__global__ __launch_bounds__(64 * WR * WT) void q8_tile_kernel(Q8MatmulArgs a, int r_tiles, int t_tiles) {
  constexpr int NW = WR * WT, RI = RT / WR / 32, TI = TT / WT / 32;
  constexpr int LA = RT / 8 / NW, LB = TT / 8 / NW;
  static_assert(RT % (8 * NW) == 0 && TT % (8 * NW) == 0, "whole loads");
  constexpr int kStep = (RT + TT) * 128;
  __shared__ __attribute__((aligned(1024))) int8_t lds[2 * kStep];
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
  const auto wr = rows_from(a.w, a.ldw, r0, a.rows, RT, (a.cols + 15) & ~15);
  const auto xr = rows_from(a.x, a.ldx, t0, a.T, TT, (a.cols + 127) & ~127);
  // a wave's load takes 8 rows of 128 bytes; the 16-byte pieces of row r lie at place
  // piece ^ r / 2 % 8: sixteen lanes that read the same piece of sixteen rows then
  // touch each of the 64 banks once (with r % 8 half of the LDS time was conflicts)
  static_assert(NW % 2 == 0, "a wave's loads all start at rows of the same r / 8 % 2");
  const int piece = ((lane & 7) ^ ((wave & 1) * 4 + (lane >> 4))) * 16, row = (lane >> 3) + 8 * wave;
  const int wo = row * (int)a.ldw + piece, xo = row * (int)a.ldx + piece;
  const int ldw8 = 8 * NW * (int)a.ldw, ldx8 = 8 * NW * (int)a.ldx;
  const uint32_t lds_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) int8_t *)lds + wave * 1024;
  const auto load = [&](int to, int k) {
#pragma unroll
    for (int j = 0; j < LA; ++j) load_lds(wr, lds_at + to + j * NW * 1024, wo, j * ldw8 + k);
#pragma unroll
    for (int j = 0; j < LB; ++j) load_lds(xr, lds_at + to + RT * 128 + j * NW * 1024, xo, j * ldx8 + k);
  };
  const int wi = wave % WR, ti = wave / WR;
  const int ra = (wi * (RT / WR) + (lane & 31)) * 128, rb = (RT + ti * (TT / WT) + (lane & 31)) * 128;
  i32x16 acc[RI][TI] = {};
  struct Frag {
    i32x4 w[RI], x[TI];
  };
  const auto read = [&](const int8_t *l, int s, Frag &f) {
    const int c = ((2 * s + (lane >> 5)) ^ (lane >> 1 & 7)) * 16;
#pragma unroll
    for (int j = 0; j < TI; ++j) f.x[j] = *(const i32x4 *)(l + rb + c + j * 4096);
#pragma unroll
    for (int i = 0; i < RI; ++i) f.w[i] = *(const i32x4 *)(l + ra + c + i * 4096);
  };
  const auto multiply = [&](const Frag &f) {
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
      for (int j = 0; j < TI; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.w[i], f.x[j], acc[i][j], 0, 0, 0);
  };
  // `reads` reads of fragments to a product, the rest of the products after them
  const auto mix = [&](auto reads) {
#pragma unroll
    for (int i = 0; i < RI * TI; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (i < RI + TI) __builtin_amdgcn_sched_group_barrier(0x100, decltype(reads)::value, 0);
    }
  };
  using One = std::integral_constant<int, 1>;
  using Two = std::integral_constant<int, 2>;
  Frag f0, f1, f2, f3;
  int cur = 0;
  const auto first_half = [&]() {
    read(lds + cur, 1, f1), multiply(f0), mix(One{});
    read(lds + cur, 2, f2), read(lds + cur, 3, f3), multiply(f1), mix(Two{});
  };
  const auto turn = [&]() {
    read(lds + kStep - cur, 0, f0), multiply(f3), mix(One{});
    cur = kStep - cur;
  };
  // at least two steps of 128 columns (launch_type's rule)
  const int steps = (a.cols + 127) / 128;
  load(0, 0);
  load(kStep, 128);
  wait_loads<LA + LB>();
  read(lds, 0, f0);
  for (int i = 2; i < steps; ++i) {
    first_half();
    // every wave has this step's fragments: its place takes the step after the next
    reads_done();
    load(cur, 128 * i);
    multiply(f2);
    wait_loads<LA + LB>();
    turn();
  }
  first_half();
  multiply(f2);
  wait_loads<0>();
  turn();
  first_half();
  multiply(f2);
  multiply(f3);
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

template <int TY>
__global__ __launch_bounds__(kThreads) void q8_matmul_kernel(Q8MatmulArgs a) {
  // a wave takes 16 rows of w and 16 tokens
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r0 = (blockIdx.x * 4 + wave) * 16, t0 = blockIdx.y * 16;
  if (r0 >= a.rows) return;
  const int r = min(r0 + (lane & 15), a.rows - 1), t = min(t0 + (lane & 15), a.T - 1);
  const int8_t *wp = a.w + r * a.ldw, *xp = a.x + t * a.ldx;
  i32x4 acc = {0, 0, 0, 0};
  for (int k = 0; k < a.cols; k += 64) {
    const int kk = k + (lane >> 4) * 16;
    i32x4 wv = {0, 0, 0, 0}, xv = *(const i32x4 *)(xp + kk);
    if (kk < a.cols) wv = *(const i32x4 *)(wp + kk);
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv, xv, acc, 0, 0, 0);
  }
  if (t0 + (lane & 15) >= a.T) return;
  const float sx = a.x_scales[t];
  for (int i = 0; i < 4; ++i) {
    const int rr = r0 + (lane >> 4) * 4 + i;
    if (rr < a.rows) store1(a.out, TY, t * a.ldo + rr, scaled(acc[i], sx, a.w_scales[rr]));
  }
}

template <int TY>
hipError_t launch_type(const Q8MatmulArgs &a, hipStream_t s) {
  if (a.T > 64 && a.cols > 128) {
    const int r = (a.rows + 255) / 256, t = (a.T + 255) / 256;
    return launch(q8_tile_kernel<TY, 256, 256, 2, 4>, dim3(r * t), dim3(512), s, a, r, t);
  }
  return launch(q8_matmul_kernel<TY>, dim3((a.rows + 63) / 64, (a.T + 15) / 16), dim3(kThreads), s, a);
}

}  // namespace

hipError_t launch_q8_matmul(const Q8MatmulArgs &a, hipStream_t s) {
  return a.type == kF32 ? launch_type<kF32>(a, s) : a.type == kBf16 ? launch_type<kBf16>(a, s) : launch_type<kF16>(a, s);
}

}  // namespace moe
