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
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_from(const int8_t *p, long long ld, int r0, int rows, int most,
                                                            int bytes) {
  const int n = min(rows - r0, most);
  return __builtin_amdgcn_make_buffer_rsrc((void *)(p + (long long)r0 * ld), 0, (n - 1) * (int)ld + bytes, 0x00027000);
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
  const auto wr = rows_from(a.w, a.ldw, r0, a.rows, RT, (a.cols + 15) & ~15);
  const auto xr = rows_from(a.x, a.ldx, t0, a.T, TT, (a.cols + 127) & ~127);
  // a wave's load takes 8 rows of 128 bytes; the 16-byte pieces of row r lie at place (piece ^ r % 8)
  const int piece = ((lane & 7) ^ (lane >> 3)) * 16, row = (lane >> 3) + 8 * wave;
  const int wo = row * (int)a.ldw + piece, xo = row * (int)a.ldx + piece;
  const int ldw8 = 8 * NW * (int)a.ldw, ldx8 = 8 * NW * (int)a.ldx;
  using lds_ptr = __attribute__((address_space(3))) void *;
  const auto load = [&](int8_t *l, int k) {
#pragma unroll
    for (int j = 0; j < LA; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, (lds_ptr)(l + (j * NW + wave) * 1024), 16, wo, j * ldw8 + k, 0, 0);
#pragma unroll
    for (int j = 0; j < LB; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, (lds_ptr)(l + RT * 128 + (j * NW + wave) * 1024), 16, xo,
                                               j * ldx8 + k, 0, 0);
  };
  const int wi = wave % WR, ti = wave / WR;
  const int ra = (wi * (RT / WR) + (lane & 31)) * 128, rb = (RT + ti * (TT / WT) + (lane & 31)) * 128;
  i32x16 acc[RI][TI] = {};
  const auto multiply = [&](const int8_t *l) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int c = ((2 * s + (lane >> 5)) ^ (lane & 7)) * 16;
      i32x4 wf[RI], xf[TI];
#pragma unroll
      for (int j = 0; j < TI; ++j) xf[j] = *(const i32x4 *)(l + rb + c + j * 4096);
#pragma unroll
      for (int i = 0; i < RI; ++i) wf[i] = *(const i32x4 *)(l + ra + c + i * 4096);
#pragma unroll
      for (int i = 0; i < RI; ++i)
#pragma unroll
        for (int j = 0; j < TI; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[i], xf[j], acc[i][j], 0, 0, 0);
    }
  };
  const int end = (a.cols + 127) & ~127;
  load(lds, 0);
  int cur = 0;
  for (int k = 128; k < end; k += 128, cur = kStep - cur) {
    __syncthreads();
    load(lds + kStep - cur, k);
    multiply(lds + cur);
  }
  __syncthreads();
  multiply(lds + cur);
#pragma unroll
  for (int j = 0; j < TI; ++j) {
    const int t = t0 + ti * (TT / WT) + j * 32 + (lane & 31);
    if (t >= a.T) continue;
    const float sx = a.x_scales[t];
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = r0 + wi * (RT / WR) + i * 32 + 8 * q + 4 * (lane >> 5);
        const long long o = t * a.ldo + r;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = scaled(acc[i][j][4 * q + e], sx, r + e < a.rows ? a.w_scales[r + e] : 0.f);
        if (r + 4 <= a.rows)
          store4(a.out, TY, o, make_float4(v[0], v[1], v[2], v[3]));
        else if (r < a.rows)
          store_few(a.out, TY, o, make_float4(v[0], v[1], v[2], v[3]), a.rows - r);
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
  if (a.T > 64) {
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
