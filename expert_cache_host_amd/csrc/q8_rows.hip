// Rows in 8-bit integers: s = max|x| / 127 (float32), code = rint(x / s).
//
// Bound by memory: a row is read once into registers, its maximum taken, and coded
// from there (rows past kHeld elements a thread are read a second time, out of the
// cache).  A row of up to 2048 columns takes one wave, a longer one a workgroup of
// four.  Codes are decided exactly: with q = rint(x * (1 / s)), one off at most, the
// rest r = x - q s is a float32 number (it is a multiple of s's last place, smaller
// than s), so that comparing 2 |r| with s corrects q and finds the halves.
#include "device_types.hpp"
#include "step_ops.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kHeld = 4;  // pieces of 8 elements a thread holds

struct Eight {
  float v[8];
};

// Elements i .. i + 7 of a row of n; those past its end are 0.
template <int TY>
__device__ __forceinline__ Eight load8(const void *p, long long row, int i, int n) {
  Eight e;
  if (i + 8 <= n) {
    if (TY == kF32) {
      __builtin_memcpy(e.v, (const float *)p + row + i, 32);
    } else {
      uint32_t b[4];
      __builtin_memcpy(b, (const uint16_t *)p + row + i, 16);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint16_t h = (uint16_t)(b[j / 2] >> (16 * (j & 1)));
        e.v[j] = TY == kBf16 ? bf16_to_f32(h) : f16_to_f32(h);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) e.v[j] = i + j < n ? load1(p, TY, row + i + j) : 0.f;
  }
  return e;
}

__device__ __forceinline__ uint32_t largest(const Eight &e, uint32_t m) {
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(e.v[j]) & 0x7fffffffu);
  return m;
}

__device__ __forceinline__ int q8_code(float x, float s, float inv) {
  float q = rintf(x * inv);
  const float r = fmaf(-q, s, x), a = 2.f * fabsf(r);
  // past the middle, or on it from an odd code
  if (a > s || (a == s && ((int)q & 1))) q += r > 0.f ? 1.f : -1.f;
  return (int)fminf(fmaxf(q, -127.f), 127.f);
}

// Scales below the normal numbers have no reciprocal in float32.
__device__ __forceinline__ int q8_code_tiny(float x, float s) {
  const double d = s;
  double q = rint((double)x / d);
  return (int)fmin(fmax(q, -127.0), 127.0);
}

__device__ __forceinline__ void store8(int8_t *p, const Eight &e, float s, float inv) {
  uint32_t b[2] = {0u, 0u};
  if (s >= 1.17549435e-38f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j / 4] |= (uint32_t)(q8_code(e.v[j], s, inv) & 255) << (8 * (j & 3));
  } else if (s > 0.f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j / 4] |= (uint32_t)(q8_code_tiny(e.v[j], s) & 255) << (8 * (j & 3));
  }
  *(uint2 *)p = make_uint2(b[0], b[1]);
}

// W waves a row.
template <int TY, int W>
__global__ __launch_bounds__(kThreads) void q8_rows_kernel(Q8RowsArgs a) {
  constexpr int kPer = 64 * W;  // threads a row
  __shared__ uint32_t part[kThreads / 64];
  const int lane = threadIdx.x % kPer, wave = threadIdx.x >> 6;
  const long long row = (long long)blockIdx.x * (kThreads / kPer) + threadIdx.x / kPer;
  const bool mine = row < a.n;
  const long long at = row * a.ldx;
  Eight held[kHeld];
  uint32_t m = 0;
  if (mine) {
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
      if (8 * (lane + h * kPer) < a.cols) held[h] = load8<TY>(a.x, at, 8 * (lane + h * kPer), a.cols);
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
      if (8 * (lane + h * kPer) < a.cols) m = largest(held[h], m);
    for (int c = 8 * (lane + kHeld * kPer); c < a.cols; c += 8 * kPer) m = largest(load8<TY>(a.x, at, c, a.cols), m);
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
  if (W > 1) {
    if ((threadIdx.x & 63) == 0) part[wave] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < W; ++i) m = max(m, part[i]);
  }
  if (!mine) return;
  // an infinity or a NaN: scale NaN, codes 0
  const float s = m < 0x7f800000u ? __uint_as_float(m) / 127.f : __builtin_nanf("");
  const float inv = 1.f / s;
  if (lane == 0) a.scales[row] = s;
  int8_t *out = a.codes + row * a.ldc;
  const int padded = (int)q8_padded(a.cols);
#pragma unroll
  for (int h = 0; h < kHeld; ++h) {
    const int c = 8 * (lane + h * kPer);
    if (c < a.cols)
      store8(out + c, held[h], s, inv);
    else if (c < padded)
      *(uint2 *)(out + c) = make_uint2(0u, 0u);
  }
  for (int c = 8 * (lane + kHeld * kPer); c < padded; c += 8 * kPer) {
    if (c < a.cols)
      store8(out + c, load8<TY>(a.x, at, c, a.cols), s, inv);
    else
      *(uint2 *)(out + c) = make_uint2(0u, 0u);
  }
}

template <int TY>
hipError_t launch_type(const Q8RowsArgs &a, hipStream_t s) {
  if (a.cols <= 64 * 8 * kHeld) return launch(q8_rows_kernel<TY, 1>, dim3((a.n + 3) / 4), dim3(kThreads), s, a);
  return launch(q8_rows_kernel<TY, 4>, dim3(a.n), dim3(kThreads), s, a);
}

}  // namespace

hipError_t launch_q8_rows(const Q8RowsArgs &a, hipStream_t s) {
  return a.type == kF32 ? launch_type<kF32>(a, s) : a.type == kBf16 ? launch_type<kBf16>(a, s) : launch_type<kF16>(a, s);
}

}  // namespace moe
