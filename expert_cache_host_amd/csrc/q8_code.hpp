// The 8-bit code of a row's element, shared by the kernels that make codes.
#pragma once
#include "device_types.hpp"

namespace moe {

struct Eight {
  float v[8];
};

// Elements i .. i + 7 of the row of n that starts at `row`; those past its end are 0.
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

// The largest magnitude's bits: infinities and NaN come out as the largest of all.
__device__ __forceinline__ uint32_t largest(const Eight &e, uint32_t m) {
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(e.v[j]) & 0x7fffffffu);
  return m;
}

__device__ __forceinline__ uint32_t wave_largest(uint32_t m) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
  return m;
}

// The scale of a row whose largest magnitude has the bits m.
__device__ __forceinline__ float q8_scale(uint32_t m) {
  return m < 0x7f800000u ? __uint_as_float(m) / 127.f : __builtin_nanf("");
}

// rint(x / s), halves to the even code, exactly.  With q = rint(x * (1 / s)), one off
// at most, the rest x - q s is a float32 number (a multiple of s's last place, smaller
// than s): comparing twice its magnitude with s corrects q and finds the halves.
__device__ __forceinline__ int q8_code(float x, float s, float inv) {
  float q = rintf(x * inv);
  const float r = fmaf(-q, s, x), a = 2.f * fabsf(r);
  if (a > s || (a == s && ((int)q & 1))) q += r > 0.f ? 1.f : -1.f;
  return (int)fminf(fmaxf(q, -127.f), 127.f);
}

// Eight codes at scale s (inv = 1 / s); scale 0 or NaN gives codes 0.
__device__ __forceinline__ uint2 q8_codes(const Eight &e, float s, float inv) {
  uint32_t b[2] = {0u, 0u};
  if (s >= 1.17549435e-38f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j / 4] |= (uint32_t)(q8_code(e.v[j], s, inv) & 255) << (8 * (j & 3));
  } else if (s > 0.f) {  // a subnormal scale has no reciprocal in float32
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double q = fmin(fmax(rint((double)e.v[j] / (double)s), -127.0), 127.0);
      b[j / 4] |= (uint32_t)((int)q & 255) << (8 * (j & 3));
    }
  }
  return make_uint2(b[0], b[1]);
}

}  // namespace moe
