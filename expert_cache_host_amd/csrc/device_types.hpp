// Device helpers of the decoder-layer operators: loads and stores of the three
// element types through float32, and the packed batch's row lookup.
#pragma once
#include <hip/hip_runtime.h>

#include "decoder_ops.hpp"

namespace moe {

__device__ __forceinline__ float bf16_to_f32(uint32_t b) {
  return __builtin_bit_cast(float, b << 16);
}

// Round to nearest even; a NaN keeps its sign and becomes quiet.
__device__ __forceinline__ uint16_t f32_to_bf16(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}

__device__ __forceinline__ float f16_to_f32(uint16_t b) {
  return (float)__builtin_bit_cast(_Float16, b);
}

__device__ __forceinline__ uint16_t f32_to_f16(float v) {
  return __builtin_bit_cast(uint16_t, (_Float16)v);
}

__device__ __forceinline__ float load1(const void *p, int type, long long i) {
  if (type == kF32) return ((const float *)p)[i];
  const uint16_t b = ((const uint16_t *)p)[i];
  return type == kBf16 ? bf16_to_f32(b) : f16_to_f32(b);
}

__device__ __forceinline__ void store1(void *p, int type, long long i, float v) {
  if (type == kF32)
    ((float *)p)[i] = v;
  else
    ((uint16_t *)p)[i] = type == kBf16 ? f32_to_bf16(v) : f32_to_f16(v);
}

// Four elements from an address aligned to four elements.
__device__ __forceinline__ float4 load4(const void *p, int type, long long i) {
  if (type == kF32) return *(const float4 *)((const float *)p + i);
  const uint2 b = *(const uint2 *)((const uint16_t *)p + i);
  if (type == kBf16)
    return make_float4(bf16_to_f32(b.x & 0xffffu), bf16_to_f32(b.x >> 16),
                       bf16_to_f32(b.y & 0xffffu), bf16_to_f32(b.y >> 16));
  return make_float4(f16_to_f32((uint16_t)b.x), f16_to_f32((uint16_t)(b.x >> 16)),
                     f16_to_f32((uint16_t)b.y), f16_to_f32((uint16_t)(b.y >> 16)));
}

__device__ __forceinline__ void store4(void *p, int type, long long i, float4 v) {
  if (type == kF32) {
    *(float4 *)((float *)p + i) = v;
    return;
  }
  uint2 b;
  if (type == kBf16) {
    b.x = f32_to_bf16(v.x) | ((uint32_t)f32_to_bf16(v.y) << 16);
    b.y = f32_to_bf16(v.z) | ((uint32_t)f32_to_bf16(v.w) << 16);
  } else {
    b.x = f32_to_f16(v.x) | ((uint32_t)f32_to_f16(v.y) << 16);
    b.y = f32_to_f16(v.z) | ((uint32_t)f32_to_f16(v.w) << 16);
  }
  *(uint2 *)((uint16_t *)p + i) = b;
}

// Sequence of packed row t (the last s with start[s] <= t), or -1 for a row
// before the first or behind the last sequence.
__device__ __forceinline__ int seq_of_row(const KvBatch &b, int t) {
  if (t < b.start[0] || t >= b.start[b.n_seqs]) return -1;
  int lo = 0, hi = b.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.start[mid] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

}  // namespace moe
