// Device helpers of the decoder-layer operators: loads and stores of the three
// element types through float32, and the packed batch's row lookup.
#pragma once
#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

#include <type_traits>

#include "decoder_ops.hpp"

namespace moe {

// Launches a kernel and returns this launch's own status.  (The thread's last HIP
// error, all that the launch syntax leaves, may be that of an earlier call of the
// caller's, which would then fail a call whose kernel runs.)
template <class... P>
hipError_t launch(void (*kernel)(P...), dim3 grid, dim3 block, hipStream_t s, std::common_type_t<P>... args) {
  void *p[] = {(void *)&args...};
  const hipError_t e = hipLaunchKernel((const void *)kernel, grid, block, p, 0, s);
  if (e != hipSuccess) (void)hipGetLastError();
  return e;
}

// The same with events recorded at the kernel's start and end.
template <class... P>
hipError_t launch_timed(void (*kernel)(P...), dim3 grid, dim3 block, hipStream_t s, hipEvent_t start, hipEvent_t stop,
                        std::common_type_t<P>... args) {
  void *p[] = {(void *)&args...};
  const hipError_t e = hipExtLaunchKernel((const void *)kernel, grid, block, p, 0, s, start, stop, 0);
  if (e != hipSuccess) (void)hipGetLastError();
  return e;
}

// The same with `lds` bytes of the workgroup's memory given at the launch.
template <class... P>
hipError_t launch_lds(void (*kernel)(P...), dim3 grid, dim3 block, size_t lds, hipStream_t s,
                      std::common_type_t<P>... args) {
  void *p[] = {(void *)&args...};
  const hipError_t e = hipLaunchKernel((const void *)kernel, grid, block, p, lds, s);
  if (e != hipSuccess) (void)hipGetLastError();
  return e;
}

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

// Four elements in one access, at any address aligned to one (the hardware takes
// vector accesses at any byte).
__device__ __forceinline__ float4 load4(const void *p, int type, long long i) {
  float4 v;
  if (type == kF32) {
    __builtin_memcpy(&v, (const float *)p + i, 16);
    return v;
  }
  uint2 b;
  __builtin_memcpy(&b, (const uint16_t *)p + i, 8);
  if (type == kBf16)
    return make_float4(bf16_to_f32(b.x & 0xffffu), bf16_to_f32(b.x >> 16),
                       bf16_to_f32(b.y & 0xffffu), bf16_to_f32(b.y >> 16));
  return make_float4(f16_to_f32((uint16_t)b.x), f16_to_f32((uint16_t)(b.x >> 16)),
                     f16_to_f32((uint16_t)b.y), f16_to_f32((uint16_t)(b.y >> 16)));
}

__device__ __forceinline__ void store4(void *p, int type, long long i, float4 v) {
  if (type == kF32) {
    __builtin_memcpy((float *)p + i, &v, 16);
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
  __builtin_memcpy((uint16_t *)p + i, &b, 8);
}

// The same for the last n < 4 elements of a row; the missing ones are 0.
__device__ __forceinline__ float4 load_few(const void *p, int type, long long i, int n) {
  return make_float4(load1(p, type, i), n > 1 ? load1(p, type, i + 1) : 0.f,
                     n > 2 ? load1(p, type, i + 2) : 0.f, 0.f);
}
__device__ __forceinline__ void store_few(void *p, int type, long long i, float4 v, int n) {
  store1(p, type, i, v.x);
  if (n > 1) store1(p, type, i + 1, v.y);
  if (n > 2) store1(p, type, i + 2, v.z);
}

constexpr int kMaxPos = 0x7fffff00;  // positions from here on are out of the cache

// Sequence of packed row t (the last s with start[s] <= t), or -1 for a row
// before the first or behind the last sequence: 64 sequences are compared at a
// time (one load's latency for up to 64 of them, two up to 4096).  Every lane of
// the wave takes part.
__device__ __forceinline__ int seq_of_row(const KvBatch &b, int t) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = b.n_seqs;  // the last s in [lo, hi) with start[s] <= t
  const int first = b.start[0], end = b.start[b.n_seqs];
  while (hi - lo > 1) {
    const int each = (hi - lo + 63) / 64, s = lo + lane * each;
    const bool before = s < hi && b.start[min(s, hi - 1)] <= t;
    lo += (max(__popcll(__ballot(before)), 1) - 1) * each;
    hi = min(hi, lo + each);
  }
  return t < first || t >= end ? -1 : __builtin_amdgcn_readfirstlane(lo);
}

}  // namespace moe
