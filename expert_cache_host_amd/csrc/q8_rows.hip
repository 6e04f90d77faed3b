// Rows in 8-bit integers: s = max|x| / 127 (float32), code = rint(x / s).
//
// A row is read once into registers, its maximum taken, and coded from there (what a
// thread cannot hold is read a second time, out of the cache).  4096 x 6144 bfloat16:
// 22 us, 3.4 TB/s, bound by vector instructions, 24 an element (the exact codes), which
// take 0.76 of the CUs' cycles; 512 x 6144: 5.6, latency.
#include "q8_code.hpp"
#include "step_ops.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kHeld = 4;  // pieces of 8 elements a thread holds

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
  m = wave_largest(m);
  if (W > 1) {
    if ((threadIdx.x & 63) == 0) part[wave] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < W; ++i) m = max(m, part[i]);
  }
  if (!mine) return;
  const float s = q8_scale(m);
  const float inv = 1.f / s;
  if (lane == 0) a.scales[row] = s;
  int8_t *out = a.codes + row * a.ldc;
  const int padded = (int)q8_padded(a.cols);
#pragma unroll
  for (int h = 0; h < kHeld; ++h) {
    const int c = 8 * (lane + h * kPer);
    if (c < a.cols)
      *(uint2 *)(out + c) = q8_codes(held[h], s, inv);
    else if (c < padded)
      *(uint2 *)(out + c) = make_uint2(0u, 0u);
  }
  for (int c = 8 * (lane + kHeld * kPer); c < padded; c += 8 * kPer) {
    if (c < a.cols)
      *(uint2 *)(out + c) = q8_codes(load8<TY>(a.x, at, c, a.cols), s, inv);
    else
      *(uint2 *)(out + c) = make_uint2(0u, 0u);
  }
}

// One wave a row where rows are short, or many enough to fill the card that way (8192 x
// 1024 float32: 11.6 us, 13.8 with four); else four (509 x 2045: 4.1 us, 6.4 with one).
template <int TY>
hipError_t launch_type(const Q8RowsArgs &a, hipStream_t s) {
  if (a.cols <= 512 || (a.cols <= 64 * 8 * kHeld && a.n >= 4096))
    return launch(q8_rows_kernel<TY, 1>, dim3((a.n + 3) / 4), dim3(kThreads), s, a);
  return launch(q8_rows_kernel<TY, 4>, dim3(a.n), dim3(kThreads), s, a);
}

}  // namespace

hipError_t launch_q8_rows(const Q8RowsArgs &a, hipStream_t s) {
  return a.type == kF32 ? launch_type<kF32>(a, s) : a.type == kBf16 ? launch_type<kBf16>(a, s) : launch_type<kF16>(a, s);
}

}  // namespace moe
