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

}  // namespace

hipError_t launch_q8_matmul(const Q8MatmulArgs &a, hipStream_t s) {
  auto *k = a.type == kF32 ? q8_matmul_kernel<kF32> : a.type == kBf16 ? q8_matmul_kernel<kBf16> : q8_matmul_kernel<kF16>;
  return launch(k, dim3((a.rows + 63) / 64, (a.T + 15) / 16), dim3(kThreads), s, a);
}

}  // namespace moe
