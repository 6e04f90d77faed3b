// The norms before and after a block, with the block's gate, the residual
// scale and the residual sum, in one pass over the rows:
//
//   n  = y / sqrt(mean(y^2) + eps) * post_w      (post_w absent: n = y)
//   h' = res_scale * h + block_scale * gate * n  (y absent: h' = res_scale * h)
//   x  = h' / sqrt(mean(h'^2) + eps) * pre_w
//
// One workgroup per row; the row stays in registers between the two sums, so
// every input is read once and every output written once.  x is formed from h'
// before its rounding to the residual's type.  Bound by memory traffic (3.9 TB/s
// at 4093 x 2045 f16 with a gate per element, 3.4 TB/s at 512 x 6144, where a large
// copy reaches 5.1; 4.8 and 3.7 on inputs in the last-level cache); a single row is
// bound by the launch and two workgroup sums (3.8 us at d = 2816).
#include <algorithm>

#include "device_types.hpp"

namespace moe {

namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

// Sum over the workgroup; `slot` (16 floats) is used by this call alone.
__device__ __forceinline__ float wg_sum(float v, float *slot) {
  v = wave_sum(v);
  const int wave = threadIdx.x >> 6, n = (blockDim.x + 63) >> 6;
  if (n == 1) return v;
  if ((threadIdx.x & 63) == 0) slot[wave] = v;
  __syncthreads();
  float r = 0.f;
  for (int i = 0; i < n; ++i) r += slot[i];
  return r;
}

// K accesses of four elements per thread (the row's last may hold fewer).
template <int K>
__global__ __launch_bounds__(1024) void block_norm_kernel(NormArgs a) {
  __shared__ float slots[2][16];
  const long long t = (long long)blockIdx.y * gridDim.x + blockIdx.x;
  if (t >= a.T) return;
  const int chunks = (a.d + 3) / 4;
  auto load = [&](const void *p, int type, long long row, int c) {
    return 4 * c + 4 <= a.d ? load4(p, type, row + 4 * c) : load_few(p, type, row + 4 * c, a.d & 3);
  };
  auto store = [&](void *p, int type, long long row, int c, float4 v) {
    if (4 * c + 4 <= a.d)
      store4(p, type, row + 4 * c, v);
    else
      store_few(p, type, row + 4 * c, v, a.d & 3);
  };
  float4 v[K], u[K];
  // the residual's and the block's row are requested together
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = k * blockDim.x + threadIdx.x;
    v[k] = u[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < chunks) {
      v[k] = load(a.h, a.h_type, t * a.ldh, c);
      if (a.y) u[k] = load(a.y, a.y_type, t * a.ldy, c);
    }
  }
#pragma unroll
  for (int k = 0; k < K; ++k)
    v[k].x *= a.res_scale, v[k].y *= a.res_scale, v[k].z *= a.res_scale, v[k].w *= a.res_scale;

  if (a.y) {
    float r = a.block_scale;
    if (a.post_w) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k)
        s = fmaf(u[k].x, u[k].x, fmaf(u[k].y, u[k].y, fmaf(u[k].z, u[k].z, fmaf(u[k].w, u[k].w, s))));
      s = wg_sum(s, slots[0]);
      r *= rsqrtf(s / (float)a.d + a.eps);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = k * blockDim.x + threadIdx.x;
      if (c < chunks) {
        float4 w = make_float4(1.f, 1.f, 1.f, 1.f), g = w;
        if (a.post_w) w = load(a.post_w, kF32, 0, c);
        if (a.gate) g = load(a.gate, a.g_type, t * a.ldg, c);
        v[k].x = fmaf(u[k].x * r * w.x, g.x, v[k].x);
        v[k].y = fmaf(u[k].y * r * w.y, g.y, v[k].y);
        v[k].z = fmaf(u[k].z * r * w.z, g.z, v[k].z);
        v[k].w = fmaf(u[k].w * r * w.w, g.w, v[k].w);
      }
    }
  }
  if (a.h_out) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = k * blockDim.x + threadIdx.x;
      if (c < chunks) store(a.h_out, a.h_type, t * a.ldho, c, v[k]);
    }
  }
  if (a.pre_w) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
      s = fmaf(v[k].x, v[k].x, fmaf(v[k].y, v[k].y, fmaf(v[k].z, v[k].z, fmaf(v[k].w, v[k].w, s))));
    s = wg_sum(s, slots[1]);
    const float r = rsqrtf(s / (float)a.d + a.eps);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = k * blockDim.x + threadIdx.x;
      if (c < chunks) {
        const float4 w = load(a.pre_w, kF32, 0, c);
        store(a.x, a.x_type, t * a.ldx, c,
              make_float4(v[k].x * r * w.x, v[k].y * r * w.y, v[k].z * r * w.z, v[k].w * r * w.w));
      }
    }
  }
}

}  // namespace

hipError_t launch_block_norm(const NormArgs &a, hipStream_t s) {
  const int chunks = (a.d + 3) / 4;
  // a grid dimension holds fewer than 2^32 threads: 2^21 rows of up to 1024
  const int gx = std::min(a.T, 1 << 21);
  const dim3 grid((unsigned)gx, (unsigned)((a.T - 1) / gx + 1));
  auto threads = [&](int k) { return dim3(((chunks + k - 1) / k + 63) / 64 * 64); };
  // Accesses per thread: as many (up to 4) as leave the chip 2^18 threads, else
  // what a workgroup of 1024 needs.  More loads in flight per thread and fewer
  // waves to meet help long batches (4093 x 2045 f16: 25.7 us with one access,
  // 21.2 with two, 18.1 with four), threads help short ones (512 x 6144: 10.3 us
  // with two, 12.0 with four).
  int k = 4;
  while (k > 1 && (long long)a.T * chunks / k < 1 << 18) k /= 2;
  while (chunks > 1024 * k) k *= 2;
  if (k <= 1) return launch(block_norm_kernel<1>, grid, threads(1), s, a);
  if (k <= 2) return launch(block_norm_kernel<2>, grid, threads(2), s, a);
  if (k <= 4) return launch(block_norm_kernel<4>, grid, threads(4), s, a);
  return launch(block_norm_kernel<8>, grid, threads(8), s, a);
}

}  // namespace moe
