// The norms before and after a block, with the block's gate, the residual
// scale and the residual sum, in one pass over the rows:
//
//   n  = y / sqrt(mean(y^2) + eps) * post_w      (post_w absent: n = y)
//   h' = res_scale * h + block_scale * gate * n  (y absent: h' = res_scale * h)
//   x  = h' / sqrt(mean(h'^2) + eps) * pre_w
//
// One workgroup per row; the row stays in registers between the two sums, so
// every input is read once and every output written once.  x is formed from h'
// before its rounding to the residual's type.  Bound by memory traffic.
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

// V elements per access (4: every row address is aligned to four elements), K
// accesses per thread.
template <int V, int K>
__global__ __launch_bounds__(1024) void block_norm_kernel(NormArgs a) {
  __shared__ float slots[2][16];
  const long long t = blockIdx.x;
  const int chunks = (a.d + V - 1) / V;
  float v[K][V], u[K][V];
  // the residual rows and the block's rows are requested together
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = k * blockDim.x + threadIdx.x;
#pragma unroll
    for (int j = 0; j < V; ++j) v[k][j] = u[k][j] = 0.f;
    if (c < chunks) {
      if constexpr (V == 4) {
        const float4 f = load4(a.h, a.h_type, t * a.ldh + 4 * c);
        v[k][0] = f.x, v[k][1] = f.y, v[k][2] = f.z, v[k][3] = f.w;
        if (a.y) {
          const float4 g = load4(a.y, a.y_type, t * a.ldy + 4 * c);
          u[k][0] = g.x, u[k][1] = g.y, u[k][2] = g.z, u[k][3] = g.w;
        }
      } else {
        v[k][0] = load1(a.h, a.h_type, t * a.ldh + c);
        if (a.y) u[k][0] = load1(a.y, a.y_type, t * a.ldy + c);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int j = 0; j < V; ++j) v[k][j] *= a.res_scale;

  if (a.y) {
    float r = a.block_scale;
    if (a.post_w) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) s = fmaf(u[k][j], u[k][j], s);
      s = wg_sum(s, slots[0]);
      r *= rsqrtf(s / (float)a.d + a.eps);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = k * blockDim.x + threadIdx.x;
      if (c < chunks) {
        float g[V], w[V];
#pragma unroll
        for (int j = 0; j < V; ++j) g[j] = w[j] = 1.f;
        if constexpr (V == 4) {
          if (a.post_w) {
            const float4 f = *(const float4 *)(a.post_w + 4 * c);
            w[0] = f.x, w[1] = f.y, w[2] = f.z, w[3] = f.w;
          }
          if (a.gate) {
            const float4 f = load4(a.gate, a.g_type, t * a.ldg + 4 * c);
            g[0] = f.x, g[1] = f.y, g[2] = f.z, g[3] = f.w;
          }
        } else {
          if (a.post_w) w[0] = a.post_w[c];
          if (a.gate) g[0] = load1(a.gate, a.g_type, t * a.ldg + c);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) v[k][j] = fmaf(u[k][j] * r * w[j], g[j], v[k][j]);
      }
    }
  }
  if (a.h_out) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = k * blockDim.x + threadIdx.x;
      if (c < chunks) {
        if constexpr (V == 4)
          store4(a.h_out, a.h_type, t * a.ldho + 4 * c,
                 make_float4(v[k][0], v[k][1], v[k][2], v[k][3]));
        else
          store1(a.h_out, a.h_type, t * a.ldho + c, v[k][0]);
      }
    }
  }
  if (a.pre_w) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) s = fmaf(v[k][j], v[k][j], s);
    s = wg_sum(s, slots[1]);
    const float r = rsqrtf(s / (float)a.d + a.eps);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = k * blockDim.x + threadIdx.x;
      if (c < chunks) {
        if constexpr (V == 4) {
          const float4 w = *(const float4 *)(a.pre_w + 4 * c);
          store4(a.x, a.x_type, t * a.ldx + 4 * c,
                 make_float4(v[k][0] * r * w.x, v[k][1] * r * w.y, v[k][2] * r * w.z,
                             v[k][3] * r * w.w));
        } else {
          store1(a.x, a.x_type, t * a.ldx + c, v[k][0] * r * a.pre_w[c]);
        }
      }
    }
  }
}

bool four_aligned(const void *p, int type, long long ld) {
  return !p || (((uintptr_t)p % (4 * type_bytes(type))) == 0 && ld % 4 == 0);
}

}  // namespace

hipError_t launch_block_norm(const NormArgs &a, hipStream_t s) {
  const bool vec = a.d % 4 == 0 && four_aligned(a.h, a.h_type, a.ldh) &&
                   four_aligned(a.y, a.y_type, a.ldy) && four_aligned(a.gate, a.g_type, a.ldg) &&
                   four_aligned(a.h_out, a.h_type, a.ldho) && four_aligned(a.x, a.x_type, a.ldx) &&
                   four_aligned(a.post_w, kF32, 0) && four_aligned(a.pre_w, kF32, 0);
  const int chunks = vec ? a.d / 4 : a.d;
  auto threads = [&](int k) { return dim3(((chunks + k - 1) / k + 63) / 64 * 64); };
  const dim3 grid((unsigned)a.T);
  if (vec) {
    if (chunks <= 1024)
      block_norm_kernel<4, 1><<<grid, threads(1), 0, s>>>(a);
    else if (chunks <= 2048)
      block_norm_kernel<4, 2><<<grid, threads(2), 0, s>>>(a);
    else
      block_norm_kernel<4, 8><<<grid, threads(8), 0, s>>>(a);
  } else {
    if (chunks <= 4096)
      block_norm_kernel<1, 4><<<grid, threads(4), 0, s>>>(a);
    else
      block_norm_kernel<1, 32><<<grid, threads(32), 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace moe
