// A few tokens times a matrix held in 4 bits:
//
//   out[t][r] = sum_g s[r][g] * sum_{c in group g} (q[r][c] - 8) * x[t][c]
//
// One wave per output row and token; a lane takes every 64th block of 32
// weights.  Codes are exact small integers, products and sums in float32.
#include "device_types.hpp"

namespace moe {

namespace {

__global__ __launch_bounds__(256) void q4_matvec_kernel(Q4MatvecArgs a) {
  const int lane = threadIdx.x & 63;
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
  const long long t = blockIdx.y;
  if (row >= a.rows) return;
  const int nb = a.cols / 32, per = a.group / 32;
  float acc = 0.f;
  for (int b = lane; b < nb; b += 64) {
    const uint4 w = *(const uint4 *)(a.q + (row * nb + b) * 16);
    const float s = f16_to_f32(a.scales[row * (nb / per) + b / per]);
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const uint32_t byte = ws[j / 4] >> (8 * (j % 4));
      sum = fmaf((float)(int)(byte & 15u) - 8.f, load1(a.x, a.type, t * a.ldx + b * 32 + j), sum);
      sum = fmaf((float)(int)((byte >> 4) & 15u) - 8.f,
                 load1(a.x, a.type, t * a.ldx + b * 32 + 16 + j), sum);
    }
    acc = fmaf(s, sum, acc);
  }
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) acc += __shfl_xor(acc, m);
  if (lane == 0) store1(a.out, a.type, t * a.ldo + row, acc);
}

}  // namespace

hipError_t launch_q4_matvec(const Q4MatvecArgs &a, hipStream_t s) {
  q4_matvec_kernel<<<dim3((unsigned)((a.rows + 3) / 4), (unsigned)a.T), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace moe
