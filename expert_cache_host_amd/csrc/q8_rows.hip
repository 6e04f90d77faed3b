// Rows in 8-bit integers: s = max|x| / 127 (float32), code = rint(x / s).
#include "device_types.hpp"
#include "step_ops.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;

// x / s to the nearest integer, halves to the even one, exactly: the quotient's
// estimate is at most one off, and the rest x - q s is exact in binary64.
__device__ __forceinline__ int q8_code(float x, double s, double inv) {
  double q = rint((double)x * inv);
  const double r = fma(-q, s, (double)x), h = 0.5 * s;
  const bool odd = ((int)q & 1) != 0;
  if (r > h || (r == h && odd)) q += 1.0;
  if (r < -h || (r == -h && odd)) q -= 1.0;
  return (int)fmin(fmax(q, -127.0), 127.0);
}

template <int TY>
__global__ __launch_bounds__(kThreads) void q8_rows_kernel(Q8RowsArgs a) {
  __shared__ float part[kThreads / 64];
  const long long row = blockIdx.x;
  const int tid = threadIdx.x;
  float m = 0.f;
  bool bad = false;
  for (int c = tid; c < a.cols; c += kThreads) {
    const float v = fabsf(load1(a.x, TY, row * a.ldx + c));
    bad |= !(v < __builtin_inff());
    m = fmaxf(m, v);
  }
  if (bad) m = __builtin_inff();
  for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  if ((tid & 63) == 0) part[tid >> 6] = m;
  __syncthreads();
  m = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
  const bool ok = m < __builtin_inff();
  const float s = ok ? m / 127.f : __builtin_nanf("");
  if (tid == 0) a.scales[row] = s;
  const bool zero = !ok || s == 0.f;
  const double sd = (double)s, inv = 1.0 / sd;
  const int padded = (int)q8_padded(a.cols);
  for (int c = 4 * tid; c < padded; c += 4 * kThreads) {
    uint32_t b = 0;
    for (int j = 0; j < 4; ++j)
      if (c + j < a.cols && !zero)
        b |= (uint32_t)(q8_code(load1(a.x, TY, row * a.ldx + c + j), sd, inv) & 255) << (8 * j);
    *(uint32_t *)(a.codes + row * a.ldc + c) = b;
  }
}

}  // namespace

hipError_t launch_q8_rows(const Q8RowsArgs &a, hipStream_t s) {
  auto *k = a.type == kF32 ? q8_rows_kernel<kF32> : a.type == kBf16 ? q8_rows_kernel<kBf16> : q8_rows_kernel<kF16>;
  return launch(k, dim3(a.n), dim3(kThreads), s, a);
}

}  // namespace moe
