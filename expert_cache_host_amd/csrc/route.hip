// Routing to experts by a rule: scores, a selection value each, groups, the k
// best and their weights.  One wave takes a token.
#include "device_types.hpp"
#include "step_ops.hpp"

namespace moe {

namespace {

constexpr int kWaves = 4;

// Selection values as unsigned numbers of the same order: 0 is "taken or outside
// of the kept groups", 1 an excluded expert (minus infinity), above that the
// value's bits.
__device__ __forceinline__ uint64_t order_key(double c) {
  const int64_t b = __builtin_bit_cast(int64_t, c + 0.0);
  const uint64_t k = b < 0 ? ~(uint64_t)b : (uint64_t)b | 0x8000000000000000ull;
  return c == -__builtin_inf() ? 1ull : k;
}

__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
  for (int off = 32; off >= 1; off >>= 1) {
    const uint64_t o = __shfl_xor(v, off, 64);
    v = o > v ? o : v;
  }
  return v;
}
__device__ __forceinline__ double wave_max(double v) {
  for (int off = 32; off >= 1; off >>= 1) v = fmax(v, __shfl_xor(v, off, 64));
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

template <int NC>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(RouteArgs a) {
  __shared__ double values[kWaves][kRouteMaxExperts];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const long long t = (long long)blockIdx.x * kWaves + wave;
  if (t >= a.T) return;
  const double ninf = -__builtin_inf();
  double z[NC], s[NC];
  uint64_t key[NC];
  // NaN counts as minus infinity, plus infinity as the largest float
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int e = lane + 64 * c;
    float v = e < a.E ? load1(a.z, a.type, t * a.ldz + e) : -__builtin_inff();
    if (v != v) v = -__builtin_inff();
    z[c] = (double)fminf(v, 3.40282347e38f);
  }
  if (a.sigmoid) {
#pragma unroll
    for (int c = 0; c < NC; ++c) s[c] = 1.0 / (1.0 + exp(-z[c]));
  } else {
    double m = ninf;
#pragma unroll
    for (int c = 0; c < NC; ++c) m = fmax(m, z[c]);
    m = wave_max(m);
    double sum = 0.0;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      s[c] = z[c] == ninf ? 0.0 : exp(z[c] - m);
      sum += s[c];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int c = 0; c < NC; ++c) s[c] = sum > 0.0 ? s[c] / sum : 0.0;
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int e = lane + 64 * c;
    double v = z[c];
    if (a.bias && e < a.E && v != ninf) {
      const float b = a.bias[e];
      v = b == b ? s[c] + (double)b : ninf;
    }
    key[c] = e < a.E ? order_key(v) : 0ull;
    // groups go by the values; with no bias a pair's sum is that of its scores
    if (e < a.E) values[wave][e] = !a.bias && a.best == 2 && v != ninf ? s[c] : v;
  }
  if (a.keep < a.groups) {
    __builtin_amdgcn_wave_barrier();
    const int n = a.E / a.groups;
    double v = ninf;
    if (lane < a.groups) {
      double v1 = ninf, v2 = ninf;
      for (int i = 0; i < n; ++i) {
        const double x = values[wave][lane * n + (i + lane) % n];
        v2 = fmax(v2, fmin(v1, x));
        v1 = fmax(v1, x);
      }
      v = a.best == 2 ? (v2 == ninf ? ninf : v1 + v2) : v1;
    }
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double o = __shfl(v, g, 64);
      rank += o > v || (o == v && g < lane);
    }
    const uint64_t kept = __ballot(lane < a.groups && rank < a.keep);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int e = lane + 64 * c;
      if (e < a.E && !(kept >> (e / n) & 1)) key[c] = 0ull;
    }
  }
  int my_e = 0;
  double my_s = 0.0;
  for (int j = 0; j < a.k; ++j) {
    uint64_t m = 0;
#pragma unroll
    for (int c = 0; c < NC; ++c) m = key[c] > m ? key[c] : m;
    m = wave_max(m);
    bool found = false;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const uint64_t at = __ballot(key[c] == m);
      if (!found && at) {
        found = true;
        const int l = __ffsll((unsigned long long)at) - 1;
        const double sv = __shfl(m > 1ull ? s[c] : 0.0, l, 64);
        if (lane == j) my_e = l + 64 * c, my_s = sv;
        if (lane == l) key[c] = 0ull;
      }
    }
  }
  double w = my_s;
  if (a.renorm) {
    const double sum = wave_sum(lane < a.k ? my_s : 0.0);
    w = sum > 0.0 ? w / sum : 0.0;
  }
  if (lane < a.k) {
    const long long o = t * a.k + lane;
    const float f = (float)((double)a.scale * w);
    a.idx[o] = my_e;
    a.w[o] = f;
    if (a.idx2) a.idx2[o] = my_e, a.w2[o] = f;
  }
}

}  // namespace

hipError_t launch_route(const RouteArgs &a, hipStream_t s) {
  auto *k = a.E <= 64 ? route_kernel<1> : a.E <= 128 ? route_kernel<2> : a.E <= 256 ? route_kernel<4> : route_kernel<8>;
  return launch(k, dim3((a.T + kWaves - 1) / kWaves), dim3(64 * kWaves), s, a);
}

}  // namespace moe
