// Routing to experts by a rule: scores, a selection value each, groups, the k best and
// their weights.  One wave takes a token.
//
// Selection values are defined in binary64, which all experts need not: their float32
// estimates tell all but the few within rounding of the k-th apart.  So a float32 that
// k estimates reach, or a few more, is found by halving (a comparison an expert, the
// counts from ballots); the experts not below it by more than the estimates' error get
// their values in binary64, a lane each, and are ranked.  Groups
// are kept by estimates too.  Where estimates cannot decide (groups too close, more than
// 64 candidates) the token is computed in binary64 throughout.  12288 tokens of 512
// bfloat16 logits with a bias: 15 us, bound by instruction issue, where binary64 for all
// took 42; 512 tokens of 256 in groups 6.4 (12).
#include "device_types.hpp"
#include "step_ops.hpp"

namespace moe {

namespace {

constexpr int kWaves = 4;
constexpr float kLow = -__builtin_inff();

// Waves exchange values with themselves through LDS: states the order to the compiler.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

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

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  const int i = __float_as_int(v);
  return __int_as_float(__builtin_amdgcn_update_dpp(i, i, CTRL, 0xF, 0xF, false));
}
// Rows of 16 lanes, then lane 15 to the next row and lane 31 to the next half.
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp<0xB1>(v));
  v = fmaxf(v, dpp<0x4E>(v));
  v = fmaxf(v, dpp<0x141>(v));
  v = fmaxf(v, dpp<0x140>(v));
  v = fmaxf(v, dpp<0x142>(v));
  v = fmaxf(v, dpp<0x143>(v));
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
// Lane i's number, i the same in every lane.
__device__ __forceinline__ double lane_of(double v, int i) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, i);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), i);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ float lane_of(float v, int i) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), i));
}

// A number of the same order as v's, -0 as +0.
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b >> 31 ? ~b : b | 0x80000000u;
}

constexpr uint32_t kLeast = 0x00800000u;  // of the lowest finite float
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key >> 31 ? key & 0x7fffffffu : ~key);
}

// A logit as it counts: NaN as minus infinity, plus infinity as the largest float.
__device__ __forceinline__ float logit_of(float v) {
  return v > kLow ? fminf(v, 3.40282347e38f) : kLow;
}

// The score of a logit that is not minus infinity; m and sum are softmax's.
__device__ __forceinline__ double score_of(const RouteArgs &a, float z, double m, double sum) {
  return a.sigmoid ? 1.0 / (1.0 + exp(-(double)z)) : exp((double)z - m) / sum;
}

struct Pick {
  int e;
  double s;  // its score, 0 of an excluded expert
};

// The k picks of a token, lane j's the j-th, all in binary64.  e's of a lane are those of
// z: lane + 64 c.
template <int NC>
__device__ __noinline__ Pick route_exactly(const RouteArgs &a, long long t, double *values) {
  const int lane = threadIdx.x & 63;
  const double ninf = -__builtin_inf();
  double z[NC], s[NC];
  uint64_t key[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int e = lane + 64 * c;
    z[c] = (double)(e < a.E ? logit_of(load1(a.z, a.type, t * a.ldz + e)) : kLow);
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
    if (e < a.E) values[e] = !a.bias && a.best == 2 && v != ninf ? s[c] : v;
  }
  if (a.keep < a.groups) {
    wave_sync();
    const int n = a.E / a.groups;
    double v = ninf;
    if (lane < a.groups) {
      double v1 = ninf, v2 = ninf;
      for (int i = 0; i < n; ++i) {
        const double x = values[lane * n + (i + lane) % n];
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
  return {my_e, my_s};
}

// Elements 4 lane .. 4 lane + 3 of each 256 (V = 4; V = 2 of 128, V = 1 of 64), C of them.
template <int V, int C>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(8))) void route_kernel(RouteArgs a) {
  constexpr int N = V * C;
  __shared__ double exact[kWaves][kRouteMaxExperts];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const long long t = (long long)blockIdx.x * kWaves + wave;
  if (t >= a.T) return;
  float *values = (float *)exact[wave];           // estimates by expert, for the groups
  int *list = (int *)exact[wave] + kRouteMaxExperts;  // candidates
  float z[N], b[N], c[N];
  const auto expert = [&](int i) { return V * lane + 64 * V * (i / V) + i % V; };
  const auto load = [&](const void *p, int type, long long at, float *v, float none) {
#pragma unroll
    for (int u = 0; u < C; ++u) {
      const int e = expert(u * V);
      if (V == 4 && e + 3 < a.E) {
        const float4 f = load4(p, type, at + e);
        v[u * V] = f.x, v[u * V + 1 % V] = f.y, v[u * V + 2 % V] = f.z, v[u * V + 3 % V] = f.w;
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) v[u * V + j] = e + j < a.E ? load1(p, type, at + e + j) : none;
      }
    }
  };
  load(a.z, a.type, t * a.ldz, z, kLow);
  if (a.bias) load(a.bias, kF32, 0, b, kLow);
#pragma unroll
  for (int i = 0; i < N; ++i) z[i] = logit_of(z[i]);
  // softmax's largest logit and sum: the estimates' in float32, the scores' in binary64
  // where the weights or a bias need it
  float m = 0.f, inv = 1.f;
  double sum = 1.0;
  if (!a.sigmoid) {
    m = kLow;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, z[i]);
    m = fmaxf(wave_max(m), -3.40282347e38f);
    if (a.bias || !a.renorm || a.best == 2) {
      sum = 0.0;
#pragma unroll
      for (int i = 0; i < N; ++i) sum += z[i] > kLow ? exp((double)z[i] - (double)m) : 0.0;
      sum = wave_sum(sum);
      inv = sum > 0.0 ? (float)(1.0 / sum) : 1.f;
    }
  }
  // estimates of the scores: off by less than 2^-21 (sigmoid), 2^-19 of the largest score
  // (softmax); with the bias's sum 2^-23 of the value more
  const auto estimate = [&](float v) {
    return a.sigmoid ? __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * v))
                     : __builtin_amdgcn_exp2f(1.44269504f * (v - m)) * inv;
  };
  const float off = a.sigmoid ? 4.8e-7f : 1.9e-6f * inv;
  // (an excluded expert's value is minus infinity)
#pragma unroll
  for (int i = 0; i < N; ++i) c[i] = !a.bias ? z[i] : z[i] > kLow && b[i] > kLow ? estimate(z[i]) + b[i] : kLow;
  const float slack = a.bias ? off : 0.f;
  bool sure = true;
  if (a.keep < a.groups) {
    const int n = a.E / a.groups;
    const bool scores = !a.bias && a.best == 2;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (expert(i) < a.E) values[expert(i)] = scores ? (z[i] > kLow ? estimate(z[i]) : kLow) : c[i];
    wave_sync();
    // as many lanes a group as fit, a power of two
    int per = 64;
    while (per * a.groups > 64) per >>= 1;
    const int g = lane / per, l = lane % per;
    float v1 = kLow, v2 = kLow;
    if (g < a.groups)
      for (int i = l; i < n; i += per) {
        const float x = values[g * n + i];
        v2 = fmaxf(v2, fminf(v1, x));
        v1 = fmaxf(v1, x);
      }
    for (int o = 1; o < per; o <<= 1) {
      const float o1 = __shfl_xor(v1, o, 64), o2 = __shfl_xor(v2, o, 64);
      v2 = fmaxf(fmaxf(v2, o2), fminf(v1, o1));
      v1 = fmaxf(v1, o1);
    }
    // (a pair's sum may pass float32: only a group without a pair is minus infinity)
    const float v = a.best == 2 ? (v2 > kLow ? fmaxf(v1 + v2, -3.40282347e38f) : kLow) : v1;
    int rank = 0;
    for (int o = 0; o < a.groups; ++o) {
      const float x = lane_of(v, o * per);
      rank += x > v || (x == v && o < g);
    }
    const uint64_t kept = __ballot(g < a.groups && rank < a.keep);
    // the last kept and the first left out have to lie apart by more than both are off (a
    // pair's sum by as much as its larger part's rounding, though the parts may cancel)
    const float last = __shfl(v, __ffsll((unsigned long long)__ballot(g < a.groups && rank == a.keep - 1)) - 1, 64);
    const float next = __shfl(v, __ffsll((unsigned long long)__ballot(g < a.groups && rank == a.keep)) - 1, 64);
    const float size = a.best == 2 ? wave_max(v > kLow ? fabsf(v1) + fabsf(v2) : 0.f) : fabsf(last) + fabsf(next);
    const float apart = a.bias || scores ? 2.f * a.best * off + 4.8e-7f * size : 0.f;
    if (apart > 0.f && !(last - next > apart)) sure = next == kLow && last == kLow;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (expert(i) < a.E && !(kept >> (expert(i) / n * per) & 1)) z[i] = c[i] = __builtin_nanf("");
    wave_sync();
  }
  int my_e = 0, count = 0;
  double my_s = 0.0;
  if (sure) {
    // the bits of a float32 that at least k estimates reach, k + 4 at most unless more
    // are equal: by halving, first from half a binary order below the largest on
    float top = kLow;
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, c[i]);
    const auto reach = [&](uint32_t to) {
      const float v = value_of(to);
      int n = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) n += __popcll(__ballot(c[i] >= v));
      return n;
    };
    uint32_t above = __builtin_amdgcn_readfirstlane(order_bits(wave_max(top))) + 1u;
    uint32_t least = above > kLeast + (1u << 22) ? above - (1u << 22) : kLeast;
    int n = reach(least);
    for (int wide = 24; n < a.k && least > kLeast; wide = 32) {
      above = least;
      least = wide == 24 && above > kLeast + (1u << 24) ? above - (1u << 24) : kLeast;
      n = reach(least);
    }
    while (n > a.k + 4 && above - least > 1u) {
      const uint32_t to = least + (above - least) / 2;
      const int got = reach(to);
      if (got >= a.k)
        least = to, n = got;
      else
        above = to;
    }
    float from = value_of(least);
    if (slack > 0.f) from = fmaxf(from - 2.f * slack - 4.8e-7f * fabsf(from), -3.40282347e38f);
    // candidates (excluded experts are none)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool in = c[i] >= from;
      const uint64_t who = __ballot(in);
      const int place = count + __popcll(who & ((1ull << lane) - 1));
      if (in && place < 64) list[place] = expert(i);
      count += __popcll(who);
    }
    sure = count <= 64 && count >= a.k;
  }
  if (sure) {
    wave_sync();
    double value = -__builtin_inf(), s = 0.0;
    int e = kRouteMaxExperts;
    if (lane < count) {
      e = list[lane];
      const float v = logit_of(load1(a.z, a.type, t * a.ldz + e));
      s = score_of(a, v, (double)m, sum);
      value = a.bias ? s + (double)a.bias[e] : (double)v;
    }
    int rank = 0;
    for (int o = 0; o < count; ++o) rank += lane_of(value, o) > value;
    // to the lane of its rank; equal values, which meet there, go by their ids
    wave_sync();
    if (lane < count) list[rank] = lane;
    wave_sync();
    if (__ballot(lane < count && list[rank] != lane)) {
      rank = 0;
      for (int o = 0; o < count; ++o) {
        const double x = lane_of(value, o);
        rank += x > value || (x == value && __builtin_amdgcn_readlane(e, o) < e);
      }
      wave_sync();
      if (lane < count) list[rank] = lane;
      wave_sync();
    }
    const int at = lane < a.k ? list[lane] : 0;
    my_e = __shfl(e, at, 64), my_s = __shfl(s, at, 64);
  } else {
    wave_sync();
    const RouteArgs copy = a;  // (the address of `a` itself would move it to memory for all)
    const Pick p = route_exactly<N>(copy, t, exact[wave]);
    my_e = p.e, my_s = p.s;
  }
  double w = my_s;
  if (a.renorm) {
    const double all = wave_sum(lane < a.k ? my_s : 0.0);
    w = all > 0.0 ? w / all : 0.0;
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

hipError_t launch_route(const RouteArgs &a, hipStream_t s, hipEvent_t start, hipEvent_t stop) {
  auto *k = a.E <= 64    ? route_kernel<1, 1>
            : a.E <= 128 ? route_kernel<2, 1>
            : a.E <= 256 ? route_kernel<4, 1>
                         : route_kernel<4, 2>;
  const dim3 grid((a.T + kWaves - 1) / kWaves), block(64 * kWaves);
  return start ? launch_timed(k, grid, block, s, start, stop, a) : launch(k, grid, block, s, a);
}

}  // namespace moe
