// The next token of each row of logits.  Weights are whole numbers, rint(2^42
// exp((z - max) / temperature)), so that their sums do not depend on the order of
// the additions; positions in the falling order are found digit by digit of the
// logit's ordered bits, with the count and the sum of the tokens at each digit.
#include "device_types.hpp"
#include "step_ops.hpp"

namespace moe {

namespace {

constexpr int kThreads = 1024;
constexpr int kBins = 2048;

// A logit as a number of the same order: NaN is minus infinity (0), plus
// infinity the largest float, -0 is +0.
__device__ __forceinline__ uint32_t order_bits(float v) {
  if (!(v > -__builtin_inff())) return 0u;
  const uint32_t b = __float_as_uint(fminf(v, 3.40282347e38f) + 0.f);
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key >> 31 ? key & 0x7fffffffu : ~key);
}

struct Row {
  float top;       // the largest logit
  double inv;      // 1 / temperature
  __device__ __forceinline__ double ratio(uint32_t key) const {
    return key ? exp(((double)value_of(key) - (double)top) * inv) : 0.0;
  }
  __device__ __forceinline__ uint64_t weight(uint32_t key) const {
    return (uint64_t)rint(ratio(key) * 4398046511104.0);
  }
};

struct Bins {
  uint32_t count[kBins];
  uint64_t sum[kBins];
};

// Position in the falling order: the key of the value there, the tokens and the
// weights before its first equal.
struct Place {
  uint32_t key;
  uint32_t count;
  uint64_t sum;
};

// The first place whose running count (by_count) or sum reaches `target` (>= 1).
template <int TY>
__device__ Place descend(const SampleArgs &a, long long row, const Row &r, bool by_count, uint64_t target,
                         Bins &bins, Place *shared) {
  Place p{0u, 0u, 0ull};
  const int tid = threadIdx.x;
  int shift = 32;
  for (int level = 0; level < 3; ++level) {
    const int bits = level < 2 ? 11 : 10;
    const int above = shift;
    shift -= bits;
    for (int i = tid; i < kBins; i += kThreads) bins.count[i] = 0u, bins.sum[i] = 0ull;
    __syncthreads();
    for (int i = tid; i < a.V; i += kThreads) {
      const uint32_t key = order_bits(load1(a.z, TY, row * a.ldz + i));
      if (above < 32 && (key >> above) != (p.key >> above)) continue;
      const int b = key >> shift & ((1 << bits) - 1);
      atomicAdd(&bins.count[b], 1u);
      atomicAdd((unsigned long long *)&bins.sum[b], (unsigned long long)r.weight(key));
    }
    __syncthreads();
    if (tid == 0) {
      int b = (1 << bits) - 1;
      for (; b > 0; --b) {
        if ((by_count ? p.count + bins.count[b] : p.sum + bins.sum[b]) >= target) break;
        p.count += bins.count[b], p.sum += bins.sum[b];
      }
      p.key |= (uint32_t)b << shift;
      *shared = p;
    }
    __syncthreads();
    p = *shared;
    __syncthreads();
  }
  return p;
}

template <int TY>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleArgs a) {
  __shared__ Bins bins;
  __shared__ Place place;
  __shared__ uint32_t part[kThreads / 64];
  __shared__ unsigned long long total, least;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const long long row = blockIdx.x;
  uint32_t top = 0;
  for (int i = tid; i < a.V; i += kThreads) top = max(top, order_bits(load1(a.z, TY, row * a.ldz + i)));
  for (int off = 32; off >= 1; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, 64));
  if (lane == 0) part[wave] = top;
  if (tid == 0) total = least = 0ull;
  __syncthreads();
  for (int i = 0; i < kThreads / 64; ++i) top = max(top, part[i]);
  __syncthreads();
  if (top == 0u) {
    if (tid == 0) {
      a.token[row] = -1;
      if (a.prob) a.prob[row] = 0.f;
    }
    return;
  }
  const double temp = a.temperatures ? (double)a.temperatures[row] : a.temperature;
  const double share = a.top_ps ? (double)a.top_ps[row] : a.top_p;
  const double min_p = a.min_ps ? (double)a.min_ps[row] : a.min_p;
  const int k = a.top_ks ? a.top_ks[row] : a.top_k;
  double u = (double)a.u[row];
  u = u >= 0.0 ? fmin(u, 1.0) : 0.0;
  uint32_t key = top;
  uint32_t rank = 0;
  double prob = 1.0;
  if (temp > 0.0) {
    const Row r{value_of(top), 1.0 / temp};
    uint64_t all = 0, big = 0;
    const double floor_p = min_p > 0.0 ? fmin(min_p, 1.0) : 0.0;  // NaN keeps all
    for (int i = tid; i < a.V; i += kThreads) {
      const uint32_t b = order_bits(load1(a.z, TY, row * a.ldz + i));
      const uint64_t w = r.weight(b);
      all += w;
      if (r.ratio(b) >= floor_p) big += w;
    }
    for (int off = 32; off >= 1; off >>= 1) all += __shfl_xor(all, off, 64), big += __shfl_xor(big, off, 64);
    if (lane == 0) atomicAdd(&total, (unsigned long long)all), atomicAdd(&least, (unsigned long long)big);
    __syncthreads();
    uint64_t kept = total;
    if (k > 0 && k < a.V) {
      const Place p = descend<TY>(a, row, r, true, (uint64_t)k, bins, &place);
      kept = min((unsigned long long)kept, (unsigned long long)(p.sum + (k - p.count) * r.weight(p.key)));
    }
    if (share < 1.0) {
      const uint64_t target = max((uint64_t)ceil(fmax(share, 0.0) * (double)kept), (uint64_t)1);
      const Place p = descend<TY>(a, row, r, false, target, bins, &place);
      const uint64_t w = max(r.weight(p.key), (uint64_t)1);
      kept = min((unsigned long long)kept, (unsigned long long)(p.sum + (target - p.sum + w - 1) / w * w));
    }
    kept = min((unsigned long long)kept, least);
    const uint64_t target = min((uint64_t)(u * (double)kept), kept - 1) + 1;
    const Place p = descend<TY>(a, row, r, false, target, bins, &place);
    key = p.key;
    rank = (uint32_t)((target - 1 - p.sum) / max(r.weight(key), (uint64_t)1));
    prob = r.ratio(key) * 4398046511104.0 / (double)kept;
  }
  // the rank-th token of that value, by ids
  uint32_t before = 0;
  for (int i0 = 0; i0 < a.V; i0 += kThreads) {
    const int i = i0 + tid;
    const bool hit = i < a.V && order_bits(load1(a.z, TY, row * a.ldz + i)) == key;
    const uint64_t m = __ballot(hit);
    if (lane == 0) part[wave] = __popcll(m);
    __syncthreads();
    uint32_t mine = before, all = 0;
    for (int j = 0; j < kThreads / 64; ++j) {
      if (j < wave) mine += part[j];
      all += part[j];
    }
    if (hit && mine + __popcll(m & ((1ull << lane) - 1)) == rank) {
      a.token[row] = i;
      if (a.prob) a.prob[row] = (float)prob;
    }
    before += all;
    __syncthreads();
    if (before > rank) break;
  }
}

}  // namespace

size_t sample_ws_bytes(int, int) { return 0; }

hipError_t launch_sample(const SampleArgs &a, hipStream_t s) {
  auto *k = a.type == kF32 ? sample_kernel<kF32> : a.type == kBf16 ? sample_kernel<kBf16> : sample_kernel<kF16>;
  return launch(k, dim3(a.T), dim3(kThreads), s, a);
}

}  // namespace moe
