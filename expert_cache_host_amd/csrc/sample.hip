// The next token of each row of logits.
//
// Weights are whole numbers, rint(2^42 exp((z - max) / temperature)), so that sums do
// not depend on the order of additions and every border is decided alike wherever it
// is computed.  A row of up to kCap tokens is sorted in LDS.  A longer one takes four
// launches, the first three over `segments` workgroups a row:
//   tops      the largest logit (and its first id);
//   bins      count and weight of the tokens by their distance from it, in kBins bins;
//   gather    from the bins' running sums: in which bins the borders of top-k, top-p
//             and min-p and the token itself can lie (each border is known to a bin,
//             which bounds the next); the tokens of those bins, a few hundred mostly,
//             are gathered;
//   resolve   one workgroup a row sorts them, and the running sums settle the borders
//             and the token exactly.
// Where they are more than kCap (nearly flat rows), resolve finds the borders digit by
// digit of the logits' ordered bits over the whole row: right, and slow.
#include "device_types.hpp"
#include "step_ops.hpp"

namespace moe {

namespace {

constexpr int kCap = 2048;       // tokens sorted in LDS
constexpr int kBins = 2048;
constexpr int kMaxSegments = 128;
constexpr int kScan = 512;       // threads of the first three kernels
constexpr double kOne = 4398046511104.0;  // 2^42: the largest token's weight

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

// exp(-d) for d >= 0 by its series around the nearest multiple of ln 2; the terms left
// out are below 2^-56 of it.  0 from 40 on, where a weight is 0 anyway.
__device__ __forceinline__ double exp_minus(double d) {
#pragma clang fp contract(off)
  if (!(d < 40.0)) return 0.0;
  const double n = rint(d * 1.4426950408889634);
  // ln 2 in two parts, the first with zeros behind so that n times it is exact
  double r = fma(n, 0x1.62e42fefap-1, -d);
  r = fma(n, 0x1.cf79abc9e3b39p-40, r);
  double p = 1.0 / 6227020800.0;
  p = fma(p, r, 1.0 / 479001600.0);
  p = fma(p, r, 1.0 / 39916800.0);
  p = fma(p, r, 1.0 / 3628800.0);
  p = fma(p, r, 1.0 / 362880.0);
  p = fma(p, r, 1.0 / 40320.0);
  p = fma(p, r, 1.0 / 5040.0);
  p = fma(p, r, 1.0 / 720.0);
  p = fma(p, r, 1.0 / 120.0);
  p = fma(p, r, 1.0 / 24.0);
  p = fma(p, r, 1.0 / 6.0);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  return __builtin_bit_cast(double, __builtin_bit_cast(int64_t, p) - ((int64_t)(int)n << 52));
}

// A row's settings and its largest logit.
struct Row {
  double top, inv;           // largest logit, 1 / temperature
  double share, least, u;    // top-p (1: all), min-p (0: all), the random number
  int k;                     // top-k (0: all)
  bool greedy;
  __device__ __forceinline__ Row(const SampleArgs &a, long long row, uint32_t top_key) {
    const double t = a.temperatures ? (double)a.temperatures[row] : a.temperature;
    greedy = !(t > 0.0);
    inv = greedy ? 1.0 : 1.0 / t;
    top = top_key ? (double)value_of(top_key) : 0.0;
    const double p = a.top_ps ? (double)a.top_ps[row] : a.top_p;
    share = p < 1.0 ? fmax(p, 0.0) : 1.0;  // NaN keeps all
    const double m = a.min_ps ? (double)a.min_ps[row] : a.min_p;
    least = m > 0.0 ? fmin(m, 1.0) : 0.0;
    k = max(a.top_ks ? a.top_ks[row] : a.top_k, 0);
    const double v = (double)a.u[row];
    u = v >= 0.0 ? fmin(v, 1.0) : 0.0;
  }
  // how far below the largest, in temperatures
  __device__ __forceinline__ double distance(uint32_t key) const {
#pragma clang fp contract(off)
    return key ? (top - (double)value_of(key)) * inv : __builtin_inf();
  }
  __device__ __forceinline__ uint64_t weight(double d) const { return (uint64_t)rint(exp_minus(d) * kOne); }
  // positions (1, 2, ...) in the running sums
  __device__ __forceinline__ uint64_t share_of(uint64_t sum) const {
    const uint64_t t = (uint64_t)ceil(share * (double)sum);
    return t < 1 ? 1 : t < sum ? t : sum;
  }
  __device__ __forceinline__ uint64_t draw(uint64_t kept) const {
    const uint64_t t = (uint64_t)(u * (double)kept);
    return (t < kept ? t : kept - 1) + 1;
  }
};

// Bins: 1/128 of a temperature wide up to 12, then 5/128 up to 32.  Tokens of weight 0
// (from 29.8 on) lie in none.
__device__ __forceinline__ int bin_of(double d) {
#pragma clang fp contract(off)
  return d < 12.0 ? (int)(d * 128.0) : 1536 + min((int)((d - 12.0) * 25.6), 511);
}

// What a row has in the workspace.
struct Space {
  unsigned long long tops[kMaxSegments];  // key << 32 | ~id
  unsigned long long sum[kBins];
  unsigned long long near[kCap];          // gathered tokens, as tops
  uint32_t count[kBins];
  uint32_t gathered, pad[3];
};

__device__ __forceinline__ unsigned long long token_of(uint32_t key, int id) {
  return (unsigned long long)key << 32 | (uint32_t)~id;
}

// Calls f(key, id) for a thread's tokens of [lo, hi) of the row, four at a time.
template <int TY, int THREADS, class F>
__device__ __forceinline__ void each_token(const SampleArgs &a, long long row, int lo, int hi, F f) {
  const long long at = row * a.ldz;
  int i = lo + 4 * threadIdx.x;
  for (; i + 3 < hi; i += 4 * THREADS) {
    const float4 v = load4(a.z, TY, at + i);
    f(order_bits(v.x), i), f(order_bits(v.y), i + 1), f(order_bits(v.z), i + 2), f(order_bits(v.w), i + 3);
  }
  for (; i < hi; ++i) f(order_bits(load1(a.z, TY, at + i)), i);
}

template <class T>
__device__ __forceinline__ T wave_max(T v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const T o = __shfl_xor(v, off, 64);
    v = o > v ? o : v;
  }
  return v;
}

// Sum of v over the threads before this one; `total` gets that of all.  `part` holds a
// number a wave.
template <class T, int THREADS>
__device__ __forceinline__ T block_before(T v, T *part, T &total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  T run = v;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const T o = __shfl_up(run, off, 64);
    if (lane >= off) run += o;
  }
  if (lane == 63) part[wave] = run;
  __syncthreads();
  T before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 64; ++i) {
    if (i < wave) before += part[i];
    total += part[i];
  }
  return before + run - v;
}

__device__ __forceinline__ void segment(const SampleArgs &a, int &lo, int &hi) {
  const int n = ((a.V + (int)gridDim.x - 1) / (int)gridDim.x + 3) & ~3;
  lo = min((int)blockIdx.x * n, a.V), hi = min(lo + n, a.V);
}

__device__ __forceinline__ unsigned long long top_of(const Space &s, int segments) {
  unsigned long long t = 0;
  for (int i = threadIdx.x & 63; i < segments; i += 64) t = max(t, s.tops[i]);
  return wave_max(t);
}

template <int TY>
__global__ __launch_bounds__(kScan) void sample_tops_kernel(SampleArgs a) {
  __shared__ unsigned long long part[kScan / 64];
  Space &s = ((Space *)a.ws)[blockIdx.y];
  int lo, hi;
  segment(a, lo, hi);
  unsigned long long t = 0;
  each_token<TY, kScan>(a, blockIdx.y, lo, hi, [&](uint32_t key, int id) {
    if (key) t = max(t, token_of(key, id));
  });
  t = wave_max(t);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = t;
  // what the next launches add to
  for (int i = blockIdx.x * kScan + threadIdx.x; i < kBins; i += gridDim.x * kScan) s.sum[i] = 0ull, s.count[i] = 0u;
  if (blockIdx.x == 0 && threadIdx.x == 0) s.gathered = 0u;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kScan / 64; ++i) t = max(t, part[i]);
    s.tops[blockIdx.x] = t;
  }
}

template <int TY>
__global__ __launch_bounds__(kScan) void sample_bins_kernel(SampleArgs a) {
  __shared__ unsigned long long sum[kBins];
  __shared__ uint32_t count[kBins];
  Space &s = ((Space *)a.ws)[blockIdx.y];
  for (int i = threadIdx.x; i < kBins; i += kScan) sum[i] = 0ull, count[i] = 0u;
  const uint32_t top = (uint32_t)(top_of(s, gridDim.x) >> 32);
  const Row r(a, blockIdx.y, top);
  if (!top || r.greedy) return;
  __syncthreads();
  int lo, hi;
  segment(a, lo, hi);
  each_token<TY, kScan>(a, blockIdx.y, lo, hi, [&](uint32_t key, int) {
    const double d = r.distance(key);
    const unsigned long long w = r.weight(d);
    if (w) {
      const int b = bin_of(d);
      atomicAdd(&count[b], 1u);
      atomicAdd(&sum[b], w);
    }
  });
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += kScan)
    if (count[i]) {
      atomicAdd(&s.count[i], count[i]);
      atomicAdd(&s.sum[i], sum[i]);
    }
}

template <int TY>
__global__ __launch_bounds__(kScan) void sample_gather_kernel(SampleArgs a) {
  constexpr int kMine = kBins / kScan;
  __shared__ unsigned long long part64[kScan / 64], ends[3], found[kCap];
  __shared__ uint32_t part32[kScan / 64], wanted[kBins / 32], mine, base;
  Space &s = ((Space *)a.ws)[blockIdx.y];
  const int tid = threadIdx.x;
  const uint32_t top = (uint32_t)(top_of(s, gridDim.x) >> 32);
  const Row r(a, blockIdx.y, top);
  if (!top || r.greedy) return;
  if (tid < kBins / 32) wanted[tid] = 0u;
  if (tid == 0) mine = 0u;
  // running counts and sums at the ends of this thread's bins
  uint32_t c[kMine + 1], tokens;
  unsigned long long w[kMine + 1], total;
  c[0] = 0u, w[0] = 0ull;
#pragma unroll
  for (int j = 0; j < kMine; ++j) c[j + 1] = c[j] + s.count[kMine * tid + j], w[j + 1] = w[j] + s.sum[kMine * tid + j];
  const uint32_t c0 = block_before<uint32_t, kScan>(c[kMine], part32, tokens);
  const unsigned long long w0 = block_before<unsigned long long, kScan>(w[kMine], part64, total);
#pragma unroll
  for (int j = 0; j <= kMine; ++j) c[j] += c0, w[j] += w0;
  const auto want = [&](int b) { atomicOr(&wanted[b >> 5], 1u << (b & 31)); };
  // what is kept lies in [lo, hi]
  unsigned long long lo = total, hi = total;
  if (r.k > 0 && (uint32_t)r.k < tokens) {
#pragma unroll
    for (int j = 0; j < kMine; ++j)
      if (c[j] < (uint32_t)r.k && (uint32_t)r.k <= c[j + 1]) want(kMine * tid + j), ends[0] = w[j], ends[1] = w[j + 1];
    __syncthreads();
    lo = max(ends[0], 1ull), hi = ends[1];
  }
  if (r.share < 1.0) {
    const unsigned long long from = r.share_of(lo), to = r.share_of(hi);
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      if (w[j] < to && w[j + 1] >= from) want(kMine * tid + j);
      if (w[j] < to && w[j + 1] >= to) ends[2] = w[j + 1];
    }
    __syncthreads();
    lo = min(lo, from), hi = min(hi, ends[2]);
  }
  if (r.least > 0.0) {
    // the border's distance, and the bins on either side of what rounding may make of it
    const double d = -log(r.least);
    const int b0 = bin_of(fmin(fmax(d - 1e-9, 0.0), 31.9)), b1 = bin_of(fmin(d + 1e-9, 31.9));
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      const int b = kMine * tid + j;
      if (b >= b0 && b <= b1) want(b);
      if (b == b0) ends[0] = w[j];
      if (b == b1) ends[1] = w[j + 1];
    }
    __syncthreads();
    lo = min(lo, max(ends[0], 1ull)), hi = min(hi, ends[1]);
  }
  const unsigned long long from = r.draw(lo), to = r.draw(hi);
#pragma unroll
  for (int j = 0; j < kMine; ++j)
    if (w[j] < to && w[j + 1] >= from) want(kMine * tid + j);
  __syncthreads();
  // (those past kCap are only counted)
  int first, last;
  segment(a, first, last);
  each_token<TY, kScan>(a, blockIdx.y, first, last, [&](uint32_t key, int id) {
    const double d = r.distance(key);
    if (!(d < 30.0)) return;
    const int b = bin_of(d);
    if (!(wanted[b >> 5] >> (b & 31) & 1u) || !r.weight(d)) return;
    const uint32_t i = atomicAdd(&mine, 1u);
    if (i < kCap) found[i] = token_of(key, id);
  });
  __syncthreads();
  const uint32_t n = mine;
  if (n == 0u) return;
  if (tid == 0) base = atomicAdd(&s.gathered, n);
  __syncthreads();
  if (base + n > kCap) return;
  for (uint32_t i = tid; i < n; i += kScan) s.near[base + i] = found[i];
}

// Sorts n (a power of two, at least 128) numbers in LDS, the largest first.  A pair's
// lanes lie in one wave while the distance is below 128: no workgroup barrier is
// needed between those steps.
template <int THREADS>
__device__ void sort_falling(unsigned long long *x, int n) {
  for (int size = 2; size <= n; size <<= 1)
    for (int step = size >> 1; step >= 1; step >>= 1) {
      for (int p = threadIdx.x; p < n / 2; p += THREADS) {
        const int i = 2 * p - (p & (step - 1));
        const unsigned long long u = x[i], v = x[i + step];
        if ((u < v) == ((i & size) == 0)) x[i] = v, x[i + step] = u;
      }
      if (step > 64 || (step == 1 && size >= 128))
        __syncthreads();
      else {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      }
    }
  __syncthreads();
}

__device__ __forceinline__ void give(const SampleArgs &a, long long row, int token, double prob) {
  a.token[row] = token;
  if (a.prob) a.prob[row] = (float)prob;
}

// The row's token from sorted tokens x[0..n): all of the row's, or (kBinned) those of
// some bins, with the row's sums and counts before each bin in before and rank.
// total and tokens are the row's; least_before the sum before the first bin in which
// min-p's border can lie.
template <int THREADS, bool kBinned>
__device__ void settle(const SampleArgs &a, long long row, const Row &r, const unsigned long long *x, int n,
                       unsigned long long *before, uint32_t *rank, unsigned long long total, uint32_t tokens,
                       unsigned long long least_before) {
  constexpr int kMine = kCap / THREADS;
  __shared__ unsigned long long part[THREADS / 64], kept;
  const int tid = threadIdx.x;
  uint32_t key[kMine];
  double d[kMine];
  unsigned long long w[kMine], sum = 0, all;
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int i = kMine * tid + j;
    key[j] = i < n ? (uint32_t)(x[i] >> 32) : 0u;
    d[j] = r.distance(key[j]);
    w[j] = r.weight(d[j]);
    sum += w[j];
  }
  unsigned long long at = block_before<unsigned long long, THREADS>(sum, part, all);
  if constexpr (kBinned) {
    // a bin's first gathered token: what its tokens' places and sums are off by
    unsigned long long e = at;
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      const int i = kMine * tid + j;
      if (w[j]) {
        const int b = bin_of(d[j]);
        if (i == 0 || bin_of(r.distance((uint32_t)(x[i - 1] >> 32))) != b) before[b] -= e, rank[b] -= (uint32_t)i;
      }
      e += w[j];
    }
    __syncthreads();
  }
  unsigned long long to[kMine];
  uint32_t place[kMine];
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int b = kBinned && w[j] ? bin_of(d[j]) : 0;
    at += w[j];
    to[j] = at + (kBinned ? before[b] : 0ull);
    place[j] = (uint32_t)(kMine * tid + j) + (kBinned ? rank[b] : 0u);
  }
  if (tid == 0) kept = total;
  __syncthreads();
  if (r.k > 0 && (uint32_t)r.k < tokens) {
#pragma unroll
    for (int j = 0; j < kMine; ++j)
      if (w[j] && place[j] == (uint32_t)r.k - 1) kept = to[j];
    __syncthreads();
  }
  unsigned long long keep = kept;
  if (r.share < 1.0) {
    const unsigned long long p = r.share_of(keep);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMine; ++j)
      if (w[j] && to[j] >= p && to[j] - w[j] < p) kept = to[j];
    __syncthreads();
    keep = min(keep, kept);
  }
  if (r.least > 0.0) {
    __syncthreads();
    if (tid == 0) kept = least_before;
    __syncthreads();
    unsigned long long m = 0;
#pragma unroll
    for (int j = 0; j < kMine; ++j)
      if (w[j] && exp_minus(d[j]) >= r.least) m = max(m, to[j]);
    if (m) atomicMax(&kept, m);
    __syncthreads();
    keep = min(keep, kept);
  }
  const unsigned long long p = r.draw(keep);
#pragma unroll
  for (int j = 0; j < kMine; ++j)
    if (w[j] && to[j] >= p && to[j] - w[j] < p)
      give(a, row, (int)~(uint32_t)x[kMine * tid + j], exp_minus(d[j]) * kOne / (double)keep);
}

// ---- rows whose gathered tokens are too many

// The value at a position of the running counts or sums: its key, and the tokens and
// weights before its first equal.
struct Place {
  uint32_t key, count;
  unsigned long long sum;
};

template <int TY, int THREADS>
__device__ Place descend(const SampleArgs &a, long long row, const Row &r, bool by_count, unsigned long long target,
                         unsigned long long *sum, uint32_t *count, Place *shared) {
  Place p{0u, 0u, 0ull};
  int shift = 32;
  for (int level = 0; level < 3; ++level) {
    const int bits = level < 2 ? 11 : 10, above = shift;
    shift -= bits;
    for (int i = threadIdx.x; i < kBins; i += THREADS) count[i] = 0u, sum[i] = 0ull;
    __syncthreads();
    each_token<TY, THREADS>(a, row, 0, a.V, [&](uint32_t key, int) {
      if (above < 32 && (key >> above) != (p.key >> above)) return;
      const unsigned long long w = r.weight(r.distance(key));
      if (!w) return;
      const int b = key >> shift & ((1 << bits) - 1);
      atomicAdd(&count[b], 1u);
      atomicAdd(&sum[b], w);
    });
    __syncthreads();
    if (threadIdx.x == 0) {
      int b = (1 << bits) - 1;
      for (; b > 0; --b) {
        if ((by_count ? p.count + count[b] : p.sum + sum[b]) >= target) break;
        p.count += count[b], p.sum += sum[b];
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

template <int TY, int THREADS>
__device__ void settle_by_digits(const SampleArgs &a, long long row, const Row &r, unsigned long long total,
                                 uint32_t tokens, unsigned long long *sum, uint32_t *count) {
  __shared__ Place shared;
  __shared__ unsigned long long kept;
  __shared__ uint32_t part[THREADS / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  unsigned long long keep = total;
  if (r.k > 0 && (uint32_t)r.k < tokens) {
    const Place p = descend<TY, THREADS>(a, row, r, true, (unsigned long long)r.k, sum, count, &shared);
    keep = p.sum + (r.k - p.count) * r.weight(r.distance(p.key));
  }
  if (r.share < 1.0) {
    const unsigned long long t = r.share_of(keep);
    const Place p = descend<TY, THREADS>(a, row, r, false, t, sum, count, &shared);
    const unsigned long long w = r.weight(r.distance(p.key));
    keep = min(keep, p.sum + (t - p.sum + w - 1) / w * w);
  }
  if (r.least > 0.0) {
    if (tid == 0) kept = 0ull;
    __syncthreads();
    unsigned long long m = 0;
    each_token<TY, THREADS>(a, row, 0, a.V, [&](uint32_t key, int) {
      const double d = r.distance(key);
      if (exp_minus(d) >= r.least) m += r.weight(d);
    });
    if (m) atomicAdd(&kept, m);
    __syncthreads();
    keep = min(keep, kept);
  }
  const unsigned long long t = r.draw(keep);
  const Place p = descend<TY, THREADS>(a, row, r, false, t, sum, count, &shared);
  const unsigned long long w = r.weight(r.distance(p.key));
  // the nth of the equal ones, by ids
  const uint32_t nth = (uint32_t)((t - 1 - p.sum) / w);
  uint32_t before = 0;
  for (int i0 = 0; i0 < a.V && before <= nth; i0 += THREADS) {
    const int i = i0 + tid;
    const bool hit = i < a.V && order_bits(load1(a.z, TY, row * a.ldz + i)) == p.key;
    const uint64_t m = __ballot(hit);
    if (lane == 0) part[wave] = __popcll(m);
    __syncthreads();
    uint32_t mine = before;
    for (int j = 0; j < THREADS / 64; ++j) {
      if (j < wave) mine += part[j];
      before += part[j];
    }
    if (hit && mine + __popcll(m & ((1ull << lane) - 1)) == nth)
      give(a, row, i, exp_minus(r.distance(p.key)) * kOne / (double)keep);
    __syncthreads();
  }
}

constexpr int kResolve = 1024;

template <int TY>
__global__ __launch_bounds__(kResolve) void sample_resolve_kernel(SampleArgs a, int segments) {
  constexpr int kMine = kBins / kResolve;
  __shared__ unsigned long long sum[kBins], x[kCap], part64[kResolve / 64], least_before;
  __shared__ uint32_t count[kBins], part32[kResolve / 64];
  Space &s = ((Space *)a.ws)[blockIdx.x];
  const long long row = blockIdx.x;
  const int tid = threadIdx.x;
  const unsigned long long first = top_of(s, segments);
  const Row r(a, row, (uint32_t)(first >> 32));
  if (!first || r.greedy) {
    if (tid == 0) give(a, row, first ? (int)~(uint32_t)first : -1, first ? 1.0 : 0.0);
    return;
  }
  uint32_t c[kMine], mine32 = 0, tokens;
  unsigned long long w[kMine], mine64 = 0, total;
#pragma unroll
  for (int j = 0; j < kMine; ++j)
    c[j] = s.count[kMine * tid + j], w[j] = s.sum[kMine * tid + j], mine32 += c[j], mine64 += w[j];
  uint32_t c0 = block_before<uint32_t, kResolve>(mine32, part32, tokens);
  unsigned long long w0 = block_before<unsigned long long, kResolve>(mine64, part64, total);
  const int n = (int)s.gathered;
  if (n > kCap) {
    settle_by_digits<TY, kResolve>(a, row, r, total, tokens, sum, count);
    return;
  }
  const int b0 = r.least > 0.0 ? bin_of(fmin(fmax(-log(r.least) - 1e-9, 0.0), 31.9)) : 0;
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int b = kMine * tid + j;
    if (b == b0) least_before = w0;
    sum[b] = w0, count[b] = c0;
    w0 += w[j], c0 += c[j];
  }
  int size = 128;
  while (size < n) size *= 2;
  for (int i = tid; i < size; i += kResolve) x[i] = i < n ? s.near[i] : 0ull;
  __syncthreads();
  sort_falling<kResolve>(x, size);
  settle<kResolve, true>(a, row, r, x, n, sum, count, total, tokens, least_before);
}

// Rows of up to kCap tokens: all of them sorted.
constexpr int kShort = 512;

template <int TY>
__global__ __launch_bounds__(kShort) void sample_short_kernel(SampleArgs a, int size) {
  __shared__ unsigned long long x[kCap], part64[kShort / 64];
  __shared__ uint32_t part32[kShort / 64];
  const long long row = blockIdx.x;
  const int tid = threadIdx.x;
  for (int i = tid; i < size; i += kShort) {
    const uint32_t key = i < a.V ? order_bits(load1(a.z, TY, row * a.ldz + i)) : 0u;
    x[i] = key ? token_of(key, i) : 0ull;
  }
  __syncthreads();
  sort_falling<kShort>(x, size);
  const unsigned long long first = x[0];
  const Row r(a, row, (uint32_t)(first >> 32));
  if (!first || r.greedy) {
    if (tid == 0) give(a, row, first ? (int)~(uint32_t)first : -1, first ? 1.0 : 0.0);
    return;
  }
  uint32_t mine32 = 0, tokens;
  unsigned long long mine64 = 0, total;
  for (int i = tid; i < a.V; i += kShort) {
    const unsigned long long w = r.weight(r.distance((uint32_t)(x[i] >> 32)));
    mine32 += w != 0, mine64 += w;
  }
  (void)block_before<uint32_t, kShort>(mine32, part32, tokens);
  (void)block_before<unsigned long long, kShort>(mine64, part64, total);
  __syncthreads();
  settle<kShort, false>(a, row, r, x, a.V, nullptr, nullptr, total, tokens, 0ull);
}

int segments_of(int T, int V) {
  int n = 512 / (T < 1 ? 1 : T);
  const int most = (V + 4095) / 4096;
  n = n < most ? n : most;
  return n < 1 ? 1 : n < kMaxSegments ? n : kMaxSegments;
}

template <int TY>
hipError_t launch_type(const SampleArgs &a, hipStream_t s) {
  if (a.V <= kCap) {
    int size = 128;
    while (size < a.V) size *= 2;
    return launch(sample_short_kernel<TY>, dim3(a.T), dim3(kShort), s, a, size);
  }
  const int n = segments_of(a.T, a.V);
  hipError_t e = launch(sample_tops_kernel<TY>, dim3(n, a.T), dim3(kScan), s, a);
  if (e == hipSuccess) e = launch(sample_bins_kernel<TY>, dim3(n, a.T), dim3(kScan), s, a);
  if (e == hipSuccess) e = launch(sample_gather_kernel<TY>, dim3(n, a.T), dim3(kScan), s, a);
  if (e == hipSuccess) e = launch(sample_resolve_kernel<TY>, dim3(a.T), dim3(kResolve), s, a, n);
  return e;
}

}  // namespace

size_t sample_ws_bytes(int T, int V) { return V <= kCap ? 0 : (size_t)T * sizeof(Space); }

hipError_t launch_sample(const SampleArgs &a, hipStream_t s) {
  return a.type == kF32 ? launch_type<kF32>(a, s) : a.type == kBf16 ? launch_type<kBf16>(a, s) : launch_type<kF16>(a, s);
}

}  // namespace moe
