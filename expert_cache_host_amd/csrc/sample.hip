// The next token of each row of logits.
//
// Weights are whole numbers, rint(2^42 exp((z - max) / temperature)), so that sums do
// not depend on the order of additions and every border is decided alike wherever it
// is computed.  Count and weight of the tokens are summed by their distance from the
// largest logit, in kBins bins; from the bins' running sums follows in which of them
// the borders of top-k, top-p and min-p and the token itself can lie (each border is
// known to a bin, which bounds the next); the tokens of those bins, a few hundred
// mostly, are gathered and sorted, and settle borders and token exactly.  Where they
// are more than kCap (nearly flat rows), the borders are found digit by digit of the
// logits' ordered bits over the whole row: right, and slow.
//
// A row of up to kShortRow tokens takes one workgroup and one launch.  A longer one
// takes four: its largest logit, its bins and the gathering each over many workgroups,
// the rest in one.  Measured: 36 rows of 645 in 11 us; one of 131072 in 24 (3 + 5 + 10 +
// 7: every workgroup of the gathering, and the last launch again, reads the 24 KB of
// bins, sums them up and searches the borders, which takes longer than its tokens do);
// 64 of 262144 float32 in 68 (13 + 23 + 24 + 9).  There the first pass reads the logits at
// 5.2 TB/s; in the second vector instructions, 28 a token, take 0.68 of the CUs' cycles
// and LDS 0.41, half of it bank conflicts; in the third they take 0.39 and 0.13, the rest
// is the borders' search and its waiting.  Rows settled by digits: 0.4 to 2.5 ms.
#include "device_types.hpp"
#include "step_ops.hpp"

namespace moe {

namespace {

constexpr int kCap = 2048;        // tokens sorted in LDS
constexpr int kFew = 256;         // of which so many by counting
constexpr int kBins = 2048;
constexpr int kMaxSegments = 128;
constexpr int kScan = 512;        // threads of a workgroup
constexpr int kShortRow = 16384;

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

// exp(-d) for 0 <= d < 40 by its series around the nearest multiple of ln 2; the terms
// left out are below 2^-56 of it.
__device__ __forceinline__ double exp_minus(double d) {
#pragma clang fp contract(off)
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

// Distances from the largest logit count in 128ths of a temperature; weights are 0 from
// kFar on (30 temperatures).
constexpr double kFar = 3840.0;

// 2^42 exp(-i / 4) and exp(-i / 128), made by every workgroup: with them a weight takes
// a polynomial of degree 5 (the terms left out are below 2^-57).
constexpr int kPlaces = 3841;             // 128ths up to kFar
constexpr double kOne = 4398046511104.0;  // 2^42: the largest token's weight
struct Table {
  double quarter[kPlaces / 32 + 1], part[32];
  __device__ __forceinline__ double at(int t) const {
#pragma clang fp contract(off)
    return quarter[t >> 5] * part[t & 31];
  }
  // (the workgroup meets before it is used)
  __device__ __forceinline__ void fill() {
    const int i = threadIdx.x;
    if (i < 32)
      part[i] = exp_minus(i * 0.0078125);
    else if (i - 32 <= kPlaces / 32)
      quarter[i - 32] = exp_minus((i - 32) * 0.25) * kOne;
  }
};

// The bin of the tokens nearest to distance t: bins are 1/128 of a temperature wide up to
// 10, then 1/32.
__device__ __forceinline__ int bin_of(int t) { return min(t, 960 + (t >> 2)); }
// Where a bin starts.
__device__ __forceinline__ double bin_start(int b) { return (b < 1280 ? b : 4 * (b - 960)) - 0.5; }

// A distance below kFar: its bin, and the two factors of its weight.
struct Spot {
  int bin;
  double whole, part;
  __device__ __forceinline__ Spot(double d, const Table &table) {
#pragma clang fp contract(off)
    // the sum with 1.5 * 2^52 rounds to a whole number, which its low bits are
    const double u = d + 6755399441055744.0;
    const int t = (int)(uint32_t)__builtin_bit_cast(uint64_t, u);
    bin = bin_of(t);
    const double f = d - (u - 6755399441055744.0);
    // exp(-f / 128)
    double p = -1.0 / (120.0 * 34359738368.0);
    p = fma(p, f, 1.0 / (24.0 * 268435456.0));
    p = fma(p, f, -1.0 / (6.0 * 2097152.0));
    p = fma(p, f, 0.5 / 16384.0);
    p = fma(p, f, -1.0 / 128.0);
    part = fma(p, f, 1.0);
    whole = table.at(t);
  }
  // rounded to a whole number by the sum with 2^52
  __device__ __forceinline__ unsigned long long weight() const {
    return __builtin_bit_cast(unsigned long long, fma(whole, part, 4503599627370496.0)) - 0x4330000000000000ull;
  }
  __device__ __forceinline__ double ratio() const { return whole * part * (1.0 / kOne); }
};

// A row's settings and its largest logit.
struct Row {
  double top, temp, inv;     // largest logit, a 128th of the temperature and its inverse
  double share, least, u;    // top-p (1: all), min-p (0: all), the random number
  int k;                     // top-k (0: all)
  bool greedy;
  __device__ __forceinline__ Row(const SampleArgs &a, long long row) {
    const double t = a.temperatures ? (double)a.temperatures[row] : a.temperature;
    greedy = !(t > 0.0);
    // (below 1e-300, whose inverse is finite, unequal float32 logits have weights 1 and 0 alike)
    temp = fmax(t, 1e-300) * 0.0078125;
    inv = greedy ? 1.0 : 1.0 / temp;
    const double p = a.top_ps ? (double)a.top_ps[row] : a.top_p;
    share = p < 1.0 ? fmax(p, 0.0) : 1.0;  // NaN keeps all
    const double m = a.min_ps ? (double)a.min_ps[row] : a.min_p;
    least = m > 0.0 ? fmin(m, 1.0) : 0.0;
    k = max(a.top_ks ? a.top_ks[row] : a.top_k, 0);
    const double v = (double)a.u[row];
    u = v >= 0.0 ? fmin(v, 1.0) : 0.0;
  }
  // how far below the largest (minus infinity and NaN: not below kFar)
  __device__ __forceinline__ double distance(float v) const {
#pragma clang fp contract(off)
    return (top - (double)v) * inv;
  }
  // positions (1, 2, ...) in the running sums
  __device__ __forceinline__ unsigned long long share_of(unsigned long long sum) const {
    const unsigned long long t = (unsigned long long)ceil(share * (double)sum);
    return t < 1 ? 1 : t < sum ? t : sum;
  }
  __device__ __forceinline__ unsigned long long draw(unsigned long long kept) const {
    const unsigned long long t = (unsigned long long)(u * (double)kept);
    return (t < kept ? t : kept - 1) + 1;
  }
};

// What a long row has in the workspace.
struct Space {
  unsigned long long tops[kMaxSegments];  // of a segment: key << 32 | ~id
  unsigned long long sum[kBins];
  uint32_t count[kBins];
  unsigned long long near[kCap];          // gathered tokens
  uint32_t gathered, pad[3];
};

__device__ __forceinline__ unsigned long long token_of(uint32_t key, int id) {
  return (unsigned long long)key << 32 | (uint32_t)~id;
}

// A thread's tokens of [lo, hi) of the row, four at a time; the first kAhead fours are
// loaded before they are needed.  One copy of the code for each four, and with `small`
// for each token: most of what a short call takes is the fetching of its instructions.
constexpr int kAhead = 2;

template <int TY, int THREADS>
struct Tokens {
  float4 first[kAhead];
  const SampleArgs &a;
  long long at;
  int lo, hi;
  template <bool kSmall, class F>
  __device__ __forceinline__ void each(F f) const {
    each<kSmall>(f, [](float v) { return v >= -3.40282347e38f; });
  }
  __device__ __forceinline__ float4 load(int i) const {
    if (i + 3 < hi) return load4(a.z, TY, at + i);
    const float none = -__builtin_inff();
    float4 v = make_float4(none, none, none, none);
    if (i < hi) {
      v = load_few(a.z, TY, at + i, hi - i);
      if (hi - i < 2) v.y = none;
      if (hi - i < 3) v.z = none;
      v.w = none;
    }
    return v;
  }
  __device__ __forceinline__ Tokens(const SampleArgs &a_, long long row, int lo_, int hi_)
      : a(a_), at(row * a_.ldz), lo(lo_), hi(hi_) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) first[j] = load(lo + 4 * ((int)threadIdx.x + THREADS * j));
  }
  // Calls f(value, id) for each (kSmall: each that is `inside`); plus infinity comes as
  // the largest float, places past the end as minus infinity.
  template <bool kSmall, class F, class I>
  __device__ __forceinline__ void each(F f, I inside) const {
    float4 v0 = first[0], v1 = first[1];
    const auto one = [&](float v, int i) { f(v > 3.40282347e38f ? 3.40282347e38f : v, i); };
#pragma unroll 1
    for (int i = lo + 4 * (int)threadIdx.x; i < hi; i += 4 * THREADS) {
      const float4 v = v0;
      v0 = v1, v1 = load(i + 4 * THREADS * kAhead);
      if constexpr (kSmall) {
        if (!(inside(v.x) || inside(v.y) || inside(v.z) || inside(v.w))) continue;
        float x = v.x, y = v.y, z = v.z;
#pragma unroll 1
        for (int e = 0; e < 4; ++e) {
          if (inside(x)) one(x, i + e);
          x = y, y = z, z = v.w;
        }
      } else {
        one(v.x, i), one(v.y, i + 1), one(v.z, i + 2), one(v.w, i + 3);
      }
    }
  }
};

template <class T>
__device__ __forceinline__ T wave_max(T v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const T o = __shfl_xor(v, off, 64);
    v = o > v ? o : v;
  }
  return v;
}

template <int THREADS>
__device__ __forceinline__ unsigned long long block_max(unsigned long long v, unsigned long long *part) {
  v = wave_max(v);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = part[threadIdx.x & (THREADS / 64 - 1)];
#pragma unroll
  for (int off = THREADS / 128; off >= 1; off >>= 1) {
    const unsigned long long o = __shfl_xor(v, off, 64);
    v = o > v ? o : v;
  }
  return v;
}

// Sum of v over the threads before this one.
template <class T, int THREADS>
__device__ __forceinline__ T block_before(T v, T *part) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  T run = v;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const T o = __shfl_up(run, off, 64);
    if (lane >= off) run += o;
  }
  if (lane == 63) part[wave] = run;
  __syncthreads();
  for (int i = 0; i < wave; ++i) run += part[i];
  return run - v;
}

__device__ __forceinline__ void segment(const SampleArgs &a, int &lo, int &hi) {
  const int n = ((a.V + (int)gridDim.x - 1) / (int)gridDim.x + 3) & ~3;
  lo = min((int)blockIdx.x * n, a.V), hi = min(lo + n, a.V);
}

__device__ __forceinline__ void give(const SampleArgs &a, long long row, int token, double prob) {
  a.token[row] = token;
  if (a.prob) a.prob[row] = (float)prob;
}

// The workgroup's memory.
template <int THREADS>
struct Lds {
  unsigned long long sum[kBins + 1];   // of a bin; then of the bins before it
  unsigned long long token[kCap], sorted[kFew];
  Table table;
  uint32_t count[kBins + 1];           // likewise
  uint32_t gathered;
  unsigned long long part[THREADS / 64];
  uint32_t part32[THREADS / 64];
};

// The last i in [0, n) with below(i), which holds up to some place from 0 on; n <= 2048.
// Every lane of the wave takes part and gets it.
template <class F>
__device__ __forceinline__ int last_below(int n, F below) {
  const int lane = threadIdx.x & 63;
  const int base = 32 * max(__popcll(__ballot(32 * lane < n && below(min(32 * lane, n - 1)))) - 1, 0);
  return base + max(__popcll(__ballot(lane < 32 && base + lane < n && below(min(base + lane, n - 1)))) - 1, 0);
}

// Adds the tokens to the bins.
template <bool kSmall, int TY, int THREADS>
__device__ __forceinline__ void add_bins(const Tokens<TY, THREADS> &tokens, const Row &r,
                                         unsigned long long *sum, uint32_t *count, const Table &table) {
  const bool counts = r.k > 0;  // (looked at for top-k alone)
  tokens.template each<kSmall>([&](float v, int) {
    // (tokens of weight 0 add nothing to a bin behind all others: no branch)
    const Spot at(fmin(r.distance(v), kFar), table);
    const unsigned long long w = at.weight();
    atomicAdd(&sum[at.bin], w);
    if (counts && w) atomicAdd(&count[at.bin], 1u);
  });
}

// The first of a thread's largest tokens.
struct First {
  float v = -__builtin_inff();
  int id = 0;
  __device__ __forceinline__ void see(float o, int i) {
    if (o > v) v = o, id = i;
  }
  __device__ __forceinline__ unsigned long long token() const {
    const uint32_t key = order_bits(v);
    return key ? token_of(key, id) : 0ull;
  }
};

template <int TY>
__global__ __launch_bounds__(kScan) void sample_tops_kernel(SampleArgs a) {
  __shared__ unsigned long long part[kScan / 64];
  Space &s = ((Space *)a.ws)[blockIdx.y];
  int lo, hi;
  segment(a, lo, hi);
  const Tokens<TY, kScan> tokens(a, blockIdx.y, lo, hi);
  // what the next launches add to
  for (int i = blockIdx.x * kScan + threadIdx.x; i < kBins; i += gridDim.x * kScan) s.sum[i] = 0ull, s.count[i] = 0u;
  if (blockIdx.x == 0 && threadIdx.x == 0) s.gathered = 0u;
  First first;
  tokens.template each<false>([&](float v, int id) { first.see(v, id); });
  const unsigned long long t = block_max<kScan>(first.token(), part);
  if (threadIdx.x == 0) s.tops[blockIdx.x] = t;
}

__device__ __forceinline__ unsigned long long top_of(const Space &s, int segments) {
  const int lane = threadIdx.x & 63;
  unsigned long long t = lane < segments ? s.tops[lane] : 0ull;
  if (lane + 64 < segments) t = max(t, s.tops[lane + 64]);
  return wave_max(t);
}

template <int TY>
__global__ __launch_bounds__(kScan) void sample_bins_kernel(SampleArgs a) {
  __shared__ unsigned long long sum[kBins];
  __shared__ uint32_t count[kBins];
  __shared__ Table table;
  Space &s = ((Space *)a.ws)[blockIdx.y];
  int lo, hi;
  segment(a, lo, hi);
  const Tokens<TY, kScan> tokens(a, blockIdx.y, lo, hi);
  Row r(a, blockIdx.y);
  const uint32_t top = (uint32_t)(top_of(s, gridDim.x) >> 32);
  for (int i = threadIdx.x; i < kBins; i += kScan) sum[i] = 0ull, count[i] = 0u;
  table.fill();
  if (!top || r.greedy) return;
  r.top = (double)value_of(top);
  __syncthreads();
  add_bins<false>(tokens, r, sum, count, table);
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += kScan) {
    if (sum[i]) atomicAdd(&s.sum[i], sum[i]);
    if (count[i]) atomicAdd(&s.count[i], count[i]);
  }
}

// The last of the table's places that is not below v (the first, if all are).
__device__ __forceinline__ int table_place(const Table &table, double v) {
  const int i = last_below(kPlaces / 2 + 1, [&](int i) { return table.at(2 * i) >= v; });
  return 2 * i + 1 < kPlaces && table.at(2 * i + 1) >= v ? 2 * i + 1 : 2 * i;
}

// Which bins are wanted: up to four runs of them.
struct Wanted {
  int first[4], last[4];
  unsigned long long before_least = 0;  // sum before the first bin in which min-p's border can lie
  __device__ __forceinline__ void add(int i, int from, int to) {
    first[i] = from, last[i] = to;
  }
  __device__ __forceinline__ bool has(int b) const {
    bool in = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) in |= b >= first[i] && b <= last[i];
    return in;
  }
};

// From the bins' counts and sums (in m; they become those of the bins before each):
// which bins are wanted.  Every wave finds them for itself.
template <int THREADS>
__device__ Wanted decide(const Row &r, Lds<THREADS> &m) {
  constexpr int kMine = kBins / THREADS;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, b0 = kMine * threadIdx.x;
  uint32_t c[kMine], run32 = 0;
  unsigned long long w[kMine], run = 0;
#pragma unroll
  for (int j = 0; j < kMine; ++j) c[j] = run32, w[j] = run, run32 += m.count[b0 + j], run += m.sum[b0 + j];
  uint32_t up32 = run32;
  unsigned long long up = run;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t o32 = __shfl_up(up32, off, 64);
    const unsigned long long o = __shfl_up(up, off, 64);
    if (lane >= off) up32 += o32, up += o;
  }
  if (lane == 63) m.part32[wave] = up32, m.part[wave] = up;
  if (threadIdx.x == 0) m.gathered = 0u;
  __syncthreads();
  up32 -= run32, up -= run;
  for (int i = 0; i < wave; ++i) up32 += m.part32[i], up += m.part[i];
#pragma unroll
  for (int j = 0; j < kMine; ++j) m.count[b0 + j] = up32 + c[j], m.sum[b0 + j] = up + w[j];
  if (threadIdx.x == THREADS - 1) m.count[kBins] = up32 + run32, m.sum[kBins] = up + run;
  __syncthreads();
  Wanted wanted;
  // the bin of a position in the running sums
  const auto bin_at = [&](unsigned long long to) { return last_below(kBins, [&](int b) { return m.sum[b] < to; }); };
  // what is kept lies in [lo, hi]
  unsigned long long lo = m.sum[kBins], hi = lo;
  wanted.first[0] = wanted.first[1] = wanted.first[2] = kBins;
  wanted.last[0] = wanted.last[1] = wanted.last[2] = -1;
  if (r.k > 0 && (uint32_t)r.k < m.count[kBins]) {
    const int b = last_below(kBins, [&](int b) { return m.count[b] < (uint32_t)r.k; });
    wanted.add(0, b, b);
    lo = max(m.sum[b], 1ull), hi = m.sum[b + 1];
  }
  if (r.share < 1.0) {
    const unsigned long long from = r.share_of(lo), to = r.share_of(hi);
    const int b = bin_at(from), e = bin_at(to);
    wanted.add(1, b, e);
    lo = min(lo, from), hi = min(hi, m.sum[e + 1]);
  }
  if (r.least > 0.0) {
    // the border lies between two entries of the table, or within rounding of them
    const int i = table_place(m.table, r.least * kOne);
    const int b = bin_of(max(i - 1, 0)), e = bin_of(min(i + 2, kPlaces - 1));
    wanted.add(2, b, e);
    wanted.before_least = m.sum[b];
    lo = min(lo, max(m.sum[b], 1ull)), hi = min(hi, m.sum[e + 1]);
  }
  wanted.add(3, bin_at(r.draw(lo)), bin_at(r.draw(hi)));
  return wanted;
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

// The gathered tokens, the largest first; where they are.
template <int THREADS>
__device__ const unsigned long long *sorted(Lds<THREADS> &m, int n) {
  if (n <= kFew) {
    // a token's place is the number of larger ones
    for (int i = threadIdx.x; i < n; i += THREADS) {
      const unsigned long long mine = m.token[i];
      int place = 0;
      for (int j = 0; j < n; ++j) place += m.token[j] > mine;
      m.sorted[place] = mine;
    }
    __syncthreads();
    return m.sorted;
  }
  int size = 512;
  while (size < n) size *= 2;
  for (int i = n + threadIdx.x; i < size; i += THREADS) m.token[i] = 0ull;
  __syncthreads();
  sort_falling<THREADS>(m.token, size);
  return m.token;
}

// The row's token from its n gathered tokens.
template <int THREADS>
__device__ void settle(const SampleArgs &a, long long row, const Row &r, Lds<THREADS> &m, int n,
                       unsigned long long before_least) {
  constexpr int kMine = kCap / THREADS;
  const int lane = threadIdx.x & 63, i0 = kMine * threadIdx.x;
  const unsigned long long *x = sorted(m, n);
  const auto spot = [&](int i) { return Spot(r.distance(value_of((uint32_t)(x[i] >> 32))), m.table); };
  int bin[kMine];
  unsigned long long w[kMine], sum = 0;
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    bin[j] = -1, w[j] = 0ull;
    if (i0 + j < n) {
      const Spot at = spot(i0 + j);
      bin[j] = at.bin, w[j] = at.weight();
    }
    sum += w[j];
  }
  const int last_bin = i0 > 0 && i0 < n ? spot(i0 - 1).bin : -1;
  unsigned long long run = block_before<unsigned long long, THREADS>(sum, m.part);
  // a bin's first gathered token: what its tokens' sums and places are off by
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    if (bin[j] >= 0 && bin[j] != (j > 0 ? bin[j - 1] : last_bin))
      m.sum[bin[j]] -= run, m.count[bin[j]] -= (uint32_t)(i0 + j);
    run += w[j];
  }
  __syncthreads();
  run -= sum;
  const unsigned long long total = m.sum[kBins];
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    run += w[j];
    w[j] = bin[j] >= 0 ? run + m.sum[bin[j]] : 0ull;
  }
  __syncthreads();
  // the running sums up to each token take the place of the bins'
  unsigned long long *to = m.sum;
#pragma unroll
  for (int j = 0; j < kMine; ++j)
    if (i0 + j < n) to[i0 + j] = w[j];
  __syncthreads();
  if (threadIdx.x >= 64) return;
  // the first token whose running sum reaches a position
  const auto token_at = [&](unsigned long long p) {
    return n - 1 - last_below(n, [&](int i) { return to[n - 1 - i] >= p; });
  };
  unsigned long long keep = total;
  if (r.k > 0 && (uint32_t)r.k < m.count[kBins])
    keep = to[last_below(n, [&](int i) { return (uint32_t)i + m.count[spot(i).bin] < (uint32_t)r.k; })];
  if (r.share < 1.0) keep = min(keep, to[token_at(r.share_of(keep))]);
  if (r.least > 0.0) {
    const int i = last_below(n, [&](int i) { return spot(i).ratio() >= r.least; });
    keep = min(keep, spot(i).ratio() >= r.least ? max(before_least, to[i]) : before_least);
  }
  const int i = token_at(r.draw(keep));
  if (lane == 0) give(a, row, (int)~(uint32_t)x[i], spot(i).ratio() * kOne / (double)keep);
}

// ---- rows whose gathered tokens are too many

// The value at a position of the running counts or sums: its key, and the tokens and
// weights before its first equal.
struct Place {
  uint32_t key, count;
  unsigned long long sum;
};

// The weight of a value, or 0.
__device__ __forceinline__ unsigned long long weight_of(const Row &r, float v, const Table &table) {
  const double d = r.distance(v);
  return d < kFar ? Spot(d, table).weight() : 0ull;
}

template <int TY, int THREADS>
__device__ Place descend(const SampleArgs &a, long long row, const Row &r, bool by_count, unsigned long long target,
                         Lds<THREADS> &m, Place *shared) {
  Place p{0u, 0u, 0ull};
  int shift = 32;
  for (int level = 0; level < 3; ++level) {
    const int bits = level < 2 ? 11 : 10, above = shift;
    shift -= bits;
    for (int i = threadIdx.x; i < kBins; i += THREADS) m.count[i] = 0u, m.sum[i] = 0ull;
    __syncthreads();
    Tokens<TY, THREADS>(a, row, 0, a.V).template each<true>([&](float v, int) {
      const uint32_t key = order_bits(v);
      if (above < 32 && (key >> above) != (p.key >> above)) return;
      const unsigned long long w = weight_of(r, v, m.table);
      if (!w) return;
      const int b = key >> shift & ((1 << bits) - 1);
      // (equal tokens of a wave are added as one: 131072 equal logits 3.2 -> 1.9 ms)
      const uint64_t here = __ballot(1);
      const uint32_t first = __builtin_amdgcn_readfirstlane(key);
      const bool alike = __ballot(key != first) == 0;
      if (alike && (int)(threadIdx.x & 63) != __ffsll((unsigned long long)here) - 1) return;
      const uint32_t n = alike ? __popcll(here) : 1u;
      atomicAdd(&m.count[b], n);
      atomicAdd(&m.sum[b], n * w);
    });
    __syncthreads();
    if (threadIdx.x == 0) {
      int b = (1 << bits) - 1;
      for (; b > 0; --b) {
        if ((by_count ? p.count + m.count[b] : p.sum + m.sum[b]) >= target) break;
        p.count += m.count[b], p.sum += m.sum[b];
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
__device__ void settle_by_digits(const SampleArgs &a, long long row, const Row &r, Lds<THREADS> &m) {
  __shared__ Place shared;
  __shared__ unsigned long long kept;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  unsigned long long keep = m.sum[kBins];
  const uint32_t tokens = m.count[kBins];
  __syncthreads();
  if (r.k > 0 && (uint32_t)r.k < tokens) {
    const Place p = descend<TY, THREADS>(a, row, r, true, (unsigned long long)r.k, m, &shared);
    keep = p.sum + (r.k - p.count) * weight_of(r, value_of(p.key), m.table);
  }
  if (r.share < 1.0) {
    const unsigned long long t = r.share_of(keep);
    const Place p = descend<TY, THREADS>(a, row, r, false, t, m, &shared);
    const unsigned long long w = weight_of(r, value_of(p.key), m.table);
    keep = min(keep, p.sum + (t - p.sum + w - 1) / w * w);
  }
  if (r.least > 0.0) {
    if (tid == 0) kept = 0ull;
    __syncthreads();
    unsigned long long sum = 0;
    Tokens<TY, THREADS>(a, row, 0, a.V).template each<true>([&](float v, int) {
      const double d = r.distance(v);
      if (!(d < kFar)) return;
      const Spot at(d, m.table);
      if (at.ratio() >= r.least) sum += at.weight();
    });
    if (sum) atomicAdd(&kept, sum);
    __syncthreads();
    keep = min(keep, kept);
  }
  const unsigned long long t = r.draw(keep);
  const Place p = descend<TY, THREADS>(a, row, r, false, t, m, &shared);
  const unsigned long long w = weight_of(r, value_of(p.key), m.table);
  // the nth of the equal ones, by ids
  const uint32_t nth = (uint32_t)((t - 1 - p.sum) / w);
  uint32_t before = 0;
  for (int i0 = 0; i0 < a.V && before <= nth; i0 += THREADS) {
    const int i = i0 + tid;
    const bool hit = i < a.V && order_bits(load1(a.z, TY, row * a.ldz + i)) == p.key;
    const uint64_t same = __ballot(hit);
    if (lane == 0) m.part32[wave] = __popcll(same);
    __syncthreads();
    uint32_t mine = before;
    for (int j = 0; j < THREADS / 64; ++j) {
      if (j < wave) mine += m.part32[j];
      before += m.part32[j];
    }
    if (hit && mine + __popcll(same & ((1ull << lane) - 1)) == nth)
      give(a, row, i, Spot(r.distance(value_of(p.key)), m.table).ratio() * kOne / (double)keep);
    __syncthreads();
  }
}

// A run of bins as a range of values, a little wider.
struct Range {
  bool on;
  float low, high;
  __device__ __forceinline__ Range(const Row &r, int first, int last) {
    const double far = bin_start(last + 1) * r.temp, near = bin_start(first) * r.temp;
    const double slack = 1e-6 * (fabs(r.top) + far);
    const float h = r.top - near + slack < 3.4e38 ? (float)(r.top - near + slack) : __builtin_inff();
    on = __builtin_amdgcn_readfirstlane(first <= last);
    low = __int_as_float(__builtin_amdgcn_readfirstlane(
        __float_as_int(fmaxf((float)(r.top - far - slack), -3.40282347e38f))));
    high = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(h)));
  }
  __device__ __forceinline__ bool has(float v) const { return v >= low && v <= high; }
};

// Puts the tokens of the wanted bins into m.token (those past kCap are only counted).
template <int TY, int THREADS>
__device__ __forceinline__ void gather(const Tokens<TY, THREADS> &tokens, const Row &r, const Wanted &wanted,
                                       Lds<THREADS> &m) {
  // most tokens are passed over by their values
  const Range a0(r, wanted.first[0], wanted.last[0]), a1(r, wanted.first[1], wanted.last[1]),
      a2(r, wanted.first[2], wanted.last[2]), a3(r, wanted.first[3], wanted.last[3]);
  tokens.template each<true>(
      [&](float v, int id) {
        const double d = r.distance(v);
        if (!(d < kFar)) return;
        const Spot at(d, m.table);
        if (!wanted.has(at.bin) || !at.weight()) return;
        const uint32_t i = atomicAdd(&m.gathered, 1u);
        if (i < kCap) m.token[i] = token_of(order_bits(v), id);
      },
      [&](float v) {
        bool in = a3.has(v);
        if (a0.on) in |= a0.has(v);
        if (a1.on) in |= a1.has(v);
        if (a2.on) in |= a2.has(v);
        return in;
      });
  __syncthreads();
}

// The row's token once m holds the bins before each bin and n gathered tokens.
template <int TY>
__device__ __forceinline__ void finish(const SampleArgs &a, long long row, const Row &r, const Wanted &wanted,
                                       Lds<kScan> &m, uint32_t n) {
  if (n > kCap)
    settle_by_digits<TY, kScan>(a, row, r, m);
  else
    settle(a, row, r, m, (int)n, wanted.before_least);
}

template <int TY>
__global__ __launch_bounds__(kScan) void sample_gather_kernel(SampleArgs a) {
  __shared__ Lds<kScan> m;
  __shared__ uint32_t base;
  Space &s = ((Space *)a.ws)[blockIdx.y];
  int lo, hi;
  segment(a, lo, hi);
  const Tokens<TY, kScan> tokens(a, blockIdx.y, lo, hi);
  Row r(a, blockIdx.y);
  for (int i = threadIdx.x; i < kBins; i += kScan) m.sum[i] = s.sum[i], m.count[i] = s.count[i];
  const uint32_t top = (uint32_t)(top_of(s, gridDim.x) >> 32);
  m.table.fill();
  if (!top || r.greedy) return;
  r.top = (double)value_of(top);
  __syncthreads();
  gather(tokens, r, decide(r, m), m);
  const uint32_t n = m.gathered;
  if (n == 0u) return;
  if (threadIdx.x == 0) base = atomicAdd(&s.gathered, n);
  __syncthreads();
  if (base + n > kCap) return;
  for (uint32_t i = threadIdx.x; i < n; i += kScan) s.near[base + i] = m.token[i];
}

// (Done by the gathering's last workgroup instead, a launch less, the fences that make
// its tokens visible across the dies took far more: 89 for 42 us at 32 x 131072.)
template <int TY>
__global__ __launch_bounds__(kScan) void sample_finish_kernel(SampleArgs a, int segments) {
  __shared__ Lds<kScan> m;
  const Space &s = ((const Space *)a.ws)[blockIdx.x];
  const long long row = blockIdx.x;
  Row r(a, row);
  const uint32_t n = s.gathered;
  for (int i = threadIdx.x; i < kBins; i += kScan) m.sum[i] = s.sum[i], m.count[i] = s.count[i];
  for (uint32_t i = threadIdx.x; i < min(n, (uint32_t)kCap); i += kScan) m.token[i] = s.near[i];
  const unsigned long long first = top_of(s, segments);
  m.table.fill();
  if (!first || r.greedy) {
    if (threadIdx.x == 0) give(a, row, first ? (int)~(uint32_t)first : -1, first ? 1.0 : 0.0);
    return;
  }
  r.top = (double)value_of((uint32_t)(first >> 32));
  __syncthreads();
  const Wanted wanted = decide(r, m);
  finish<TY>(a, row, r, wanted, m, n);
}

template <int TY>
__global__ __launch_bounds__(kScan) void sample_row_kernel(SampleArgs a) {
  __shared__ Lds<kScan> m;
  const long long row = blockIdx.x;
  const Tokens<TY, kScan> tokens(a, row, 0, a.V);
  Row r(a, row);
  for (int i = threadIdx.x; i < kBins; i += kScan) m.sum[i] = 0ull, m.count[i] = 0u;
  m.table.fill();
  First mine;
  tokens.template each<false>([&](float v, int id) { mine.see(v, id); });
  const unsigned long long first = block_max<kScan>(mine.token(), m.part);
  if (!first || r.greedy) {
    if (threadIdx.x == 0) give(a, row, first ? (int)~(uint32_t)first : -1, first ? 1.0 : 0.0);
    return;
  }
  r.top = (double)value_of((uint32_t)(first >> 32));
  add_bins<true>(tokens, r, m.sum, m.count, m.table);
  __syncthreads();
  const Wanted wanted = decide(r, m);
  gather(tokens, r, wanted, m);
  finish<TY>(a, row, r, wanted, m, m.gathered);
}

int segments_of(int T, int V) {
  int n = 512 / (T < 1 ? 1 : T);
  const int most = (V + 4095) / 4096;
  n = n < most ? n : most;
  return n < 1 ? 1 : n < kMaxSegments ? n : kMaxSegments;
}

template <int TY>
hipError_t launch_type(const SampleArgs &a, hipStream_t s) {
  if (a.V <= kShortRow) return launch(sample_row_kernel<TY>, dim3(a.T), dim3(kScan), s, a);
  const int n = segments_of(a.T, a.V);
  hipError_t e = launch(sample_tops_kernel<TY>, dim3(n, a.T), dim3(kScan), s, a);
  if (e == hipSuccess) e = launch(sample_bins_kernel<TY>, dim3(n, a.T), dim3(kScan), s, a);
  if (e == hipSuccess) e = launch(sample_gather_kernel<TY>, dim3(n, a.T), dim3(kScan), s, a);
  if (e == hipSuccess) e = launch(sample_finish_kernel<TY>, dim3(a.T), dim3(kScan), s, a, n);
  return e;
}

}  // namespace

size_t sample_ws_bytes(int T, int V) { return V <= kShortRow ? 0 : (size_t)T * sizeof(Space); }

hipError_t launch_sample(const SampleArgs &a, hipStream_t s) {
  return a.type == kF32 ? launch_type<kF32>(a, s) : a.type == kBf16 ? launch_type<kBf16>(a, s) : launch_type<kF16>(a, s);
}

}  // namespace moe
