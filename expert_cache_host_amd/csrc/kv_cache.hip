// New tokens' keys and values into the paged 4-bit cache, and rows read back.
//
// Per block of 32 elements along the head: m = the first element of largest
// magnitude, d = fp16(m / -8) (saturating), code = clamp(floor(x / d + 8.5), 0,
// 15), value = d * (code - 8).  Keys are rotated by their position first: the
// angle (position * inv_freq), its sine and cosine and the rotation in 64 bits,
// the result rounded once to 32, so that a code depends on the inputs alone and
// not on the order or rounding of the steps.  A code's border d * (n - 1/2) is
// exact in float32 (11 + 4 bits), so the float32 estimate of the code is
// corrected by exact comparisons.
#include "device_types.hpp"

namespace moe {

namespace {

// Finite value of v: NaN counts as 0, infinities as the largest float.
__device__ __forceinline__ float finite_of(float v) {
  return v != v ? 0.f : fminf(fmaxf(v, -3.40282347e38f), 3.40282347e38f);
}

// Where position `pos` of sequence `s` lies: (page * kv_heads * page_tokens +
// offset in the page), or -1 when the sequence has no valid page there.  Head
// h's row is at this + h * page_tokens.
__device__ __forceinline__ long long cache_row(const KvCache &c, const KvBatch &b, int s,
                                               long long pos) {
  if (pos < 0) return -1;
  const long long pi = pos / c.page_tokens;
  if (pi >= b.max_pages) return -1;
  const int page = b.pages[(long long)s * b.max_pages + pi];
  if (page < 0 || page >= c.n_pages) return -1;
  return (long long)page * c.kv_heads * c.page_tokens + (pos - pi * c.page_tokens);
}

constexpr int kAppendThreads = 256;

// Code of x at scale d (d != 0): the largest n in 0..15 whose lower border d *
// (n - 8.5) x has reached, in the direction of d's sign.
__device__ __forceinline__ uint32_t q4_code(float x, float d, float inv) {
  float n = fminf(fmaxf(floorf(fmaf(x, inv, 8.5f)), 0.f), 15.f);
  // x / d >= n - 8.5, exactly: compare x with d * (n - 8.5) on d's side
  const float lo = d * (n - 8.5f), hi = d * (n - 7.5f);
  const bool below = d > 0.f ? x < lo : x > lo;
  const bool above = d > 0.f ? x >= hi : x <= hi;
  if (below && n > 0.f) n -= 1.f;
  if (above && n < 15.f) n += 1.f;
  return (uint32_t)n;
}

// One workgroup per new token.
__global__ __launch_bounds__(kAppendThreads) void kv_append_kernel(KvAppendArgs a) {
  __shared__ double2 cs[256];
  const int t = blockIdx.x, tid = threadIdx.x;
  const int s = seq_of_row(a.b, t);
  if (s < 0) return;
  const long long i = (long long)t - a.b.start[s], past = a.b.past[s];
  if (i < 0 || past < 0) return;
  const long long pos = past + i;
  const int D = a.c.head_dim, half = a.rot_dim / 2;
  for (int j = tid; j < half; j += kAppendThreads) {
    double sn, c;
    sincos((double)pos * (double)a.inv_freq[j], &sn, &c);
    cs[j] = make_double2(c, sn);
  }
  __syncthreads();
  auto turned = [&](const void *p, long long row, int e) -> float {
    const float x = load1(p, a.type, row + e);
    if (e >= a.rot_dim) return x;
    const int j = a.interleaved ? e >> 1 : e % half;
    const bool second = a.interleaved ? (e & 1) : e >= half;
    const int mate = a.interleaved ? e ^ 1 : second ? e - half : e + half;
    const double m = (double)load1(p, a.type, row + mate);
    const double2 w = cs[j];
    return second ? (float)((double)x * w.x + m * w.y) : (float)((double)x * w.x - m * w.y);
  };
  if (a.q)
    for (int e = tid; e < a.q_heads * D; e += kAppendThreads)
      store1(a.q_out, a.type, t * a.ldqo + e, turned(a.q, t * a.ldq + e / D * D, e % D));

  const long long row0 = cache_row(a.c, a.b, s, pos);
  if (row0 < 0) return;
  // one block per 32 lanes: keys, then values
  const int nb = D / 32, blocks = a.c.kv_heads * nb, l = tid & 31;
  for (int n = tid >> 5; n < 2 * blocks; n += kAppendThreads / 32) {
    const bool is_v = n >= blocks;
    const int hb = is_v ? n - blocks : n, head = hb / nb, b = hb % nb;
    const float x = finite_of(is_v ? load1(a.v, a.type, t * a.ldv + head * D + b * 32 + l)
                                   : turned(a.k, t * a.ldk + head * D, b * 32 + l));
    // first element of largest magnitude: larger magnitudes first, then lower lanes
    unsigned long long best =
        ((unsigned long long)(__builtin_bit_cast(uint32_t, x) & 0x7fffffffu) << 32) |
        (uint32_t)(31 - l);
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) {
      const unsigned long long o = __shfl_xor(best, m, 32);
      best = o > best ? o : best;
    }
    const float m = __shfl(x, 31 - (int)(uint32_t)best, 32);
    const float d32 = fminf(fmaxf(m / -8.f, -65504.f), 65504.f);
    uint16_t dh = f32_to_f16(d32);
    const float d = f16_to_f32(dh);
    if (d == 0.f) dh = 0;
    const uint32_t code = d == 0.f ? 8u : q4_code(x, d, 1.f / d);
    const uint32_t up = __shfl_down(code, 16, 32);
    const long long row = row0 + (long long)head * a.c.page_tokens;
    if (l < 16) {
      const uint8_t byte = (uint8_t)(code | (up << 4));
      if (is_v)
        a.c.v_q[row * (D / 2) + l * nb + b] = byte;
      else
        a.c.k_q[row * (D / 2) + b * 16 + l] = byte;
    }
    if (l == 0) (is_v ? a.c.v_s : a.c.k_s)[row * nb + b] = dh;
  }
}

// One workgroup per row: the values the cache holds for it.
__global__ __launch_bounds__(256) void kv_read_kernel(KvReadArgs a) {
  const int t = blockIdx.x;
  const int s = seq_of_row(a.b, t);
  if (s < 0) return;
  const long long i = (long long)t - a.b.start[s], past = a.b.past[s];
  if (i < 0 || past < 0) return;
  const int D = a.c.head_dim, nb = D / 32, n = a.c.kv_heads * D;
  const long long row0 = cache_row(a.c, a.b, s, past + i);
  for (int e = threadIdx.x; e < 2 * n; e += 256) {
    const bool is_v = e >= n;
    const int f = is_v ? e - n : e, head = f / D, x = f % D, b = x / 32, l = x % 32;
    float val = 0.f;
    if (row0 >= 0) {
      const long long row = row0 + (long long)head * a.c.page_tokens;
      const uint8_t byte = is_v ? a.c.v_q[row * (D / 2) + (l & 15) * nb + b]
                                : a.c.k_q[row * (D / 2) + b * 16 + (l & 15)];
      const int code = l < 16 ? byte & 15 : byte >> 4;
      val = f16_to_f32((is_v ? a.c.v_s : a.c.k_s)[row * nb + b]) * (float)(code - 8);
    }
    (is_v ? a.v : a.k)[(long long)t * n + f] = val;
  }
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs &a, hipStream_t s) {
  if (a.b.T == 0) return hipSuccess;
  kv_append_kernel<<<dim3((unsigned)a.b.T), kAppendThreads, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvReadArgs &a, hipStream_t s) {
  if (a.b.T == 0) return hipSuccess;
  kv_read_kernel<<<dim3((unsigned)a.b.T), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace moe
