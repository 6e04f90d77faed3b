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
//
// Long prompts are bound by memory (queries in and out above all), single tokens
// by latency: a token's heads go to several workgroups, each of which computes
// the token's sines and cosines once.  Measured: 5391 float32 tokens of 16 + 2 * 8
// heads of 256: 64 us to append (4.3 TB/s), 26 us to read back; 4 bfloat16 tokens
// of 32 + 2 * 8 heads of 128: 7.1 us for both.
#include "device_types.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;

// Finite value of v: NaN counts as 0, infinities as the largest float.
__device__ __forceinline__ float finite_of(float v) {
  return v != v ? 0.f : fminf(fmaxf(v, -3.40282347e38f), 3.40282347e38f);
}

// A new token: its sequence, position and place in the cache.
struct Place {
  int s;          // -1: a row of no sequence
  long long pos;  // -1: none (no sequence, or a negative past)
  // page * kv_heads * page_tokens + offset in the page, or -1 when the sequence
  // has no valid page there; head h's row is at this + h * page_tokens
  long long row;
};

__device__ __forceinline__ Place place_of(const KvCache &c, const KvBatch &b, int t) {
  Place p{seq_of_row(b, t), -1, -1};
  if (p.s < 0) return p;
  const long long i = (long long)t - b.start[p.s], past = b.past[p.s];
  if (i < 0 || past < 0) return p;
  p.pos = past + i;
  const long long pi = p.pos / c.page_tokens;
  if (pi >= b.max_pages || p.pos >= kMaxPos) return p;
  const int page = b.pages[(long long)p.s * b.max_pages + pi];
  if (page >= 0 && page < c.n_pages)
    p.row = (long long)page * c.kv_heads * c.page_tokens + (p.pos - pi * c.page_tokens);
  return p;
}

// Cosines and sines of the token's pairs.
__device__ __forceinline__ void fill_angles(const KvAppendArgs &a, long long pos, double2 *cs) {
  for (int j = threadIdx.x; j < a.rot_dim / 2; j += kThreads) {
    double sn, c;
    sincos((double)pos * (double)a.inv_freq[j], &sn, &c);
    cs[j] = make_double2(c, sn);
  }
  __syncthreads();
}

// The first (second) coordinate of the pair (x, y) turned.
__device__ __forceinline__ float turn_first(float x, float y, double2 w) {
  return (float)((double)x * w.x - (double)y * w.y);
}
__device__ __forceinline__ float turn_second(float x, float y, double2 w) {
  return (float)((double)y * w.x + (double)x * w.y);
}

// Code of x at scale d (d != 0, inv about 1 / d): the largest n in 0..15 whose
// lower border d * (n - 8.5) x has reached, in the direction of d's sign.
__device__ __forceinline__ uint32_t q4_code(float x, float d, float inv) {
  float n = fminf(fmaxf(floorf(fmaf(x, inv, 8.5f)), 0.f), 15.f);
  // x / d >= n - 8.5, exactly: compare |d| (n - 8.5) with x on d's side
  const float y = d > 0.f ? x : -x, e = fabsf(d);
  if (y < e * (n - 8.5f) && n > 0.f) n -= 1.f;
  if (y >= e * (n - 7.5f) && n < 15.f) n += 1.f;
  return (uint32_t)n;
}

// The scale of a block whose first largest element is m.
__device__ __forceinline__ uint16_t q4_scale(float m) {
  const uint16_t h = f32_to_f16(fminf(fmaxf(m / -8.f, -65504.f), 65504.f));
  return (h & 0x7fffu) == 0 ? (uint16_t)0 : h;
}

// ---- rot_dim a multiple of 8: four elements an access

// Eight elements of a head as they are rotated together: pairs 4 i .. 4 i + 3 of
// the rotated part, or 8 elements of the rest.  at(j) is where the first and the
// second four lie in the head.
struct Chunk {
  int lo, hi;   // first elements of the two fours
  int pair;     // first pair, or -1 in the part that is not rotated
  __device__ __forceinline__ Chunk(int i, int rot, bool inter) {
    if (8 * i >= rot || inter) {
      lo = 8 * i, hi = 8 * i + 4;
      pair = 8 * i < rot ? 4 * i : -1;
    } else {
      lo = 4 * i, hi = rot / 2 + 4 * i;
      pair = 4 * i;
    }
  }
  __device__ __forceinline__ void turn(float4 &x, float4 &y, bool inter, const double2 *cs) const {
    if (pair < 0) return;
    const double2 w0 = cs[pair], w1 = cs[pair + 1], w2 = cs[pair + 2], w3 = cs[pair + 3];
    if (inter) {
      x = make_float4(turn_first(x.x, x.y, w0), turn_second(x.x, x.y, w0),
                      turn_first(x.z, x.w, w1), turn_second(x.z, x.w, w1));
      y = make_float4(turn_first(y.x, y.y, w2), turn_second(y.x, y.y, w2),
                      turn_first(y.z, y.w, w3), turn_second(y.z, y.w, w3));
    } else {
      const float4 a = x, b = y;
      x = make_float4(turn_first(a.x, b.x, w0), turn_first(a.y, b.y, w1),
                      turn_first(a.z, b.z, w2), turn_first(a.w, b.w, w3));
      y = make_float4(turn_second(a.x, b.x, w0), turn_second(a.y, b.y, w1),
                      turn_second(a.z, b.z, w2), turn_second(a.w, b.w, w3));
    }
  }
};

template <int CTRL>
__device__ __forceinline__ uint32_t quad(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}

// The block that a quad of lanes holds (lane g: elements 4 g .. 4 g + 3 in x, 4 g
// + 16 .. in y): word g of its codes, and its scale in every lane.
__device__ __forceinline__ uint32_t encode_block(const float4 x, const float4 y, uint16_t &scale) {
  const float v[8] = {finite_of(x.x), finite_of(x.y), finite_of(x.z), finite_of(x.w),
                      finite_of(y.x), finite_of(y.y), finite_of(y.z), finite_of(y.w)};
  const int g = threadIdx.x & 3;
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
  top = max(top, quad<0xB1>(top));
  top = max(top, quad<0x4E>(top));
  // the first element of that magnitude, with its sign in the lowest bit
  uint32_t first = 0xffffu;
#pragma unroll
  for (int j = 7; j >= 0; --j)
    if ((__float_as_uint(v[j]) & 0x7fffffffu) == top)
      first = (uint32_t)(4 * g + (j & 3) + (j >> 2) * 16) << 1 | __float_as_uint(v[j]) >> 31;
  first = min(first, quad<0xB1>(first));
  first = min(first, quad<0x4E>(first));
  scale = q4_scale(__uint_as_float(top | first << 31));
  const float d = f16_to_f32(scale);
  if (d == 0.f) return 0x88888888u;
  const float inv = 1.f / d;
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) w |= q4_code(v[j], d, inv) << (8 * (j & 3) + 4 * (j >> 2));
  return w;
}

// Workgroups 0 .. kv_groups - 1 of a token take its KV heads, `heads` each, the
// others its query heads.
template <int TY>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(KvAppendArgs a, int kv_groups,
                                                             int heads) {
  __shared__ double2 cs[128];
  __shared__ __attribute__((aligned(16))) float rows[kThreads * 8];  // rotated keys
  __shared__ __attribute__((aligned(16))) uint8_t bytes[kThreads * 4];  // the values' codes
  const int tid = threadIdx.x, D = a.c.head_dim, per = D / 8;
  const long long t = blockIdx.x;
  const Place p = place_of(a.c, a.b, (int)t);
  if (p.pos < 0) return;
  const bool inter = a.interleaved != 0;
  if ((int)blockIdx.y >= kv_groups) {
    if (a.rot_dim) fill_angles(a, p.pos, cs);
    const int groups = gridDim.y - kv_groups;
    for (int i = ((int)blockIdx.y - kv_groups) * kThreads + tid; i < a.q_heads * per;
         i += groups * kThreads) {
      const Chunk c(i % per, a.rot_dim, inter);
      const long long at = i / per * D;
      float4 x = load4(a.q, TY, t * a.ldq + at + c.lo), y = load4(a.q, TY, t * a.ldq + at + c.hi);
      c.turn(x, y, inter, cs);
      store4(a.q_out, TY, t * a.ldqo + at + c.lo, x);
      store4(a.q_out, TY, t * a.ldqo + at + c.hi, y);
    }
    return;
  }
  if (p.row < 0) return;
  // `heads` of them fit the workgroup's threads, a chunk or a quarter block each
  const int h0 = blockIdx.y * heads, n = min(heads, a.c.kv_heads - h0), nb = D / 32;
  const int head = h0 + tid / per;
  const bool mine = tid < n * per;
  // values: quarter block tid % per of its head
  const int b = tid % per >> 2, g = tid & 3;
  uint16_t scale;
  uint32_t w;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
  if (mine) {
    const long long at = t * a.ldv + (long long)head * D + b * 32 + 4 * g;
    x = load4(a.v, TY, at), y = load4(a.v, TY, at + 16);
  }
  float4 kx = make_float4(0.f, 0.f, 0.f, 0.f), ky = kx;
  const Chunk c(tid % per, a.rot_dim, inter);
  if (mine) {
    const long long at = t * a.ldk + (long long)head * D;
    kx = load4(a.k, TY, at + c.lo), ky = load4(a.k, TY, at + c.hi);
  }
  if (a.rot_dim) fill_angles(a, p.pos, cs);
  const long long row = p.row + (long long)head * a.c.page_tokens;
  w = encode_block(x, y, scale);
  if (mine) {
    if (g == 0) a.c.v_s[row * nb + b] = scale;
    // byte j of the block goes to place j * nb + b of the head's codes
#pragma unroll
    for (int j = 0; j < 4; ++j)
      bytes[tid / per * (D / 2) + (4 * g + j) * nb + b] = (uint8_t)(w >> (8 * j));
    c.turn(kx, ky, inter, cs);
    *(float4 *)&rows[tid / per * D + c.lo] = kx;
    *(float4 *)&rows[tid / per * D + c.hi] = ky;
  }
  __syncthreads();
  if (mine) {
    // four bytes a thread
    *(uint32_t *)(a.c.v_q + row * (D / 2) + tid % per * 4) = *(const uint32_t *)&bytes[tid * 4];
    x = *(const float4 *)&rows[tid / per * D + b * 32 + 4 * g];
    y = *(const float4 *)&rows[tid / per * D + b * 32 + 4 * g + 16];
  }
  w = encode_block(x, y, scale);
  if (mine) {
    *(uint32_t *)(a.c.k_q + row * (D / 2) + b * 16 + 4 * g) = w;
    if (g == 0) a.c.k_s[row * nb + b] = scale;
  }
}

// ---- any rot_dim: an element per thread, a workgroup per token (4 bfloat16 tokens of
// 32 + 8 heads of 128: 18.7 us against 4.9 us with fours)

__global__ __launch_bounds__(kThreads) void kv_append_any_kernel(KvAppendArgs a) {
  __shared__ double2 cs[128];
  const int t = blockIdx.x, tid = threadIdx.x;
  const Place p = place_of(a.c, a.b, t);
  if (p.pos < 0) return;
  const int D = a.c.head_dim, half = a.rot_dim / 2;
  fill_angles(a, p.pos, cs);
  auto turned = [&](const void *r, long long row, int e) -> float {
    const float x = load1(r, a.type, row + e);
    if (e >= a.rot_dim) return x;
    const int j = a.interleaved ? e >> 1 : e % half;
    const bool second = a.interleaved ? (e & 1) : e >= half;
    const int mate = a.interleaved ? e ^ 1 : second ? e - half : e + half;
    const float m = load1(r, a.type, row + mate);
    return second ? turn_second(m, x, cs[j]) : turn_first(x, m, cs[j]);
  };
  if (a.q)
    for (int e = tid; e < a.q_heads * D; e += kThreads)
      store1(a.q_out, a.type, t * a.ldqo + e, turned(a.q, t * a.ldq + e / D * D, e % D));
  if (p.row < 0) return;
  // one block per 32 lanes: keys, then values
  const int nb = D / 32, blocks = a.c.kv_heads * nb, l = tid & 31;
  for (int n = tid >> 5; n < 2 * blocks; n += kThreads / 32) {
    const bool is_v = n >= blocks;
    const int hb = is_v ? n - blocks : n, head = hb / nb, b = hb % nb;
    const float x = finite_of(is_v ? load1(a.v, a.type, t * a.ldv + head * D + b * 32 + l)
                                   : turned(a.k, t * a.ldk + head * D, b * 32 + l));
    // first element of largest magnitude: larger magnitudes first, then lower lanes
    unsigned long long best = ((unsigned long long)(__float_as_uint(x) & 0x7fffffffu) << 32) |
                              (uint32_t)(31 - l);
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) {
      const unsigned long long o = __shfl_xor(best, m, 32);
      best = o > best ? o : best;
    }
    const uint16_t scale = q4_scale(__shfl(x, 31 - (int)(uint32_t)best, 32));
    const float d = f16_to_f32(scale);
    const uint32_t code = d == 0.f ? 8u : q4_code(x, d, 1.f / d);
    const uint32_t up = __shfl_down(code, 16, 32);
    const long long row = p.row + (long long)head * a.c.page_tokens;
    if (l < 16) {
      const uint8_t byte = (uint8_t)(code | (up << 4));
      if (is_v)
        a.c.v_q[row * (D / 2) + l * nb + b] = byte;
      else
        a.c.k_q[row * (D / 2) + b * 16 + l] = byte;
    }
    if (l == 0) (is_v ? a.c.v_s : a.c.k_s)[row * nb + b] = scale;
  }
}

// The values the cache holds for a row: a quarter block (8 elements) per thread,
// keys' then values'; four threads write 128 contiguous bytes in two stores.
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvReadArgs a) {
  const int t = blockIdx.x;
  const Place p = place_of(a.c, a.b, t);
  if (p.s < 0) return;
  const int D = a.c.head_dim, nb = D / 32, per = D / 8, n = a.c.kv_heads * per;
  for (int i = blockIdx.y * kThreads + threadIdx.x; i < 2 * n; i += gridDim.y * kThreads) {
    const bool is_v = i >= n;
    const int j = is_v ? i - n : i, head = j / per, b = j % per >> 2, g = j & 3;
    uint32_t w = 0x88888888u;
    float d = 0.f;
    if (p.row >= 0) {
      const long long row = p.row + (long long)head * a.c.page_tokens;
      if (is_v) {
        const uint8_t *q = a.c.v_q + row * (D / 2) + 4 * g * nb + b;
        w = q[0] | (uint32_t)q[nb] << 8 | (uint32_t)q[2 * nb] << 16 | (uint32_t)q[3 * nb] << 24;
      } else {
        w = *(const uint32_t *)(a.c.k_q + row * (D / 2) + b * 16 + 4 * g);
      }
      d = f16_to_f32((is_v ? a.c.v_s : a.c.k_s)[row * nb + b]);
    }
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = d * (float)((int)(w >> (8 * (e & 3) + 4 * (e >> 2)) & 15u) - 8);
    float *o = (is_v ? a.v : a.k) + ((long long)t * a.c.kv_heads + head) * D + b * 32 + 4 * g;
    store4(o, kF32, 0, make_float4(v[0], v[1], v[2], v[3]));
    store4(o, kF32, 16, make_float4(v[4], v[5], v[6], v[7]));
  }
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs &a, hipStream_t s) {
  if (a.b.T == 0) return hipSuccess;
  if (a.rot_dim % 8) return launch(kv_append_any_kernel, dim3((unsigned)a.b.T), kThreads, s, a);
  const int per = a.c.head_dim / 8, fit = kThreads / per;
  const int heads = fit < a.c.kv_heads ? fit : a.c.kv_heads;
  const int kv_groups = (a.c.kv_heads + heads - 1) / heads;
  // query heads: a chunk per thread for few tokens, more for many, where the
  // sines and cosines would be computed once too often
  int q_groups = (a.q_heads * per + kThreads - 1) / kThreads;
  if (a.b.T > 512) q_groups = (q_groups + 3) / 4;
  const dim3 grid((unsigned)a.b.T, (unsigned)(kv_groups + q_groups));
  if (a.type == kF32) return launch(kv_append_kernel<kF32>, grid, kThreads, s, a, kv_groups, heads);
  if (a.type == kBf16) return launch(kv_append_kernel<kBf16>, grid, kThreads, s, a, kv_groups, heads);
  return launch(kv_append_kernel<kF16>, grid, kThreads, s, a, kv_groups, heads);
}

hipError_t launch_kv_read(const KvReadArgs &a, hipStream_t s) {
  if (a.b.T == 0) return hipSuccess;
  int groups = (2 * a.c.kv_heads * (a.c.head_dim / 8) + kThreads - 1) / kThreads;
  if (a.b.T > 512) groups = (groups + 3) / 4;
  return launch(kv_read_kernel, dim3((unsigned)a.b.T, (unsigned)groups), kThreads, s, a);
}

}  // namespace moe
