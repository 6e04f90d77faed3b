// Attention of the new tokens over the paged 4-bit cache:
//
//   out = softmax(scale * q K^T) V over the keys a row may see: positions up to
//   its own, within `window` positions when window > 0, on valid pages; a row
//   that sees no key gets 0.
//
// One wave per row and query head: 64 keys a step, a key per lane for the
// scores, a few elements of the head per lane for the weighted sum, with the
// running maximum and sum of the softmax in float32.
#include "device_types.hpp"

namespace moe {

namespace {

__global__ __launch_bounds__(64) void kv_attend_kernel(KvAttendArgs a) {
  __shared__ float qs[256], ps[64];
  __shared__ long long rows[64];
  const int t = blockIdx.x, qh = blockIdx.y, lane = threadIdx.x;
  const int s = seq_of_row(a.b, t);
  if (s < 0) return;
  const long long i = (long long)t - a.b.start[s], past = a.b.past[s];
  if (i < 0) return;
  const int D = a.c.head_dim, nb = D / 32, head = qh / (a.q_heads / a.c.kv_heads);
  const long long pos = past + i;
  const long long hi = past < 0 ? 0 : min(pos + 1, (long long)a.b.max_pages * a.c.page_tokens);
  const long long lo = a.window > 0 ? max(0ll, pos + 1 - a.window) : 0;
  for (int e = lane; e < D; e += 64) qs[e] = load1(a.q, a.type, t * a.ldq + qh * D + e) * a.scale;
  __syncthreads();
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (long long k0 = lo; k0 < hi; k0 += 64) {
    const long long key = k0 + lane;
    long long row = -1;
    if (key < hi) {
      const int page = a.b.pages[(long long)s * a.b.max_pages + key / a.c.page_tokens];
      if (page >= 0 && page < a.c.n_pages)
        row = ((long long)page * a.c.kv_heads + head) * a.c.page_tokens + key % a.c.page_tokens;
    }
    float z = -INFINITY;
    if (row >= 0) {
      z = 0.f;
      for (int b = 0; b < nb; ++b) {
        float sum = 0.f;
        for (int j = 0; j < 16; ++j) {
          const uint32_t byte = a.c.k_q[row * (D / 2) + b * 16 + j];
          sum = fmaf((float)(int)(byte & 15u) - 8.f, qs[b * 32 + j], sum);
          sum = fmaf((float)(int)(byte >> 4) - 8.f, qs[b * 32 + 16 + j], sum);
        }
        z = fmaf(f16_to_f32(a.c.k_s[row * nb + b]), sum, z);
      }
    }
    float top = z;
    for (int x = 32; x >= 1; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
    const float mn = fmaxf(m, top), ref = mn == -INFINITY ? 0.f : mn;
    const float alpha = expf(m - ref), p = expf(z - ref);
    m = mn;
    float sum = p;
    for (int x = 32; x >= 1; x >>= 1) sum += __shfl_xor(sum, x);
    l = l * alpha + sum;
    ps[lane] = p;
    rows[lane] = row;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] *= alpha;
    for (int j = 0; j < 64; ++j) {
      const long long r = rows[j];
      if (r < 0) continue;
      const float pj = ps[j];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = lane + 64 * e;
        if (d < D) {
          const uint32_t byte = a.c.v_q[r * (D / 2) + (d & 15) * nb + d / 32];
          const int code = (d & 16) ? byte >> 4 : byte & 15;
          o[e] = fmaf(pj, f16_to_f32(a.c.v_s[r * nb + d / 32]) * (float)(code - 8), o[e]);
        }
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int d = lane + 64 * e;
    if (d < D) store1(a.out, a.type, t * a.ldo + qh * D + d, l == 0.f ? 0.f : o[e] / l);
  }
}

}  // namespace

int kv_attend_splits(const KvCache &, const KvBatch &, int, int, int) { return 1; }

size_t kv_attend_ws_bytes(const KvCache &, const KvBatch &, int, int, int) { return 0; }

hipError_t launch_kv_attend(const KvAttendArgs &a, hipStream_t s) {
  if (a.b.T == 0) return hipSuccess;
  kv_attend_kernel<<<dim3((unsigned)a.b.T, (unsigned)a.q_heads), 64, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace moe
