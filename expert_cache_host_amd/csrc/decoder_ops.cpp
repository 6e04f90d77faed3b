// C entries of the decoder-layer operators (declared in include/moe_cache.h):
// argument checks, then one launcher.  They hold no state, allocate nothing and
// wait for nothing, so they may be captured into a HIP graph and called from
// several threads and streams at once.
#include "decoder_ops.hpp"

#include <cmath>
#include <cstdio>

#include "../../include/moe_cache.h"
#include "errors.hpp"

namespace {

using moe::clear_error;

moe_status einval(const char *msg) { return moe::set_error(MOE_EINVAL, msg); }

moe_status done(hipError_t e) {
  if (e == hipSuccess) return MOE_OK;
  char buf[256];
  std::snprintf(buf, sizeof buf, "launch failed: %s", hipGetErrorString(e));
  return moe::set_error(MOE_EHIP, buf);
}

bool bad_type(int32_t t) { return t != MOE_F32 && t != MOE_BF16 && t != MOE_F16; }

bool misaligned(const void *p, int32_t type) {
  return (uintptr_t)p % (uintptr_t)moe::type_bytes(type) != 0;
}

// nullptr, or what is wrong with the cache.
const char *cache_fault(const moe_kv_cache *c) {
  if (!c) return "cache is NULL";
  if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales) return "cache pointer is NULL";
  if (c->n_pages < 1) return "n_pages must be >= 1";
  if (c->page_tokens < 16 || c->page_tokens % 16 || c->page_tokens > MOE_KV_MAX_PAGE_TOKENS)
    return "page_tokens must be a multiple of 16 in [16, 65536]";
  if (c->kv_heads < 1 || c->kv_heads > MOE_KV_MAX_HEADS) return "kv_heads must be in [1, 1024]";
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return "head_dim must be 64, 128 or 256";
  for (const void *p : {(const void *)c->k_codes, (const void *)c->k_scales,
                        (const void *)c->v_codes, (const void *)c->v_scales})
    if ((uintptr_t)p % 16) return "cache pointers must be 16-byte aligned";
  return nullptr;
}

const char *batch_fault(const moe_kv_batch *b) {
  if (!b) return "batch is NULL";
  if (!b->pages || !b->start || !b->past) return "batch pointer is NULL";
  if (b->n_seqs < 1) return "n_seqs must be >= 1";
  if (b->max_pages < 1) return "max_pages must be >= 1";
  if (b->n_rows < 0 || b->n_rows > MOE_KV_MAX_ROWS) return "n_rows must be in [0, 2^23]";
  for (const void *p : {(const void *)b->pages, (const void *)b->start, (const void *)b->past})
    if ((uintptr_t)p % 4) return "batch pointers must be 4-byte aligned";
  return nullptr;
}

moe::KvCache to_cache(const moe_kv_cache *c) {
  return {(uint8_t *)c->k_codes, (uint8_t *)c->v_codes, (uint16_t *)c->k_scales,
          (uint16_t *)c->v_scales, c->n_pages, c->page_tokens, c->kv_heads, c->head_dim};
}

moe::KvBatch to_batch(const moe_kv_batch *b) {
  return {b->pages, b->start, b->past, b->n_seqs, b->max_pages, b->n_rows};
}

// A grid dimension holds fewer than 2^32 threads, 2^24 workgroups of attention; a
// tile holds at least 8 of a KV head's rows.
const char *tiles_fault(const moe_kv_cache *c, const moe_kv_batch *b, int32_t q_heads) {
  if ((int64_t)b->n_rows * (q_heads / c->kv_heads) / 8 + b->n_seqs >= 1 << 24)
    return "n_rows * q_heads / kv_heads / 8 + n_seqs must stay below 2^24";
  return nullptr;
}

const char *heads_fault(const moe_kv_cache *c, int32_t q_heads) {
  if (q_heads < 1 || q_heads > MOE_KV_MAX_HEADS) return "q_heads must be in [1, 1024]";
  if (q_heads % c->kv_heads) return "q_heads must be a multiple of kv_heads";
  return nullptr;
}

}  // namespace

extern "C" {

moe_status moe_block_norm(const void *h, int32_t h_type, int64_t h_stride, const void *y,
                          int32_t y_type, int64_t y_stride, const float *post_w, const void *gate,
                          int32_t gate_type, int64_t gate_stride, const float *pre_w,
                          int32_t n_tokens, int32_t d, float res_scale, float block_scale,
                          float eps, void *h_out, int64_t h_out_stride, void *x, int32_t x_type,
                          int64_t x_stride, moe_stream_t stream) {
  clear_error();
  if (n_tokens < 0) return einval("n_tokens must be >= 0");
  if (d < 1 || d > MOE_NORM_MAX_D) return einval("d must be in [1, 32768]");
  if (bad_type(h_type) || (y && bad_type(y_type)) || (gate && bad_type(gate_type)) ||
      (x && bad_type(x_type)))
    return einval("element type must be MOE_F32, MOE_BF16 or MOE_F16");
  if (!(eps >= 0.f) || !std::isfinite(eps)) return einval("eps must be finite and >= 0");
  if (n_tokens == 0) return MOE_OK;  // empty tensors have no address to judge by
  if (!y && (post_w || gate)) return einval("post_w and gate need y");
  if ((x == nullptr) != (pre_w == nullptr)) return einval("x and pre_w go together");
  if (!h_out && !x) return einval("nothing to write: h_out and x are NULL");
  if (h_stride < 0 || (y && y_stride < 0) || (gate && gate_stride < 0))
    return einval("input strides must be >= 0");
  if ((h_out && h_out_stride < d && n_tokens > 1) || (x && x_stride < d && n_tokens > 1))
    return einval("output strides must be >= d");
  if (!h) return einval("h is NULL");
  if (misaligned(h, h_type) || (y && misaligned(y, y_type)) || (gate && misaligned(gate, gate_type)) ||
      misaligned(h_out, h_type) || (x && misaligned(x, x_type)) || (uintptr_t)post_w % 4 ||
      (uintptr_t)pre_w % 4)
    return einval("a pointer is not aligned to its element type");
  moe::NormArgs a{};
  a.h = h, a.y = y, a.gate = gate, a.post_w = post_w, a.pre_w = pre_w, a.h_out = h_out, a.x = x;
  a.ldh = h_stride, a.ldy = y_stride, a.ldg = gate_stride, a.ldho = h_out_stride, a.ldx = x_stride;
  a.h_type = h_type, a.y_type = y_type, a.g_type = gate_type, a.x_type = x_type;
  a.T = n_tokens, a.d = d;
  a.res_scale = res_scale, a.block_scale = block_scale, a.eps = eps;
  return done(moe::launch_block_norm(a, stream));
}

moe_status moe_q4_matvec(const void *codes, const void *scales, int32_t rows, int32_t cols,
                         int32_t group, const void *x, int32_t type, int64_t x_stride,
                         int32_t n_tokens, void *out, int64_t out_stride, moe_stream_t stream) {
  clear_error();
  if (bad_type(type)) return einval("element type must be MOE_F32, MOE_BF16 or MOE_F16");
  if (group != 32 && group != 64 && group != 128) return einval("group must be 32, 64 or 128");
  if (rows < 1 || rows > MOE_Q4_MAX_ROWS) return einval("rows must be in [1, 2^30]");
  if (cols < group || cols % group) return einval("cols must be a multiple of group");
  if (n_tokens < 0 || n_tokens > MOE_Q4_MAX_TOKENS) return einval("n_tokens must be in [0, 65536]");
  if (x_stride < 0) return einval("x_stride must be >= 0");
  if (n_tokens > 1 && out_stride < rows) return einval("out_stride must be >= rows");
  if (n_tokens == 0) return MOE_OK;
  if (!codes || !scales || !x || !out) return einval("NULL argument");
  if ((uintptr_t)codes % 16) return einval("codes must be 16-byte aligned");
  if ((uintptr_t)scales % 2 || misaligned(x, type) || misaligned(out, type))
    return einval("a pointer is not aligned to its element type");
  moe::Q4MatvecArgs a{};
  a.q = (const uint8_t *)codes, a.scales = (const uint16_t *)scales, a.x = x, a.out = out;
  a.ldx = x_stride, a.ldo = out_stride, a.type = type, a.T = n_tokens;
  a.rows = rows, a.cols = cols, a.group = group;
  return done(moe::launch_q4_matvec(a, stream));
}

moe_status moe_kv_append(const moe_kv_cache *cache, const moe_kv_batch *batch, int32_t type,
                         const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                         const float *inv_freq, int32_t rot_dim, int32_t interleaved,
                         const void *q, int64_t q_stride, int32_t q_heads, void *q_out,
                         int64_t q_out_stride, moe_stream_t stream) {
  clear_error();
  if (const char *f = cache_fault(cache)) return einval(f);
  if (const char *f = batch_fault(batch)) return einval(f);
  if (bad_type(type)) return einval("element type must be MOE_F32, MOE_BF16 or MOE_F16");
  if (rot_dim < 0 || rot_dim % 2 || rot_dim > cache->head_dim)
    return einval("rot_dim must be even and in [0, head_dim]");
  if (rot_dim && (!inv_freq || (uintptr_t)inv_freq % 4)) return einval("inv_freq is NULL or misaligned");
  if (interleaved != 0 && interleaved != 1) return einval("interleaved must be 0 or 1");
  if (batch->n_rows == 0) return MOE_OK;
  if ((q == nullptr) != (q_out == nullptr)) return einval("q and q_out go together");
  if (q) {
    if (const char *f = heads_fault(cache, q_heads)) return einval(f);
    if (q == q_out) return einval("q_out must not be q");
    if (q_stride < 0) return einval("input strides must be >= 0");
    if (batch->n_rows > 1 && q_out_stride < (int64_t)q_heads * cache->head_dim)
      return einval("q_out_stride must be >= q_heads * head_dim");
  }
  if (k_stride < 0 || v_stride < 0) return einval("input strides must be >= 0");
  if (!k || !v) return einval("k or v is NULL");
  if (misaligned(k, type) || misaligned(v, type) || misaligned(q, type) || misaligned(q_out, type))
    return einval("a pointer is not aligned to its element type");
  moe::KvAppendArgs a{};
  a.c = to_cache(cache), a.b = to_batch(batch);
  a.q = q, a.k = k, a.v = v, a.q_out = q_out;
  a.ldq = q_stride, a.ldk = k_stride, a.ldv = v_stride, a.ldqo = q_out_stride;
  a.inv_freq = inv_freq, a.type = type, a.q_heads = q ? q_heads : 0;
  a.rot_dim = rot_dim, a.interleaved = interleaved;
  return done(moe::launch_kv_append(a, stream));
}

moe_status moe_kv_read(const moe_kv_cache *cache, const moe_kv_batch *batch, float *k, float *v,
                       moe_stream_t stream) {
  clear_error();
  if (const char *f = cache_fault(cache)) return einval(f);
  if (const char *f = batch_fault(batch)) return einval(f);
  if (batch->n_rows == 0) return MOE_OK;
  if (!k || !v) return einval("k or v is NULL");
  if ((uintptr_t)k % 4 || (uintptr_t)v % 4) return einval("a pointer is not aligned to its element type");
  moe::KvReadArgs a{};
  a.c = to_cache(cache), a.b = to_batch(batch), a.k = k, a.v = v;
  return done(moe::launch_kv_read(a, stream));
}

int64_t moe_kv_attend_workspace(const moe_kv_cache *cache, const moe_kv_batch *batch, int32_t type,
                                int32_t q_heads, int32_t window) {
  clear_error();
  const char *f = cache_fault(cache);
  if (!f) f = batch_fault(batch);
  if (!f && bad_type(type)) f = "element type must be MOE_F32, MOE_BF16 or MOE_F16";
  if (!f) f = heads_fault(cache, q_heads);
  if (!f && window < 0) f = "window must be >= 0";
  if (!f) f = tiles_fault(cache, batch, q_heads);
  if (f) return einval(f);
  return (int64_t)moe::kv_attend_ws_bytes(to_cache(cache), to_batch(batch), type, q_heads, window);
}

moe_status moe_kv_attend(const moe_kv_cache *cache, const moe_kv_batch *batch, int32_t type,
                         const void *q, int64_t q_stride, int32_t q_heads, float scale,
                         int32_t window, void *out, int64_t out_stride, void *workspace,
                         int64_t workspace_bytes, moe_stream_t stream) {
  clear_error();
  if (const char *f = cache_fault(cache)) return einval(f);
  if (const char *f = batch_fault(batch)) return einval(f);
  if (bad_type(type)) return einval("element type must be MOE_F32, MOE_BF16 or MOE_F16");
  if (const char *f = heads_fault(cache, q_heads)) return einval(f);
  if (!std::isfinite(scale)) return einval("scale must be finite");
  if (window < 0) return einval("window must be >= 0");
  if (q_stride < 0) return einval("input strides must be >= 0");
  if (batch->n_rows > 1 && out_stride < (int64_t)q_heads * cache->head_dim)
    return einval("out_stride must be >= q_heads * head_dim");
  if (const char *f = tiles_fault(cache, batch, q_heads)) return einval(f);
  if (batch->n_rows == 0) return MOE_OK;
  if (!q || !out) return einval("q or out is NULL");
  if (misaligned(q, type) || misaligned(out, type))
    return einval("a pointer is not aligned to its element type");
  moe::KvAttendArgs a{};
  a.c = to_cache(cache), a.b = to_batch(batch);
  const int64_t need = (int64_t)moe::kv_attend_ws_bytes(a.c, a.b, type, q_heads, window);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return einval("workspace is smaller than moe_kv_attend_workspace says");
  if ((uintptr_t)workspace % 16) return einval("workspace must be 16-byte aligned");
  a.q = q, a.out = out, a.ldq = q_stride, a.ldo = out_stride, a.type = type;
  a.q_heads = q_heads, a.window = window, a.scale = scale, a.ws = workspace;
  return done(moe::launch_kv_attend(a, stream));
}

}  // extern "C"
