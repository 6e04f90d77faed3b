// C entries of the operators between a prompt and its next token (declared in
// include/moe_cache.h): argument checks, then the launchers.  They hold no state,
// allocate nothing and wait for nothing, as those of decoder_ops.cpp.
#include "step_ops.hpp"

#include <cmath>
#include <cstdio>

#include "../../include/moe_cache.h"
#include "errors.hpp"
#include "route_rule.hpp"

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

const char *codes_fault(const void *codes, int64_t stride, int64_t least, int32_t n) {
  if (!codes) return "codes are NULL";
  if ((uintptr_t)codes % 16) return "codes must be 16-byte aligned";
  if (n > 1 && (stride < least || stride % 16 || stride > (1 << 22)))
    return "codes' stride must be a multiple of 16 that holds a padded row, at most 2^22";
  return nullptr;
}

const char *q8_sizes_fault(int32_t n_tokens, int32_t rows, int32_t cols) {
  if (cols < 1 || cols > MOE_Q8_MAX_COLS) return "cols must be in [1, 131072]";
  if (rows < 1 || rows > MOE_Q8_MAX_ROWS) return "rows must be in [1, 2^24)";
  if (n_tokens < 0 || n_tokens > MOE_Q8_MAX_TOKENS) return "n_tokens must be in [0, 2^20]";
  // a grid holds fewer than 2^32 threads, 512 a tile of 256 x 256
  if ((int64_t)((n_tokens + 255) / 256) * ((rows + 255) / 256) >= 1 << 22)
    return "n_tokens / 256 * rows / 256 must stay below 2^22";
  return nullptr;
}

}  // namespace

extern "C" {

moe_status moe_q8_rows(const void *x, int32_t type, int64_t x_stride, int32_t n_rows, int32_t cols, void *codes,
                       int64_t codes_stride, float *scales, moe_stream_t stream) {
  clear_error();
  if (bad_type(type)) return einval("element type must be MOE_F32, MOE_BF16 or MOE_F16");
  if (cols < 1 || cols > MOE_Q8_MAX_COLS) return einval("cols must be in [1, 131072]");
  if (n_rows < 0 || n_rows > MOE_Q8_MAX_ROWS) return einval("n_rows must be in [0, 2^24)");
  if (x_stride < 0) return einval("x_stride must be >= 0");
  if (n_rows == 0) return MOE_OK;
  if (!x || !scales) return einval("x or scales is NULL");
  if (const char *f = codes_fault(codes, codes_stride, moe::q8_padded(cols), n_rows)) return einval(f);
  if (misaligned(x, type) || (uintptr_t)scales % 4) return einval("a pointer is not aligned to its element type");
  moe::Q8RowsArgs a{};
  a.x = x, a.codes = (int8_t *)codes, a.scales = scales;
  a.ldx = x_stride, a.ldc = codes_stride, a.type = type, a.n = n_rows, a.cols = cols;
  return done(moe::launch_q8_rows(a, stream));
}

moe_status moe_q8_matmul(const void *x, int64_t x_stride, const float *x_scales, int32_t n_tokens, const void *w,
                         int64_t w_stride, const float *w_scales, int32_t rows, int32_t cols, void *out, int32_t type,
                         int64_t out_stride, moe_stream_t stream) {
  clear_error();
  if (bad_type(type)) return einval("element type must be MOE_F32, MOE_BF16 or MOE_F16");
  if (const char *f = q8_sizes_fault(n_tokens, rows, cols)) return einval(f);
  if (n_tokens > 1 && out_stride < rows) return einval("out_stride must be >= rows");
  if (n_tokens == 0) return MOE_OK;
  if (const char *f = codes_fault(x, x_stride, moe::q8_padded(cols), n_tokens)) return einval(f);
  if (const char *f = codes_fault(w, w_stride, (cols + 15) / 16 * 16, rows)) return einval(f);
  if (!x_scales || !w_scales || !out) return einval("NULL argument");
  if ((uintptr_t)x_scales % 4 || (uintptr_t)w_scales % 4 || misaligned(out, type))
    return einval("a pointer is not aligned to its element type");
  moe::Q8MatmulArgs a{};
  a.x = (const int8_t *)x, a.w = (const int8_t *)w, a.x_scales = x_scales, a.w_scales = w_scales, a.out = out;
  a.ldx = n_tokens > 1 ? x_stride : moe::q8_padded(cols), a.ldw = rows > 1 ? w_stride : moe::q8_padded(cols);
  a.ldo = out_stride, a.type = type;
  a.T = n_tokens, a.rows = rows, a.cols = cols;
  return done(moe::launch_q8_matmul(a, stream));
}

int64_t moe_q8_linear_workspace(int32_t n_tokens, int32_t rows, int32_t cols) {
  clear_error();
  if (const char *f = q8_sizes_fault(n_tokens, rows, cols)) return einval(f);
  return (int64_t)n_tokens * (moe::q8_padded(cols) + 4);
}

moe_status moe_q8_linear(const void *x, int32_t type, int64_t x_stride, int32_t n_tokens, const void *w,
                         int64_t w_stride, const float *w_scales, int32_t rows, int32_t cols, void *out,
                         int32_t out_type, int64_t out_stride, void *workspace, int64_t workspace_bytes,
                         moe_stream_t stream) {
  clear_error();
  if (bad_type(type) || bad_type(out_type)) return einval("element type must be MOE_F32, MOE_BF16 or MOE_F16");
  if (const char *f = q8_sizes_fault(n_tokens, rows, cols)) return einval(f);
  if (x_stride < 0) return einval("x_stride must be >= 0");
  if (n_tokens > 1 && out_stride < rows) return einval("out_stride must be >= rows");
  if (n_tokens == 0) return MOE_OK;
  if (const char *f = codes_fault(w, w_stride, (cols + 15) / 16 * 16, rows)) return einval(f);
  if (!x || !w_scales || !out) return einval("NULL argument");
  if (misaligned(x, type) || (uintptr_t)w_scales % 4 || misaligned(out, out_type))
    return einval("a pointer is not aligned to its element type");
  const int64_t padded = moe::q8_padded(cols);
  if (!workspace || workspace_bytes < n_tokens * (padded + 4))
    return einval("workspace is smaller than moe_q8_linear_workspace says");
  if ((uintptr_t)workspace % 16) return einval("workspace must be 16-byte aligned");
  moe::Q8RowsArgs q{};
  q.x = x, q.codes = (int8_t *)workspace, q.scales = (float *)((char *)workspace + n_tokens * padded);
  q.ldx = x_stride, q.ldc = padded, q.type = type, q.n = n_tokens, q.cols = cols;
  moe::Q8MatmulArgs a{};
  a.x = q.codes, a.w = (const int8_t *)w, a.x_scales = q.scales, a.w_scales = w_scales, a.out = out;
  a.ldx = padded, a.ldw = rows > 1 ? w_stride : padded, a.ldo = out_stride, a.type = out_type;
  a.T = n_tokens, a.rows = rows, a.cols = cols;
  return done(moe::launch_q8_linear(q, a, stream));
}

moe_status moe_route(const void *logits, int32_t type, int64_t stride, const float *bias, int32_t n_tokens,
                     int32_t n_experts, const moe_route_rule *rule, int32_t *idx, float *w, moe_stream_t stream) {
  clear_error();
  if (bad_type(type)) return einval("element type must be MOE_F32, MOE_BF16 or MOE_F16");
  if (const char *f = moe::rule_fault(rule, n_experts)) return einval(f);
  if (n_tokens < 0 || n_tokens > MOE_ROUTE_MAX_TOKENS) return einval("n_tokens must be in [0, 2^24]");
  if (stride < 0) return einval("stride must be >= 0");
  if (n_tokens == 0) return MOE_OK;
  if (!logits || !idx || !w) return einval("NULL argument");
  if (misaligned(logits, type) || (uintptr_t)bias % 4 || (uintptr_t)idx % 4 || (uintptr_t)w % 4)
    return einval("a pointer is not aligned to its element type");
  moe::RouteArgs a = moe::route_args(*rule);
  a.z = logits, a.bias = bias, a.idx = idx, a.w = w;
  a.ldz = stride, a.type = type, a.T = n_tokens, a.E = n_experts;
  return done(moe::launch_route(a, stream));
}

int64_t moe_sample_workspace(int32_t n_rows, int32_t vocab) {
  clear_error();
  if (n_rows < 0 || n_rows > MOE_SAMPLE_MAX_ROWS) return einval("n_rows must be in [0, 65535]");
  if (vocab < 1 || vocab > MOE_SAMPLE_MAX_VOCAB) return einval("vocab must be in [1, 2^20]");
  return (int64_t)moe::sample_ws_bytes(n_rows, vocab);
}

moe_status moe_sample(const void *logits, int32_t type, int64_t stride, int32_t n_rows, int32_t vocab, const float *u,
                      const moe_sample_opts *opts, int32_t *token, float *prob, void *workspace,
                      int64_t workspace_bytes, moe_stream_t stream) {
  clear_error();
  if (bad_type(type)) return einval("element type must be MOE_F32, MOE_BF16 or MOE_F16");
  if (n_rows < 0 || n_rows > MOE_SAMPLE_MAX_ROWS) return einval("n_rows must be in [0, 65535]");
  if (vocab < 1 || vocab > MOE_SAMPLE_MAX_VOCAB) return einval("vocab must be in [1, 2^20]");
  if (stride < 0) return einval("stride must be >= 0");
  if (!opts) return einval("opts is NULL");
  if (!opts->temperatures && !(opts->temperature >= 0.0 && std::isfinite(opts->temperature)))
    return einval("temperature must be finite and >= 0");
  if (!opts->top_ks && opts->top_k < 0) return einval("top_k must be >= 0");
  if (!opts->top_ps && !(opts->top_p >= 0.0 && opts->top_p <= 1.0)) return einval("top_p must be in [0, 1]");
  if (!opts->min_ps && !(opts->min_p >= 0.0 && opts->min_p <= 1.0)) return einval("min_p must be in [0, 1]");
  if (n_rows == 0) return MOE_OK;
  if (!logits || !u || !token) return einval("NULL argument");
  if (misaligned(logits, type) || (uintptr_t)u % 4 || (uintptr_t)token % 4 || (uintptr_t)prob % 4 ||
      (uintptr_t)opts->temperatures % 4 || (uintptr_t)opts->top_ks % 4 || (uintptr_t)opts->top_ps % 4 ||
      (uintptr_t)opts->min_ps % 4)
    return einval("a pointer is not aligned to its element type");
  const int64_t need = (int64_t)moe::sample_ws_bytes(n_rows, vocab);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return einval("workspace is smaller than moe_sample_workspace says");
  if ((uintptr_t)workspace % 16) return einval("workspace must be 16-byte aligned");
  moe::SampleArgs a{};
  a.z = logits, a.u = u, a.token = token, a.prob = prob, a.ws = workspace;
  a.temperatures = opts->temperatures, a.top_ps = opts->top_ps, a.min_ps = opts->min_ps, a.top_ks = opts->top_ks;
  a.temperature = opts->temperature, a.top_p = opts->top_p, a.min_p = opts->min_p, a.top_k = opts->top_k;
  a.ldz = stride, a.type = type, a.T = n_rows, a.V = vocab;
  return done(moe::launch_sample(a, stream));
}

}  // extern "C"
