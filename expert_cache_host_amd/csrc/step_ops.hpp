// Operators between a prompt and its next token: products in 8-bit integers,
// routing to experts by a rule, sampling.  Arguments as checked by step_ops.cpp,
// launchers in q8_rows.hip, q8_matmul.hip, route.hip and sample.hip.  Every
// launcher returns the launch's status and allocates nothing.
#pragma once
#include "decoder_ops.hpp"

namespace moe {

// Rows of 8-bit codes are zeroed up to a multiple of this many columns.
constexpr int kQ8Pad = 128;
inline constexpr long long q8_padded(long long cols) { return (cols + kQ8Pad - 1) / kQ8Pad * kQ8Pad; }

struct Q8RowsArgs {
  const void *x;      // [n] rows of cols, stride ldx
  int8_t *codes;      // [n] rows of q8_padded(cols), stride ldc
  float *scales;      // [n]
  long long ldx, ldc;
  int type, n, cols;
};
hipError_t launch_q8_rows(const Q8RowsArgs &a, hipStream_t s);

struct Q8MatmulArgs {
  const int8_t *x, *w;          // [T] and [rows] rows of codes, strides ldx and ldw
  const float *x_scales, *w_scales;
  void *out;                    // [T] rows of `rows`, stride ldo
  long long ldx, ldw, ldo;
  int type, T, rows, cols;
};
hipError_t launch_q8_matmul(const Q8MatmulArgs &a, hipStream_t s);
// Both: q's codes and scales are a.x and a.x_scales, memory that may stay unwritten.
hipError_t launch_q8_linear(const Q8RowsArgs &q, const Q8MatmulArgs &a, hipStream_t s);

constexpr int kRouteMaxExperts = 512, kRouteMaxTopk = 64, kRouteMaxGroups = 64;

struct RouteArgs {
  const void *z;      // [T] rows of E logits, stride ldz
  const float *bias;  // [E] or null
  int32_t *idx;       // [T][k]
  float *w;           // [T][k]
  int32_t *idx2;      // second copies (page-locked memory), or null
  float *w2;
  long long ldz;
  int type, T, E, k, sigmoid, groups, keep, best, renorm;
  float scale;
};
// start, stop: events recorded at the kernel's start and end, or null.
hipError_t launch_route(const RouteArgs &a, hipStream_t s, hipEvent_t start = nullptr, hipEvent_t stop = nullptr);

struct SampleArgs {
  const void *z;   // [T] rows of V logits, stride ldz
  const float *u;  // [T]
  // settings of each row, or null: those of the call
  const float *temperatures, *top_ps, *min_ps;
  const int32_t *top_ks;
  double temperature, top_p, min_p;
  int32_t *token;  // [T]
  float *prob;     // [T] or null
  void *ws;
  long long ldz;
  int top_k, type, T, V;
};
size_t sample_ws_bytes(int T, int V);
hipError_t launch_sample(const SampleArgs &a, hipStream_t s);

}  // namespace moe
