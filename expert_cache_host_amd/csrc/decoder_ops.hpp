// Operators of the decoder layer around the MoE layer: arguments as checked by
// decoder_ops.cpp, launchers in block_norm.hip, q4_matvec.hip, kv_cache.hip
// and kv_attend.hip.  Every launcher returns the launch's status and allocates
// nothing.
#pragma once
#include <hip/hip_runtime_api.h>

#include <cstddef>
#include <cstdint>

namespace moe {

// Element types (MOE_F32, MOE_BF16, MOE_F16 of the C header).
enum : int { kF32 = 0, kBf16 = 1, kF16 = 2 };
inline constexpr int type_bytes(int t) { return t == kF32 ? 4 : 2; }

constexpr int kNormMaxD = 32768;

struct NormArgs {
  const void *h, *y, *gate;       // y may be null; gate null, [d] or [T][d]
  const float *post_w, *pre_w;    // may be null
  void *h_out, *x;                // may be null
  long long ldh, ldy, ldg, ldho, ldx;  // row strides in elements (ldg 0: one row for all)
  int h_type, y_type, g_type, x_type;
  int T, d;
  float res_scale, block_scale, eps;
};
hipError_t launch_block_norm(const NormArgs &a, hipStream_t s);

struct Q4MatvecArgs {
  const uint8_t *q;       // [rows][cols/32][16]
  const uint16_t *scales; // binary16 [rows][cols/group]
  const void *x;          // [T] rows of cols, stride ldx
  void *out;              // [T] rows of `rows`, stride ldo
  long long ldx, ldo;
  int type, T, rows, cols, group;
};
hipError_t launch_q4_matvec(const Q4MatvecArgs &a, hipStream_t s);

// The paged 4-bit cache (moe_kv_cache of the C header).
struct KvCache {
  uint8_t *k_q, *v_q;
  uint16_t *k_s, *v_s;
  int n_pages, page_tokens, kv_heads, head_dim;
};
// The packed batch: sequence s owns rows start[s] .. start[s+1]-1, which stand
// at positions past[s], past[s] + 1, ... of its pages.
struct KvBatch {
  const int32_t *pages, *start, *past;
  int n_seqs, max_pages, T;
};

struct KvAppendArgs {
  KvCache c;
  KvBatch b;
  const void *q, *k, *v;
  void *q_out;
  long long ldq, ldk, ldv, ldqo;
  const float *inv_freq;
  int type, q_heads, rot_dim, interleaved;
};
hipError_t launch_kv_append(const KvAppendArgs &a, hipStream_t s);

struct KvReadArgs {
  KvCache c;
  KvBatch b;
  float *k, *v;  // [T][kv_heads][head_dim]
};
hipError_t launch_kv_read(const KvReadArgs &a, hipStream_t s);

struct KvAttendArgs {
  KvCache c;
  KvBatch b;
  const void *q;
  void *out;
  long long ldq, ldo;
  int type, q_heads, window;
  float scale;
  void *ws;
};
// Workspace of a call of these sizes.
size_t kv_attend_ws_bytes(const KvCache &c, const KvBatch &b, int type, int q_heads, int window);
hipError_t launch_kv_attend(const KvAttendArgs &a, hipStream_t s);

}  // namespace moe
