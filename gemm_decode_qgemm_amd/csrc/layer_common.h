// layer_common.h -- arguments and device helpers of the decoder-layer
// kernels: head norm with rotation, the 8-bit key/value cache, attention over
// it, and the mixture-of-experts layer.  Internal header.
#pragma once

#include "qg_common.h"

namespace qg {

struct NormRopeArgs {
  const uint16_t *q, *k;            // bf16, strides in elements
  int64_t q_ts, q_hs, k_ts, k_hs;   // per token and per head
  int64_t tokens;
  int hq, hkv, d, rot, pairs, max_pos;
  float eps, inv_d;
  const uint16_t *qw, *kw;          // bf16 [d] or null
  const float* cos_sin;             // [max_pos, rot]
  const int32_t* positions;
  uint16_t *q_out, *k_out;
  uint32_t* status;
  int iters, chunks;                // set by the launcher
};

// The cache (include/qgemm.h): pages of 64 tokens, a scale per 16 tokens.
constexpr int kPage = QG_KV8_PAGE;
constexpr int kBlock = QG_KV8_BLOCK;

struct Kv8Args {
  int8_t* codes;
  float* scales;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* cu;                // null: `rows / b` rows per sequence
  int64_t pages, width, rows;
  int b, hkv, d;
};

// bf16 pair (lo, hi) rounded to nearest even (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  bf16x2_t v;
  v[0] = (__bf16)lo;
  v[1] = (__bf16)hi;
  return __builtin_bit_cast(uint32_t, v);
}

// A barrier for LDS alone: loads from memory stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// First byte of the codes of (page, head): keys, then 64 d bytes of values.
__device__ __forceinline__ size_t kv8_base(int64_t page, int hkv, int h, int d) {
  return ((size_t)page * hkv + h) * (2 * kPage) * (size_t)d;
}

// The page that holds tokens [64 i, 64 i + 64) of a sequence, or -1 where the
// table has no such column or its entry names no page.
__device__ __forceinline__ int kv8_page(const int32_t* row, int64_t width, int64_t pages, int64_t i) {
  if (i < 0 || i >= width) return -1;
  const int p = row[i];
  return p >= 0 && p < pages ? p : -1;
}

// The rows of sequence b among `rows` (clipped to them).
__device__ __forceinline__ void kv8_rows(const int32_t* cu, int64_t rows, int nb, int b, int64_t& r0, int64_t& n) {
  if (cu) {
    r0 = cu[b];
    int64_t r1 = cu[b + 1];
    r0 = r0 < 0 ? 0 : r0;
    r1 = r1 > rows ? rows : r1;
    n = r1 > r0 ? r1 - r0 : 0;
  } else {
    n = rows / nb;
    r0 = n * b;
  }
}

// How qg_attn_kv8 splits the pages of its sequences (attn_kv8.hip): each in `splits`,
// or over `slots` workgroups by their lengths where slots > 0 (`splits` where those
// turn out to be about equal).
struct AttnSplit {
  int splits, slots;
};

// Residual addition and RMS norm (rms_norm.hip).
enum RmsOut { kRmsBf16, kRmsF32, kRmsQ8Row, kRmsQ8Group };

struct RmsNormArgs {
  const void *x, *res;              // rows of h channels, strides in elements; res may be null
  int64_t x_stride, res_stride, rows;
  int h, x_f32, res_f32, out;       // out: RmsOut
  float eps;
  const uint16_t* w;                // bf16 [h] or null
  void* y;                          // kRmsBf16, kRmsF32
  int8_t* codes;                    // else
  float* scales;
  void* res_out;                    // in the residual's type
};

// Low-rank adapters (lora.hip).
struct LoraArgs {
  const uint16_t *x, *a, *b;        // bf16 [m, k], [adapters, r, k], [adapters, n, r]
  const int32_t* ids;               // [m]
  const float* scales;              // [adapters] or null
  const void* y;                    // [m, n], rows y_stride apart
  void* out;                        // rows out_stride apart
  int64_t y_stride, out_stride;
  int m, k, n, r, adapters, y_f32, out_f32, splits;
  float* part;                      // [splits, m, r]
  uint32_t* status;
};

// The choice of experts (moe_route.hip).
struct RouteArgs {
  const void* logits;               // [t, e]
  const float* bias;                // [e] or null
  int64_t t;
  int e, k, half, sigmoid, groups, top_groups, best, renorm;
  int whole, lanes, shift, lanes16, shift16;   // set by the launcher (moe_route.hip)
  float scale;
  int32_t* ids;                     // [t, k]
  float* weights;                   // [t, k]
};

// Verification of drafted tokens (verify.hip).
struct VerifyArgs {
  const void *target, *draft;       // [rows, v], [rows - b, v] or null
  const int32_t *tokens, *cu;
  const float *u, *u_next;
  int64_t rows, v;
  int b, half;
  int32_t *lens, *accepted, *next;
  double* part;                     // [b, pieces]
  uint32_t* status;
  int64_t piece;                    // set by the launcher, as what follows
  int pieces, whole;                // whole: rows can be read 16 bytes at a time
};

}  // namespace qg
