// api_serving.hip -- the C ABI of the serving-step operators declared in
// include/qgemm.h: the residual norm with 8-bit rows, adapters beside a
// projection, the choice of experts and the verification of drafted tokens.  As
// in api.hip, every rule is checked before anything is launched, and the library
// never allocates and never synchronizes.
#include <cmath>

#include "layer_common.h"
#include "qgemm.h"

namespace qg {
hipError_t launch_rms_norm(const RmsNormArgs& a, hipStream_t stream);
int lora_splits(int64_t m, int64_t k, int64_t r, int64_t adapters);
hipError_t launch_lora_add(LoraArgs a, hipStream_t stream);
hipError_t launch_moe_route(RouteArgs a, hipStream_t stream);
int64_t verify_ws_bytes(int64_t b, int64_t v);
hipError_t launch_verify_drafts(VerifyArgs a, hipStream_t stream);
}  // namespace qg

namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 40;
// The x extent of a grid, below 2^32 threads: a row for each workgroup of 1024, eight
// tokens for each of 512.
constexpr int64_t kMaxNormRows = ((int64_t)1 << 22) - 1;
constexpr int64_t kMaxRouteTokens = 8 * (((int64_t)1 << 23) - 1);
constexpr int64_t kMaxWidth = 32768;                     // channels of a normed row

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

int32_t hip_status(hipError_t e) { return e == hipSuccess ? QG_OK : QG_E_HIP; }

bool dtype_ok(int32_t t) { return t == QG_BF16 || t == QG_F32; }

// Rows for 16-byte loads.
bool row_stride_ok(int64_t stride, int64_t rows, int64_t h) {
  return rows <= 1 || (stride >= h && stride <= kMaxStride && stride % 8 == 0);
}

// The rules that both norms share; fills in what they share.
int32_t check_norm(const void* x, int32_t x_dtype, int64_t x_stride, const void* residual, int32_t res_dtype,
                   int64_t res_stride, int64_t rows, int64_t h, const void* w, float eps, const void* res_out,
                   qg::RmsNormArgs* a) {
  if (rows < 0 || rows > kMaxNormRows || h < 8 || h > kMaxWidth || h % 8 != 0) return QG_E_SHAPE;
  if (!(eps >= 0.0f) || std::isinf(eps)) return QG_E_SHAPE;
  if (!dtype_ok(x_dtype) || (residual && !dtype_ok(res_dtype))) return QG_E_DTYPE;
  if (rows > 0 && (!x || (residual != nullptr) != (res_out != nullptr))) return QG_E_NULL;
  if (!row_stride_ok(x_stride, rows, h) || (residual && !row_stride_ok(res_stride, rows, h))) return QG_E_STRIDE;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(w, 16) || !aligned(res_out, 16)) return QG_E_ALIGN;
  a->x = x, a->res = residual, a->x_stride = x_stride, a->res_stride = res_stride, a->rows = rows, a->h = (int)h;
  a->x_f32 = x_dtype == QG_F32, a->res_f32 = residual && res_dtype == QG_F32;
  a->eps = eps;
  a->w = static_cast<const uint16_t*>(w);
  a->res_out = const_cast<void*>(res_out);
  return QG_OK;
}

// The shape rules of qg_lora_add.
int32_t lora_shape(int64_t m, int64_t k, int64_t n, int64_t r, int64_t adapters) {
  if (m < 0 || k < 8 || k % 8 != 0 || k > QG_LORA_MAX_DIM || n < 1 || n > QG_LORA_MAX_DIM) return QG_E_SHAPE;
  if (r < 8 || r > QG_LORA_MAX_RANK || r % 8 != 0 || adapters < 1 || adapters > 0x7fffffff) return QG_E_SHAPE;
  return m > QG_MAX_M ? QG_E_M_RANGE : QG_OK;
}

int64_t lora_ws(int64_t m, int64_t k, int64_t r, int64_t adapters) {
  return m == 0 ? 0 : qg::lora_splits(m, k, r, adapters) * m * r * 4;
}

// The shape rules of qg_verify_drafts.
int32_t verify_shape(int64_t rows, int64_t b, int64_t v) {
  if (b < 0 || b > 65535 || rows < b || rows > 0x7fffffff || v < 1 || v > 0x7fffffff) return QG_E_SHAPE;
  return QG_OK;
}

}  // namespace

extern "C" {

int32_t qg_rms_norm(const void* x, int32_t x_dtype, int64_t x_row_stride, const void* residual, int32_t residual_dtype,
                    int64_t residual_row_stride, int64_t rows, int64_t h, const void* w, float eps, void* y,
                    int32_t y_dtype, void* residual_out, void* stream) {
  qg::RmsNormArgs a{};
  const int32_t st = check_norm(x, x_dtype, x_row_stride, residual, residual_dtype, residual_row_stride, rows, h, w, eps,
                                residual_out, &a);
  if (st != QG_OK) return st;
  if (!dtype_ok(y_dtype)) return QG_E_DTYPE;
  if (!aligned(y, 16)) return QG_E_ALIGN;
  if (rows == 0) return QG_OK;
  if (!y) return QG_E_NULL;
  a.y = y;
  a.out = y_dtype == QG_F32 ? qg::kRmsF32 : qg::kRmsBf16;
  return hip_status(qg::launch_rms_norm(a, static_cast<hipStream_t>(stream)));
}

int32_t qg_rms_norm_q8(const void* x, int32_t x_dtype, int64_t x_row_stride, const void* residual,
                       int32_t residual_dtype, int64_t residual_row_stride, int64_t rows, int64_t h, const void* w,
                       float eps, int8_t* codes, float* scales, int32_t group_scales, void* residual_out,
                       void* stream) {
  qg::RmsNormArgs a{};
  const int32_t st = check_norm(x, x_dtype, x_row_stride, residual, residual_dtype, residual_row_stride, rows, h, w, eps,
                                residual_out, &a);
  if (st != QG_OK) return st;
  if (group_scales && h % QG_GROUP != 0) return QG_E_SHAPE;
  if (!aligned(codes, 8) || !aligned(scales, 4)) return QG_E_ALIGN;
  if (rows == 0) return QG_OK;
  if (!codes || !scales) return QG_E_NULL;
  a.codes = codes, a.scales = scales;
  a.out = group_scales ? qg::kRmsQ8Group : qg::kRmsQ8Row;
  return hip_status(qg::launch_rms_norm(a, static_cast<hipStream_t>(stream)));
}

int64_t qg_lora_add_workspace_bytes(int64_t m, int64_t k, int64_t n, int64_t r, int64_t adapters) {
  const int32_t st = lora_shape(m, k, n, r, adapters);
  return st != QG_OK ? st : lora_ws(m, k, r, adapters);
}

int32_t qg_lora_add(const void* x_bf16, int64_t m, int64_t k, const void* a_bf16, const void* b_bf16, int64_t r,
                    int64_t adapters, const int32_t* ids, const float* scales, const void* y, int32_t y_dtype,
                    int64_t y_row_stride, int64_t n, void* out, int32_t out_dtype, int64_t out_row_stride, void* ws,
                    int64_t ws_bytes, uint32_t* status_dev, void* stream) {
  const int32_t st = lora_shape(m, k, n, r, adapters);
  if (st != QG_OK) return st;
  if (!dtype_ok(y_dtype) || !dtype_ok(out_dtype)) return QG_E_DTYPE;
  if (m > 1 && (y_row_stride < n || out_row_stride < n || y_row_stride > kMaxStride || out_row_stride > kMaxStride))
    return QG_E_STRIDE;
  if (!aligned(x_bf16, 16) || !aligned(a_bf16, 16) || !aligned(b_bf16, 16) || !aligned(ids, 4) || !aligned(scales, 4) ||
      !aligned(y, y_dtype == QG_F32 ? 4 : 2) || !aligned(out, out_dtype == QG_F32 ? 4 : 2) || !aligned(ws, 16) ||
      !aligned(status_dev, 4))
    return QG_E_ALIGN;
  if (m == 0) return QG_OK;
  if (!x_bf16 || !a_bf16 || !b_bf16 || !ids || !y || !out || !ws) return QG_E_NULL;
  if (ws_bytes < lora_ws(m, k, r, adapters)) return QG_E_BUFFER;
  qg::LoraArgs a{};
  a.x = static_cast<const uint16_t*>(x_bf16);
  a.a = static_cast<const uint16_t*>(a_bf16);
  a.b = static_cast<const uint16_t*>(b_bf16);
  a.ids = ids, a.scales = scales, a.y = y, a.out = out, a.y_stride = y_row_stride, a.out_stride = out_row_stride;
  a.m = (int)m, a.k = (int)k, a.n = (int)n, a.r = (int)r, a.adapters = (int)adapters;
  a.y_f32 = y_dtype == QG_F32, a.out_f32 = out_dtype == QG_F32;
  a.splits = qg::lora_splits(m, k, r, adapters);
  a.part = static_cast<float*>(ws);
  a.status = status_dev;
  return hip_status(qg::launch_lora_add(a, static_cast<hipStream_t>(stream)));
}

int32_t qg_moe_route(const void* logits, int32_t logits_dtype, int64_t t, int64_t e, int64_t top_k, int32_t sigmoid,
                     const float* bias, int64_t groups, int64_t top_groups, int32_t group_best, int32_t renormalize,
                     float scale, int32_t* ids, float* weights, void* stream) {
  if (t < 0 || t > kMaxRouteTokens || e < 1 || e > 512 || top_k < 1 || top_k > 32) return QG_E_SHAPE;
  if (groups < 1 || groups > 64 || e % groups != 0 || top_groups < 1 || top_groups > groups) return QG_E_SHAPE;
  if (group_best < 1 || group_best > 2 || group_best > e / groups || top_k > top_groups * (e / groups))
    return QG_E_SHAPE;
  if (std::isnan(scale) || std::isinf(scale)) return QG_E_SHAPE;
  if (!dtype_ok(logits_dtype)) return QG_E_DTYPE;
  if (!aligned(logits, logits_dtype == QG_F32 ? 4 : 2) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
    return QG_E_ALIGN;
  if (t == 0) return QG_OK;
  if (!logits || !ids || !weights) return QG_E_NULL;
  qg::RouteArgs a{};
  a.logits = logits, a.bias = bias, a.t = t, a.e = (int)e, a.k = (int)top_k;
  a.half = logits_dtype == QG_BF16, a.sigmoid = sigmoid != 0;
  a.groups = (int)groups, a.top_groups = (int)top_groups, a.best = group_best, a.renorm = renormalize != 0;
  a.scale = scale, a.ids = ids, a.weights = weights;
  return hip_status(qg::launch_moe_route(a, static_cast<hipStream_t>(stream)));
}

int64_t qg_verify_drafts_workspace_bytes(int64_t rows, int64_t b, int64_t v) {
  const int32_t st = verify_shape(rows, b, v);
  return st != QG_OK ? st : qg::verify_ws_bytes(b, v);
}

int32_t qg_verify_drafts(const void* target, const void* draft, int32_t dtype, int64_t rows, int64_t v,
                         const int32_t* tokens, const float* u, const float* u_next, const int32_t* cu, int64_t b,
                         int32_t* lens, int32_t* accepted, int32_t* next, void* ws, int64_t ws_bytes,
                         uint32_t* status_dev, void* stream) {
  const int32_t st = verify_shape(rows, b, v);
  if (st != QG_OK) return st;
  if (!dtype_ok(dtype)) return QG_E_DTYPE;
  const uintptr_t el = dtype == QG_F32 ? 4 : 2;
  if (!aligned(target, el) || !aligned(draft, el) || !aligned(tokens, 4) || !aligned(u, 4) || !aligned(u_next, 4) ||
      !aligned(cu, 4) || !aligned(lens, 4) || !aligned(accepted, 4) || !aligned(next, 4) || !aligned(ws, 16) ||
      !aligned(status_dev, 4))
    return QG_E_ALIGN;
  if (b == 0) return QG_OK;
  if (!target || !u_next || !cu || !accepted || !next || (rows > b && (!tokens || !u))) return QG_E_NULL;
  const int64_t need = qg::verify_ws_bytes(b, v);
  if (need > 0 && (!ws || ws_bytes < need)) return ws ? QG_E_BUFFER : QG_E_NULL;
  qg::VerifyArgs a{};
  a.target = target, a.draft = draft, a.tokens = tokens, a.cu = cu, a.u = u, a.u_next = u_next;
  a.rows = rows, a.v = v, a.b = (int)b, a.half = dtype == QG_BF16;
  a.lens = lens, a.accepted = accepted, a.next = next;
  a.part = static_cast<double*>(ws);
  a.status = status_dev;
  return hip_status(qg::launch_verify_drafts(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
