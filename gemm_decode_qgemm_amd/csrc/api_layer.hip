// api_layer.hip -- the C ABI of the decoder-layer operators declared in
// include/qgemm.h: argument checks on the host, then kernel launches on the
// caller's stream.  As in api.hip, every rule is checked before anything is
// launched, and the library never allocates and never synchronizes.
#include <cmath>

#include "layer_common.h"
#include "qgemm.h"

namespace qg {
hipError_t launch_qk_norm_rope(NormRopeArgs a, hipStream_t stream);
hipError_t launch_kv8_append(const Kv8Args& c, const void* k, int64_t k_ts, int64_t k_hs, const void* v, int64_t v_ts,
                             int64_t v_hs, int64_t max_new, uint32_t* status, hipStream_t stream);
hipError_t launch_kv8_read(const Kv8Args& c, int64_t max_len, void* k, void* v, int f32, hipStream_t stream);
AttnSplit attn_kv8_split(int64_t b, int64_t rows, int hkv, int d, int64_t rows_per_head, int64_t max_len, int window,
                         int64_t max_q);
hipError_t launch_attn_kv8(const Kv8Args& c, const void* q, int64_t q_ts, int64_t q_hs, int hq, int max_q,
                           int64_t max_len, int window, float scale, void* out, int out_f32, AttnSplit by, float* part,
                           uint32_t* status, hipStream_t stream);
int64_t moe_ws_bytes(int64_t t, int64_t h, int64_t e, int64_t inter, int64_t k);
hipError_t launch_moe_w4a16(const void* x, int t, int h, const void* router, int e, const void* gate_up,
                            int64_t gate_up_bytes, const void* down, int64_t down_bytes, int inter, int k, int renorm,
                            void* y, int y_f32, void* ws, const int32_t* ids, const float* weights, uint32_t* status,
                            hipStream_t stream);
}  // namespace qg

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 30;   // tokens, positions, lengths
constexpr int64_t kMaxGrid = 65535;              // the y and z extents of a grid
constexpr int64_t kMaxBlocks = ((int64_t)1 << 24) - 1;   // its x extent: below 2^32 threads at 256
constexpr int32_t kMaxHeads = 4096;
constexpr int32_t kMaxSplits = 256;
constexpr int64_t kMaxDim = (int64_t)1 << 20;    // channels and hidden columns of an expert

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

int32_t hip_status(hipError_t e) { return e == hipSuccess ? QG_OK : QG_E_HIP; }

// Strides of [rows, heads, d] in elements, for 16-byte loads of channels.
bool strides_ok(int64_t token, int64_t head, int64_t rows, int32_t heads, int32_t d) {
  const int64_t most = (int64_t)1 << 40;
  if (token % 8 != 0 || head % 8 != 0 || token < 0 || head < 0 || token > most || head > most) return false;
  return (heads <= 1 || head >= d) && (rows <= 1 || token >= d);
}

bool cache_d(int32_t d) { return d == 64 || d == 128 || d == 192 || d == 256; }

// The rules that every call on the cache shares.
int32_t check_cache(const void* codes, const void* scales, int64_t pages, int32_t hkv, int32_t d, const void* table,
                    int64_t width, const void* lens, int64_t b) {
  if (!codes || !scales || !table || !lens) return QG_E_NULL;
  if (pages < 1 || pages > 0x7fffffff || width < 1 || width > kMaxRows || b < 1 || b > kMaxGrid) return QG_E_SHAPE;
  if (hkv < 1 || hkv > kMaxHeads || !cache_d(d)) return QG_E_HEADS;
  if (b * hkv > kMaxBlocks) return QG_E_SHAPE;
  if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(table, 4) || !aligned(lens, 4)) return QG_E_ALIGN;
  return QG_OK;
}

// Rows of new tokens or queries of b sequences.
int32_t check_rows(int64_t rows, const void* cu, int64_t b) {
  if (rows < 0 || rows > kMaxRows || (!cu && rows % b != 0)) return QG_E_SHAPE;
  return aligned(cu, 4) ? QG_OK : QG_E_ALIGN;
}

qg::Kv8Args cache_args(const int8_t* codes, const float* scales, int64_t pages, int32_t hkv, int32_t d,
                       const int32_t* table, int64_t width, const int32_t* lens, const int32_t* cu, int64_t rows,
                       int64_t b) {
  return {const_cast<int8_t*>(codes), const_cast<float*>(scales), table, lens, cu, pages, width, rows, (int)b, hkv, d};
}

// The shape rules of qg_attn_kv8 and the split it will use.
int32_t attn_shape(int64_t b, int64_t rows, int32_t hq, int32_t hkv, int32_t d, int64_t max_q, int64_t max_len,
                   int32_t window, int32_t splits, qg::AttnSplit* out) {
  if (b < 1 || b > kMaxGrid || rows < 0 || rows > kMaxRows || max_q < 1 || max_q > kMaxGrid || max_len < 0 ||
      max_len > 0x7fffffff || window < 0 ||
      window > kMaxRows)
    return QG_E_SHAPE;
  if (hkv < 1 || hkv > kMaxHeads || hq < 1 || hq > kMaxHeads || hq % hkv != 0 || !cache_d(d)) return QG_E_HEADS;
  const int64_t per_head = max_q * (hq / hkv);
  if ((per_head + 15) / 16 * hkv > kMaxGrid) return QG_E_SHAPE;
  if (splits < 0 || splits > kMaxSplits) return QG_E_SPLIT;
  *out = splits ? qg::AttnSplit{splits, 0} : qg::attn_kv8_split(b, rows, hkv, d, per_head, max_len, window, max_q);
  return QG_OK;
}

int64_t attn_ws(int64_t b, int64_t rows, int32_t hq, int32_t d, int64_t max_q, qg::AttnSplit by) {
  if (by.slots > 0) return by.slots * max_q * hq * (d + 2) * 4 + b * 8;
  return by.splits > 1 ? (int64_t)by.splits * rows * hq * (d + 2) * 4 : 0;
}

constexpr int64_t kMaxExperts = 512, kMaxPicks = 32;

// The shape rules of qg_moe_w4a16.
int32_t moe_shape(int64_t t, int64_t h, int64_t e, int64_t inter, int64_t k) {
  if (t < 0 || h < 1 || inter < 1 || h > kMaxDim || inter > kMaxDim) return QG_E_SHAPE;
  if (e < 1 || e > kMaxExperts || k < 1 || k > kMaxPicks || k > e) return QG_E_SHAPE;
  if (h % QG_TILE_K != 0 || inter % QG_TILE_K != 0) return QG_E_K_MULTIPLE;
  return t > QG_MAX_M ? QG_E_M_RANGE : QG_OK;
}

// The rules that both layers share.
int32_t moe_check(const void* x, int64_t t, int64_t h, int64_t e, const void* gate_up, int64_t gate_up_bytes,
                  const void* down, int64_t down_bytes, int64_t inter, int64_t k, const void* y, int32_t y_dtype,
                  const void* ws) {
  const int32_t st = moe_shape(t, h, e, inter, k);
  if (st != QG_OK) return st;
  if (y_dtype != QG_BF16 && y_dtype != QG_F32) return QG_E_DTYPE;
  if (gate_up_bytes < e * qg_int4_packed_bytes(2 * inter, h) || down_bytes < e * qg_int4_packed_bytes(h, inter))
    return QG_E_BUFFER;
  if (!aligned(x, 16) || !aligned(gate_up, 16) || !aligned(down, 16) || !aligned(y, 16) || !aligned(ws, 16))
    return QG_E_ALIGN;
  return QG_OK;
}

}  // namespace

extern "C" {

int32_t qg_qk_norm_rope(const void* q, int64_t q_ts, int64_t q_hs, const void* k, int64_t k_ts, int64_t k_hs,
                        int64_t tokens, int32_t hq, int32_t hkv, int32_t d, const void* q_w, const void* k_w,
                        const float* cos_sin, int64_t max_pos, int32_t rot, int32_t adjacent_pairs,
                        const int32_t* positions, float eps, void* q_out, void* k_out, uint32_t* status_dev,
                        void* stream) {
  if (tokens < 0 || tokens > 4 * kMaxBlocks || max_pos < 1 || max_pos > 0x7fffffff) return QG_E_SHAPE;
  if (hq < 0 || hkv < 0 || hq > kMaxHeads || hkv > kMaxHeads || hq + hkv < 1) return QG_E_HEADS;
  if (d < 16 || d > 512 || d % 16 != 0 || rot < 0 || rot > d || rot % 16 != 0) return QG_E_HEADS;
  if (!(eps >= 0.0f) || std::isinf(eps)) return QG_E_SHAPE;
  if (tokens == 0) return QG_OK;
  if ((hq > 0 && (!q || !q_out)) || (hkv > 0 && (!k || !k_out)) || !positions || (rot > 0 && !cos_sin))
    return QG_E_NULL;
  if ((hq > 0 && !strides_ok(q_ts, q_hs, tokens, hq, d)) || (hkv > 0 && !strides_ok(k_ts, k_hs, tokens, hkv, d)))
    return QG_E_STRIDE;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_w, 16) || !aligned(k_w, 16) || !aligned(cos_sin, 16) ||
      !aligned(positions, 4) || !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(status_dev, 4))
    return QG_E_ALIGN;
  qg::NormRopeArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.q_ts = q_ts, a.q_hs = q_hs, a.k_ts = k_ts, a.k_hs = k_hs;
  a.tokens = tokens;
  a.hq = hq, a.hkv = hkv, a.d = d, a.rot = rot, a.pairs = adjacent_pairs != 0, a.max_pos = (int)max_pos;
  a.eps = eps, a.inv_d = 1.0f / (float)d;
  a.qw = static_cast<const uint16_t*>(q_w);
  a.kw = static_cast<const uint16_t*>(k_w);
  a.cos_sin = cos_sin;
  a.positions = positions;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_out = static_cast<uint16_t*>(k_out);
  a.status = status_dev;
  return hip_status(qg::launch_qk_norm_rope(a, static_cast<hipStream_t>(stream)));
}

int32_t qg_kv8_append(const void* k, int64_t k_ts, int64_t k_hs, const void* v, int64_t v_ts, int64_t v_hs,
                      int64_t rows, int8_t* codes, float* scales, int64_t pages, int32_t hkv, int32_t d,
                      const int32_t* block_table, int64_t table_width, const int32_t* lens, const int32_t* cu,
                      int64_t b, int64_t max_new, uint32_t* status_dev, void* stream) {
  int32_t st = check_cache(codes, scales, pages, hkv, d, block_table, table_width, lens, b);
  if (st == QG_OK) st = check_rows(rows, cu, b);
  if (st != QG_OK) return st;
  if (max_new < 0 || (max_new + QG_KV8_PAGE - 2) / QG_KV8_PAGE + 1 > kMaxGrid) return QG_E_SHAPE;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(status_dev, 4)) return QG_E_ALIGN;
  if (rows == 0 || max_new == 0) return QG_OK;
  if (!k || !v) return QG_E_NULL;
  if (!strides_ok(k_ts, k_hs, rows, hkv, d) || !strides_ok(v_ts, v_hs, rows, hkv, d)) return QG_E_STRIDE;
  const qg::Kv8Args c = cache_args(codes, scales, pages, hkv, d, block_table, table_width, lens, cu, rows, b);
  return hip_status(qg::launch_kv8_append(c, k, k_ts, k_hs, v, v_ts, v_hs, max_new, status_dev,
                                          static_cast<hipStream_t>(stream)));
}

int32_t qg_kv8_read(const int8_t* codes, const float* scales, int64_t pages, int32_t hkv, int32_t d,
                    const int32_t* block_table, int64_t table_width, const int32_t* lens, int64_t b, int64_t max_len,
                    void* k_out, void* v_out, int32_t out_dtype, void* stream) {
  int32_t st = check_cache(codes, scales, pages, hkv, d, block_table, table_width, lens, b);
  if (st != QG_OK) return st;
  if (max_len < 0 || (max_len + QG_KV8_PAGE - 1) / QG_KV8_PAGE > kMaxGrid) return QG_E_SHAPE;
  if (out_dtype != QG_BF16 && out_dtype != QG_F32) return QG_E_DTYPE;
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return QG_E_ALIGN;
  if (max_len == 0) return QG_OK;
  if (!k_out || !v_out) return QG_E_NULL;
  const qg::Kv8Args c = cache_args(codes, scales, pages, hkv, d, block_table, table_width, lens, nullptr, 0, b);
  return hip_status(qg::launch_kv8_read(c, max_len, k_out, v_out, out_dtype == QG_F32,
                                        static_cast<hipStream_t>(stream)));
}

int64_t qg_attn_kv8_workspace_bytes(int64_t b, int64_t rows, int32_t hq, int32_t hkv, int32_t d, int64_t max_q,
                                    int64_t max_len, int32_t window, int32_t splits) {
  qg::AttnSplit by;
  const int32_t st = attn_shape(b, rows, hq, hkv, d, max_q, max_len, window, splits, &by);
  return st != QG_OK ? st : attn_ws(b, rows, hq, d, max_q, by);
}

int32_t qg_attn_kv8(const void* q, int64_t q_ts, int64_t q_hs, int64_t rows, int32_t hq, const int8_t* codes,
                    const float* scales, int64_t pages, int32_t hkv, int32_t d, const int32_t* block_table,
                    int64_t table_width, const int32_t* lens, const int32_t* cu, int64_t b, int64_t max_q,
                    int64_t max_len, int32_t window, float scale, void* out, int32_t out_dtype, int32_t splits,
                    void* ws, int64_t ws_bytes, uint32_t* status_dev, void* stream) {
  int32_t st = check_cache(codes, scales, pages, hkv, d, block_table, table_width, lens, b);
  if (st == QG_OK) st = check_rows(rows, cu, b);
  if (st != QG_OK) return st;
  qg::AttnSplit by;
  st = attn_shape(b, rows, hq, hkv, d, max_q, max_len, window, splits, &by);
  if (st != QG_OK) return st;
  if (out_dtype != QG_BF16 && out_dtype != QG_F32) return QG_E_DTYPE;
  if (std::isnan(scale) || std::isinf(scale)) return QG_E_SHAPE;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(ws, 16) || !aligned(status_dev, 4)) return QG_E_ALIGN;
  if (rows == 0) return QG_OK;
  if (!q || !out) return QG_E_NULL;
  if (!strides_ok(q_ts, q_hs, rows, hq, d)) return QG_E_STRIDE;
  const int64_t need = attn_ws(b, rows, hq, d, max_q, by);
  if (need > 0 && (!ws || ws_bytes < need)) return ws ? QG_E_BUFFER : QG_E_NULL;
  const qg::Kv8Args c = cache_args(codes, scales, pages, hkv, d, block_table, table_width, lens, cu, rows, b);
  return hip_status(qg::launch_attn_kv8(c, q, q_ts, q_hs, hq, (int)max_q, max_len, window, scale, out,
                                        out_dtype == QG_F32, by,
                                        static_cast<float*>(ws), status_dev, static_cast<hipStream_t>(stream)));
}

int64_t qg_moe_w4a16_workspace_bytes(int64_t t, int64_t h, int64_t e, int64_t inter, int64_t top_k) {
  const int32_t st = moe_shape(t, h, e, inter, top_k);
  return st != QG_OK ? st : qg::moe_ws_bytes(t, h, e, inter, top_k);
}

int32_t qg_moe_w4a16(const void* x_bf16, int64_t t, int64_t h, const void* router_bf16, int64_t e, const void* gate_up,
                     int64_t gate_up_bytes, const void* down, int64_t down_bytes, int64_t inter, int64_t top_k,
                     int32_t renormalize, void* y, int32_t y_dtype, void* ws, int64_t ws_bytes, void* stream) {
  const int32_t st = moe_check(x_bf16, t, h, e, gate_up, gate_up_bytes, down, down_bytes, inter, top_k, y, y_dtype, ws);
  if (st != QG_OK) return st;
  if (!aligned(router_bf16, 16)) return QG_E_ALIGN;
  if (t == 0) return QG_OK;
  if (!x_bf16 || !router_bf16 || !gate_up || !down || !y || !ws) return QG_E_NULL;
  if (ws_bytes < qg::moe_ws_bytes(t, h, e, inter, top_k)) return QG_E_BUFFER;
  return hip_status(qg::launch_moe_w4a16(x_bf16, (int)t, (int)h, router_bf16, (int)e, gate_up,
                                         qg_int4_packed_bytes(2 * inter, h), down, qg_int4_packed_bytes(h, inter),
                                         (int)inter, (int)top_k, renormalize != 0, y, y_dtype == QG_F32, ws, nullptr,
                                         nullptr, nullptr, static_cast<hipStream_t>(stream)));
}

int32_t qg_moe_w4a16_picked(const void* x_bf16, int64_t t, int64_t h, const int32_t* ids, const float* weights,
                            int64_t e, const void* gate_up, int64_t gate_up_bytes, const void* down,
                            int64_t down_bytes, int64_t inter, int64_t top_k, void* y, int32_t y_dtype, void* ws,
                            int64_t ws_bytes, uint32_t* status_dev, void* stream) {
  const int32_t st = moe_check(x_bf16, t, h, e, gate_up, gate_up_bytes, down, down_bytes, inter, top_k, y, y_dtype, ws);
  if (st != QG_OK) return st;
  if (!aligned(ids, 4) || !aligned(weights, 4) || !aligned(status_dev, 4)) return QG_E_ALIGN;
  if (t == 0) return QG_OK;
  if (!x_bf16 || !ids || !weights || !gate_up || !down || !y || !ws) return QG_E_NULL;
  if (ws_bytes < qg::moe_ws_bytes(t, h, e, inter, top_k)) return QG_E_BUFFER;
  return hip_status(qg::launch_moe_w4a16(x_bf16, (int)t, (int)h, nullptr, (int)e, gate_up,
                                         qg_int4_packed_bytes(2 * inter, h), down, qg_int4_packed_bytes(h, inter),
                                         (int)inter, (int)top_k, 0, y, y_dtype == QG_F32, ws, ids, weights, status_dev,
                                         static_cast<hipStream_t>(stream)));
}

}  // extern "C"
