/*
 * qgemm.h -- C ABI of the MI355X (gfx950) decode-time weight-only quantized
 * linear layer:   y[m, n] = sum_k x[m, k] * dequant(W)[n, k]  (* scale[n]).
 *
 * Pages this library implements (cited by title and section):
 *  [P1] executorch "backends/cuda/tests/test_int4_quantized_gemm.py":
 *       `_packed_with_dense` (INT4, group 32, asymmetric, min-max),
 *       module docstring and `_dequant_matmul` (dequant + F.linear reference),
 *       `Int4QuantizedGemmLegalityTest` (validate before launching: dtype,
 *       shape, "K must be a multiple of 256", static M), `Int4QuantizedGemmRulesTest.
 *       test_split_k_needs_one_k_tile_per_split` (split <= K / 256),
 *       `SUPPORTED_BUCKETS` (decode M up to 64), `Int4QuantizedGemmTest.
 *       test_cuda_graph_replay_matches_eager` (bit-identical replays),
 *       `Int4QuantizedGemmPrecisionTest` (int8 activations, W4A8).
 *  [P3] gpt-fast issue #114 "Question about the generated code of
 *       WeightOnlyInt8Linear": `WeightOnlyInt8Linear.forward`
 *       (y = F.linear(x, W.to(bf16)) * scales; the int8->bf16 convert must be
 *       fused into the GEMV, never materialized).
 *
 * Conventions for every entry point:
 *  - All data pointers are DEVICE pointers (HIP global memory) on the current
 *    device, 16-byte aligned; arrays are row-major and contiguous.
 *    bf16 / fp16 values are their 16-bit IEEE patterns.
 *  - `stream` is a hipStream_t (NULL = the default stream).  Calls are
 *    asynchronous on that stream; the library never allocates, never
 *    synchronizes, and keeps no mutable global state (calls are re-entrant),
 *    with one exception: qgemm_w4a16_noalloc, which uses the library's own
 *    static device scratch (see there).
 *  - The caller owns every buffer.  Outputs must not alias inputs.
 *  - On an argument error the call returns a negative qg_status and launches
 *    nothing (the checks run on the host before any launch).  A HIP launch
 *    failure returns QG_E_HIP.  Data-dependent conditions (non-finite
 *    weights, scale overflow) are reported through the optional device word
 *    `status_dev`: kernels OR flag bits into it; the caller zeroes it first.
 *  - Results are deterministic: identical inputs, split and device give
 *    bit-identical outputs, eager or replayed from a HIP graph (no floating
 *    point atomics anywhere).
 */
#ifndef QGEMM_H
#define QGEMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- packed INT4 group-32 weight layout, version 1 ----------------------
 * The weight is stored as tiles of 64 rows x 256 k (8 groups of 32 per row),
 * each exactly 9472 bytes = 74 lines of 128 bytes:
 *   [0, 8192)     codes: 16-byte chunk of (group j, row r) at (j*64 + r)*16;
 *                 LE dword d of a chunk holds k = 8d+e of the group at nibble
 *                 position p = (e & 1)*4 + (e >> 1), i.e. bits [4p, 4p+4).
 *                 (dword >> 4i) & 0x000F000F then yields the codes of
 *                 k = 8d+2i and 8d+2i+1 in its low and high 16-bit halves.
 *   [8192, 9216)  fp16 scales: row r's 8 scales at 8192 + 16r, group j at +2j
 *   [9216, 9472)  zero points: row r's LE 32-bit word at 9216 + 4r,
 *                 group j in bits [4j, 4j+4)
 * Tiles are row-block major: tile = (n / 64) * (K / 256) + k / 256.  Rows
 * n >= N of the last row block are zero.  A wavefront (64 lanes, lane = row)
 * reads each region as whole 128-byte lines with one 16-byte load per lane. */
#define QG_INT4_LAYOUT_VERSION 1
#define QG_TILE_ROWS 64
#define QG_TILE_K 256
#define QG_TILE_BYTES 9472

/* ---- packed INT4 layout, version 2: scale codes --------------------------
 * The stored form of [P1] `_packed_with_dense`: a group's scale is a uint8
 * code times a per-row fp16 step ([P1] legality rules "scale codes must be
 * uint8", "scale_step must be float16", step shape [N, 1]).  Each 64-row
 * block is a 128-byte head (row r's fp16 step at 2r) followed by K/256 tiles
 * of 8960 bytes = 70 lines:
 *   [0, 8192)     codes, exactly as version 1
 *   [8192, 8704)  scale codes: row r's 8 bytes at 8192 + 8r, group j at +j
 *   [8704, 8960)  zero points: row r's LE 32-bit word at 8704 + 4r, group j
 *                 in bits [4j, 4j+4)
 * Row blocks follow each other; rows n >= N of the last block are zero.
 * 0.546875 bytes per weight + 2 per row (version 1: 0.578125). */
#define QG_DQ_HEAD_BYTES 128
#define QG_DQ_TILE_BYTES 8960
#define QG_GROUP 32
#define QG_MAX_M 64

enum qg_dtype { QG_BF16 = 0, QG_F32 = 1 };

enum qg_status {
    QG_OK = 0,
    QG_E_NULL = -1,        /* a required pointer is NULL */
    QG_E_SHAPE = -2,       /* m, n or k < 1 */
    QG_E_K_MULTIPLE = -3,  /* K % 256 != 0 ([P1] "K must be a multiple of 256") */
    QG_E_M_RANGE = -4,     /* M > 64 ([P1] "static M must be within" the buckets) */
    QG_E_SPLIT = -5,       /* split_k not in {0,1,2,4,8} or split_k > K/256 */
    QG_E_BUFFER = -6,      /* packed_bytes or ws_bytes too small */
    QG_E_ALIGN = -7,       /* a data pointer is not 16-byte aligned */
    QG_E_DTYPE = -8,       /* y_dtype is not QG_BF16 / QG_F32 */
    QG_E_HIP = -9,         /* a HIP launch failed */
    QG_E_BITS = -10,       /* a code width other than 5 or 6 (INT5 / INT6 entry points) */
    QG_E_SCRATCH = -11,    /* qgemm_w4a16_noalloc: the split's partial sums exceed QG_SCRATCH_BYTES */
    QG_E_HEADS = -12,      /* a head size, head count or rotated width the decoder-layer operators do not take */
    QG_E_STRIDE = -13      /* a stride that is no multiple of 8 elements, or is too small */
};

/* status_dev flag bits */
#define QG_FLAG_NONFINITE 1u   /* a weight group/row held Inf or NaN */
#define QG_FLAG_OVERFLOW 2u    /* an INT4 group's range exceeded 15 * 65504 */
#define QG_FLAG_POSITION 4u    /* qg_qk_norm_rope: a position outside the table */
#define QG_FLAG_PAGE 8u        /* kv8_append, attn_kv8: a page that the table or the cache does not hold */
#define QG_FLAG_INDEX 16u      /* an adapter, an expert, a token or row offsets outside what there is */

/* Human-readable name of a qg_status value (static string). */
const char *qg_status_string(int32_t status);

/* Bytes of the packed INT4 buffer for an N x K weight:
 * ceil(N/64) * (K/256) * 9472 (= N*K/2 codes + N*K/32 * 2.5 bytes of fp16
 * scale and 4-bit zero when N % 64 == 0).  Returns a negative qg_status for
 * N < 1, K < 1 or K % 256 != 0. */
int64_t qg_int4_packed_bytes(int64_t n, int64_t k);

/* The split-K factor the library uses when a qgemm call passes split_k = 0
 * (a static table keyed by the shape), or a negative qg_status. */
int32_t qg_default_split_k(int64_t m, int64_t n, int64_t k);

/* The split-K factor qgemm_wn_a16 (INT5 / INT6) uses for split_k = 0: the
 * table above for m <= 4; for m > 4 the smallest split with
 * ceil(n/64) * split >= 400 (at most 8, at most k/256), one step smaller when
 * that leaves under 4 tiles of 256 k per split while ceil(n/64) * split/2
 * still reaches 256.  Negative qg_status on bad arguments. */
int32_t qg_default_split_k_intn(int64_t m, int64_t n, int64_t k);

/* The split-K factor qgemm_w4a8_g32 and qgemm_w4a8_g32_dq use for
 * split_k = 0: qg_default_split_k up to 32 rows; above 32 rows the smallest
 * split with ceil(n/64) * split >= 1200, at most 8 and with at least 3 tiles
 * of 256 k per split (these kernels also multiply in each group's activation
 * scale, and more splits pay).  Negative qg_status on bad arguments. */
int32_t qg_default_split_k_g32(int64_t m, int64_t n, int64_t k);

/* Workspace bytes a qgemm call needs for (m, n, k, split_k): split * m * n * 4
 * (fp32 partial sums) when the split is above 1, else 0.  For split_k = 0
 * the largest need of the defaults is assumed (qg_default_split_k,
 * qg_default_split_k_intn and qg_default_split_k_g32 at m rows), so one
 * workspace serves every entry point's default.  For m > 4 it also holds what the W4A8 entry
 * points need there: m * k * 2 bytes of quantized activations, max(256,
 * 8 * k) bytes of activation scales (per row, or per group of 32 as
 * k/32 x 64 floats) and split * m * n * 4 bytes of partial sums (at split 1
 * too).  Negative qg_status on bad arguments. */
int64_t qg_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t split_k);

/* ---- quantize_int4_g32 ---------------------------------------------------
 * [P1] `_packed_with_dense`: QuantConfig(bits=4, group_size=32,
 * symmetric=False, method="min_max").  For each row n and each group g of 32
 * consecutive k:
 *   lo = min(0, min v), hi = max(0, max v), r = hi - lo  (binary64)
 *   s  = the smallest positive fp16 with 15*s >= r  (1.0 when r == 0)
 *   zp = clamp(rint(-lo / s), 0, 15)                  (binary32, half-even)
 *   q  = clamp(rint(v / s) + zp, 0, 15)
 * and writes (q, s, zp) in the layout above.  Every dequantized value
 * (q - zp) * s lies within s/2 of its input.
 *   w_bf16        in : bf16 [n, k]
 *   packed        out: qg_int4_packed_bytes(n, k) bytes (padding rows zeroed)
 *   packed_bytes  in : size of `packed`
 *   status_dev    in/out, may be NULL: ORed with QG_FLAG_NONFINITE (that
 *                 group: codes 0, scale NaN, zp 0) and QG_FLAG_OVERFLOW
 *                 (that group's scale saturates at 65504).
 * Errors: QG_E_NULL, QG_E_SHAPE, QG_E_K_MULTIPLE, QG_E_BUFFER, QG_E_ALIGN. */
int32_t quantize_int4_g32(const void *w_bf16, int64_t n, int64_t k, void *packed,
                          int64_t packed_bytes, uint32_t *status_dev, void *stream);

/* ---- quantize_int8_rowwise -----------------------------------------------
 * Per-output-channel symmetric int8, the weight format of [P3]
 * `WeightOnlyInt8Linear` (int8 [out, in] plus one scale per output row):
 *   a = max_k |w[n, k]|;  s = the smallest positive bf16 with 127*s >= a
 *   (1.0 when a == 0);  q = clamp(rint(w / s), -127, 127)  (binary32).
 *   w_bf16      in : bf16 [n, k]      q  out: int8 [n, k]
 *   scale_bf16  out: bf16 [n]
 *   status_dev  in/out, may be NULL: QG_FLAG_NONFINITE (that row: q 0, s NaN).
 * Errors: QG_E_NULL, QG_E_SHAPE, QG_E_K_MULTIPLE (K % 256), QG_E_ALIGN. */
int32_t quantize_int8_rowwise(const void *w_bf16, int64_t n, int64_t k, int8_t *q,
                              void *scale_bf16, uint32_t *status_dev, void *stream);

/* ---- qgemm_w4a16 ---------------------------------------------------------
 * [P1] module docstring / `_dequant_matmul`: y = x . dequant(W)^T with the
 * packed INT4 g32 weight above, dequantized in registers (no bf16 copy of W
 * is ever written).  Accumulation is fp32.
 *   x_bf16   in : bf16 [m, k], 1 <= m <= 64      packed  in: [n, k] weight
 *   y        out: [m, n], bf16 (round to nearest even) or fp32 per y_dtype
 *   split_k  0 (library table) or 1, 2, 4, 8 with split_k <= k/256
 *   ws       fp32 workspace of qg_workspace_bytes(m, n, k, split_k) bytes
 *            (NULL allowed when that is 0); contents on return unspecified.
 * M <= 4 runs the VALU GEMV; 5 <= M <= 64 the MFMA kernel (rows padded to
 * 16 and masked).  split_k > 1 adds a second, atomic-free pass that sums the
 * partials in ascending split order.
 * Errors: QG_E_NULL, QG_E_SHAPE, QG_E_K_MULTIPLE, QG_E_M_RANGE, QG_E_SPLIT,
 * QG_E_BUFFER, QG_E_ALIGN, QG_E_DTYPE, QG_E_HIP. */
int32_t qgemm_w4a16(const void *x_bf16, int64_t m, int64_t k, const void *packed,
                    int64_t packed_bytes, int64_t n, void *y, int32_t y_dtype,
                    int32_t split_k, void *ws, int64_t ws_bytes, void *stream);

/* ---- qgemm_w4a16_noalloc -------------------------------------------------
 * For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): qgemm_w4a16
 * without a workspace argument.  The split-K partial sums (split * m * n * 4
 * bytes when the split is above 1) go to a static device array of
 * QG_SCRATCH_BYTES inside the library, one per device, which each device the
 * library runs on holds until the process ends.  The call allocates nothing
 * (no hipMalloc, no hipFree, no allocating library routine); its first call
 * on a device looks the array's address up once (hipGetSymbolAddress).
 * Every call on a device shares that device's array and leaves its
 * contents behind: calls that overlap on one device (concurrent streams,
 * threads) race and must be serialized by the caller.  Nothing in the array
 * needs to start at zero (each call writes every partial it reads).
 * Arguments, kernels, results (bit-identical to qgemm_w4a16 at the same
 * split) and errors as qgemm_w4a16, plus QG_E_SCRATCH when an explicit
 * split_k needs more than QG_SCRATCH_BYTES (nothing is launched); the
 * default split (split_k = 0) always fits. */
#define QG_SCRATCH_BYTES (16 * 1024 * 1024)
int32_t qgemm_w4a16_noalloc(const void *x_bf16, int64_t m, int64_t k, const void *packed,
                            int64_t packed_bytes, int64_t n, void *y, int32_t y_dtype,
                            int32_t split_k, void *stream);

/* Bytes of the version 2 (scale-code) buffer for an N x K weight:
 * ceil(N/64) * (128 + (K/256) * 8960), or a negative qg_status as above. */
int64_t qg_int4_dq_packed_bytes(int64_t n, int64_t k);

/* ---- quantize_int4_g32_dq ------------------------------------------------
 * [P1] `_packed_with_dense` in its stored form (uint8 scale codes with a
 * per-row fp16 `scale_step`).  Per row n, with lo, hi and r of each group as
 * in quantize_int4_g32:
 *   step = the smallest positive fp16 with 3825*step >= max_g r  (3825 =
 *          255*15; 1.0 when every r is 0)
 *   c    = the smallest integer in 1..255 with 15*c*step >= r, per group
 *   s    = c * step  (exact in binary32), then zp and q exactly as in
 *          quantize_int4_g32 with that s.
 * Zero points stay integers 0..15 (a zero_point_step of 1).  Every
 * dequantized value (q - zp) * s lies within s/2 of its input.
 *   w_bf16        in : bf16 [n, k]
 *   packed        out: qg_int4_dq_packed_bytes(n, k) bytes, layout version 2
 *   packed_bytes  in : size of `packed`
 *   status_dev    in/out, may be NULL: QG_FLAG_NONFINITE (that row: step
 *                 NaN, every code 0), QG_FLAG_OVERFLOW (max_g r above
 *                 3825 * 65504: step 65504, codes at most 255).
 * Two launches on `stream` (row steps, then tiles).
 * Errors: QG_E_NULL, QG_E_SHAPE, QG_E_K_MULTIPLE, QG_E_BUFFER, QG_E_ALIGN. */
int32_t quantize_int4_g32_dq(const void *w_bf16, int64_t n, int64_t k, void *packed,
                             int64_t packed_bytes, uint32_t *status_dev, void *stream);

/* ---- qgemm_w4a16_dq ------------------------------------------------------
 * qgemm_w4a16 on a version 2 (scale-code) weight:
 *   y[m, n] = sum_g c[n,g] * step[n] * sum_{k in g} x[m,k] * (q[n,k] - zp[n,g]),
 * dequantized in registers, fp32 accumulation, on the same kernels and
 * buckets as qgemm_w4a16 (1 <= m <= 64).  Arguments, workspace
 * (qg_workspace_bytes) and errors as qgemm_w4a16, with packed_bytes checked
 * against qg_int4_dq_packed_bytes. */
int32_t qgemm_w4a16_dq(const void *x_bf16, int64_t m, int64_t k, const void *packed,
                       int64_t packed_bytes, int64_t n, void *y, int32_t y_dtype,
                       int32_t split_k, void *ws, int64_t ws_bytes, void *stream);

/* ---- INT5 / INT6 group-32 (the pages' INT5/INT6 quantized-GEMM family) ---
 * Executorch pull request #23737 lists INT5 and INT6 layers next to INT4
 * (INT6: 4096x5376, 5376x21504, 6656x19968, 1024x6656); the quantizer
 * recipe is [P1] `_packed_with_dense` with 2^bits - 1 steps:
 *   s  = the smallest positive fp16 with L*s >= r, L = 31 (INT5) or 63 (INT6)
 *   zp = clamp(rint(-lo / s), 0, L);  q = clamp(rint(v / s) + zp, 0, L)
 * (lo, hi, r as in quantize_int4_g32).  Packed layout: tiles of 64 rows x
 * 256 k, row-block major, 8192 + 2048*hb + 1536 bytes (hb = bits - 4; 11776
 * for INT5, 13824 for INT6):
 *   [0, 8192)             the low 4 bits of every code, exactly as version 1
 *   [8192, +2048 hb)      high-bit planes: the (4 hb)-byte chunk of (group j,
 *                         row r) at 8192 + (j*64 + r)*4*hb.  For code dword d
 *                         and pair p (k = 8d+2p even, 8d+2p+1 odd) INT5 keeps
 *                         the even k's bit at 4d + p and the odd k's at
 *                         16 + 4d + p of the LE chunk; INT6 keeps in LE dword
 *                         d/2 the even k's bits b = 0, 1 at 8(d%2) + 2p + b,
 *                         the odd k's 16 higher
 *   [.., +1024)           fp16 scales: row r's 8 at +16r, group j at +2j
 *   [.., +512)            zero points, one byte each: row r at +8r, group j at +j
 * Rows n >= N of the last row block are zero. */
int64_t qg_intn_packed_bytes(int64_t n, int64_t k, int32_t bits);

/* bf16 [n, k] -> the INT5 / INT6 packed weight above.  Arguments, status
 * flags (per group, as quantize_int4_g32, with L*65504 for the overflow) and
 * errors as quantize_int4_g32, plus QG_E_BITS. */
int32_t quantize_intn_g32(const void *w_bf16, int64_t n, int64_t k, int32_t bits, void *packed,
                          int64_t packed_bytes, uint32_t *status_dev, void *stream);

/* y[m, n] = x . dequant(W)^T for an INT5 / INT6 packed weight, 1 <= m <= 64
 * (the INT4 kernels' buckets: M <= 4 GEMVs, 5..64 the matrix cores),
 * dequantized in registers, fp32 accumulation.
 * Arguments, workspace (qg_workspace_bytes) and errors as qgemm_w4a16, with
 * packed_bytes checked against qg_intn_packed_bytes, plus QG_E_BITS. */
int32_t qgemm_wn_a16(const void *x_bf16, int64_t m, int64_t k, int32_t bits, const void *packed,
                     int64_t packed_bytes, int64_t n, void *y, int32_t y_dtype, int32_t split_k,
                     void *ws, int64_t ws_bytes, void *stream);

/* ---- qgemm_w8a16 ---------------------------------------------------------
 * [P3] `WeightOnlyInt8Linear.forward`: y[m, n] = (sum_k x[m,k] * W[n,k]) *
 * scale[n], fp32 accumulation, the int8 -> float convert fused into the dot
 * product.  W int8 [n, k] row-major as given (no repacking, 16-byte aligned),
 * scale bf16 [n] (2-byte aligned).
 *   x_bf16 in: bf16 [m, k], 1 <= m <= 64;  y out: [m, n] bf16 or fp32.
 * M <= 4 runs the VALU GEMV (k <= 65536, QG_E_SHAPE above); 5 <= M <= 64 the
 * matrix cores (the [P3] question of a fused kernel above batch size 1):
 * bf16 products of x with the exact w + 128, accumulated over all of K, then
 * y = s * (sum - 128 * sum_k x).
 * Errors: QG_E_NULL, QG_E_SHAPE, QG_E_K_MULTIPLE, QG_E_M_RANGE, QG_E_ALIGN,
 * QG_E_DTYPE, QG_E_HIP. */
int32_t qgemm_w8a16(const void *x_bf16, int64_t m, int64_t k, const int8_t *w,
                    const void *scale_bf16, int64_t n, void *y, int32_t y_dtype,
                    void *stream);

/* ---- qgemm_w4a8 ----------------------------------------------------------
 * [P1] `Int4QuantizedGemmPrecisionTest`: the decode kernels run the packed
 * INT4 weight against int8 activations.  Each row of x is quantized inside
 * the call (per-row symmetric absmax: a = max|x|, inv = 127/a, sx = a/127,
 * xq = clamp(rint(x * inv), -127, 127) in binary32; a == 0, and a row so
 * small that 127/a overflows binary32 (a <= 127 * 2^-128), give a zero row;
 * a row holding a NaN or an infinity gives a NaN row),
 * then  y[m,n] = sx[m] * sum_g s[n,g] * sum_{k in g} xq[m,k] * (q[n,k] - zp[n,g])
 * with exact integer group dots.  Arguments and errors as qgemm_w4a16
 * (1 <= m <= 64).  For m > 4 the call quantizes x once into the workspace
 * (xq held exactly as bf16 integers), runs the bf16 matrix-core kernel of
 * qgemm_w4a16 on it (exact products, the same integer group dots), and
 * applies sx after the split-K sum; the workspace is required there at any
 * split (qg_workspace_bytes).  The per-row scale is
 * the pages' precision class on gaussian activations; rows with a few large
 * outlier channels lose precision (qgemm_w4a8_g32 below keeps it). */
int32_t qgemm_w4a8(const void *x_bf16, int64_t m, int64_t k, const void *packed,
                   int64_t packed_bytes, int64_t n, void *y, int32_t y_dtype,
                   int32_t split_k, void *ws, int64_t ws_bytes, void *stream);

/* ---- qgemm_w4a8_g32 ------------------------------------------------------
 * [P1] `Int4QuantizedGemmPrecisionTest` with its outlier activations
 * (channels 0, K/3, 2K/3, K-1 scaled by 50, 35, 25, 20): W4A8 with one
 * activation scale per group of 32 consecutive k of a row, so an outlier
 * only coarsens its own group.  Per row m and group g:
 *   a = max |x[m, 32g .. 32g+31]|, inv = 127/a, sx[m,g] = a/127 (binary32),
 *   xq = clamp(rint(x * inv), -127, 127); a == 0 or 127/a overflowing gives a
 *   zero group, a NaN or an infinity in the group a NaN row;
 *   y[m,n] = sum_g sx[m,g] * s[n,g] * sum_{k in g} xq[m,k] * (q[n,k] - zp[n,g]).
 * Arguments, buffers, workspace and errors as qgemm_w4a8.  For m = 5..64 the
 * call quantizes x once into the workspace (xq as exact bf16 integers, the
 * group scales group-major) and runs the matrix-core kernel of qgemm_w4a16
 * on xq, multiplying each group's exact integer dot by s[n,g] * sx[m,g]: one
 * pass over the weight; the workspace is required there at any split
 * (qg_workspace_bytes). */
int32_t qgemm_w4a8_g32(const void *x_bf16, int64_t m, int64_t k, const void *packed,
                       int64_t packed_bytes, int64_t n, void *y, int32_t y_dtype,
                       int32_t split_k, void *ws, int64_t ws_bytes, void *stream);

/* ---- qgemm_w4a8_dq / qgemm_w4a8_g32_dq -----------------------------------
 * qgemm_w4a8 and qgemm_w4a8_g32 on a version 2 (scale-code) weight: the
 * same activation quantization, a group's weight scale c[n,g] * step[n]:
 *   per row:      y = sx[m] * sum_g c*step * sum_{k in g} xq (q - zp)
 *   per group 32: y = sum_g sx[m,g] * c*step * sum_{k in g} xq (q - zp).
 * Arguments, workspace and errors as qgemm_w4a8 and qgemm_w4a8_g32
 * (1 <= m <= 64, the same two forms above 4 rows), with
 * packed_bytes checked against qg_int4_dq_packed_bytes. */
int32_t qgemm_w4a8_dq(const void *x_bf16, int64_t m, int64_t k, const void *packed,
                      int64_t packed_bytes, int64_t n, void *y, int32_t y_dtype,
                      int32_t split_k, void *ws, int64_t ws_bytes, void *stream);
int32_t qgemm_w4a8_g32_dq(const void *x_bf16, int64_t m, int64_t k, const void *packed,
                          int64_t packed_bytes, int64_t n, void *y, int32_t y_dtype,
                          int32_t split_k, void *ws, int64_t ws_bytes, void *stream);

/* ---- qgemm_w4a8_rows -----------------------------------------------------
 * The W4A8 calls above on rows that come quantized (qg_rms_norm_q8, or codes of the
 * caller's): no pass over x for its scales.
 *   xq       in : int8 [m, k];   scales in : fp32 [m], or [m, k / 32] with
 *                 group_scales not 0; value = code * scale
 *   packed   in : version 1, or version 2 with scale_codes not 0
 * The sums are those of qgemm_w4a8 (qgemm_w4a8_g32) for the same codes and
 * scales.  Other arguments, workspace and errors as there. */
int32_t qgemm_w4a8_rows(const int8_t *xq, const float *scales, int32_t group_scales, int64_t m, int64_t k,
                        const void *packed, int64_t packed_bytes, int32_t scale_codes, int64_t n, void *y,
                        int32_t y_dtype, int32_t split_k, void *ws, int64_t ws_bytes, void *stream);

/* ==========================================================================
 * Operators of a decoder layer around the quantized linears.  They follow the
 * conventions above (device pointers, caller's stream and buffers, checks
 * before any launch, bit-identical repeats).  They are this library's own:
 * the pages it implements stop at the linear layer.
 * ======================================================================= */

/* ---- qg_qk_norm_rope -----------------------------------------------------
 * RMS norm of every query and key head and the rotation of its first `rot`
 * channels by position, in one pass, fp32, rounded once to bf16:
 *   x' = x * rsqrt(mean(x^2) + eps) * w
 *   (a, b) -> (a cos - b sin, b cos + a sin)
 * with (a, b) = channels (i, rot/2 + i), or (2i, 2i + 1) where adjacent_pairs
 * is not 0, and cos, sin = cos_sin[position][i], cos_sin[position][rot/2 + i].
 *   q, k       in : bf16 [tokens, hq, d] and [tokens, hkv, d]; strides in
 *                   elements per token and per head (multiples of 8; channels
 *                   contiguous), so both may be columns of one projection
 *   q_w, k_w   in : bf16 [d], or NULL for a norm without weights
 *   cos_sin    in : fp32 [max_pos, rot]       positions in : int32 [tokens]
 *   q_out      out: bf16 [tokens, hq, d], k_out bf16 [tokens, hkv, d]
 *   status_dev    : QG_FLAG_POSITION where a position is outside [0, max_pos)
 *                   (that token's heads become NaN); may be NULL
 * d: a multiple of 16 up to 512; rot: a multiple of 16 up to d (0: no
 * rotation).  tokens = 0 is fine; so are hq = 0 or hkv = 0 with their
 * pointers NULL.
 * Errors: QG_E_NULL, QG_E_SHAPE, QG_E_HEADS, QG_E_STRIDE, QG_E_ALIGN. */
int32_t qg_qk_norm_rope(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k,
                        int64_t k_token_stride, int64_t k_head_stride, int64_t tokens, int32_t hq,
                        int32_t hkv, int32_t d, const void *q_w, const void *k_w, const float *cos_sin,
                        int64_t max_pos, int32_t rot, int32_t adjacent_pairs, const int32_t *positions,
                        float eps, void *q_out, void *k_out, uint32_t *status_dev, void *stream);

/* ---- the 8-bit key/value cache -------------------------------------------
 * Pages of 64 tokens of every key/value head, as int8 codes with one fp32
 * scale per block of 16 tokens, head, and keys / values; a value is code *
 * scale.  d is 64, 128, 192 or 256.
 *   codes  int8 [pages, hkv, 2, 64 d]: keys, then values.  Channel c of token
 *          t of the page: keys at t d + c; values at
 *          64 c + 16 ((t % 16) / 4) + 4 (t / 16) + t % 4
 *          (a channel's 64 tokens together, in the order in which one lane of
 *          the attention kernel needs them).
 *   scales fp32 [pages, hkv, 2, 4]: block t / 16.
 * A sequence's tokens [64 i, 64 i + 64) are in page block_table[b][i] (int32
 * [b, table_width]; entries past its length are not read).  lens: int32 [b],
 * tokens of each sequence.  Rows of new tokens or queries lie one sequence
 * after another: sequence b has rows cu[b] .. cu[b + 1] - 1 (int32 [b + 1]),
 * or rows / b each where cu is NULL (rows a multiple of b); they are its last
 * tokens, so the last row is token lens[b] - 1.  Rows before token 0 (more
 * rows than tokens) are skipped by the append and see nothing.
 * A page that is not there (a table column past table_width, or an entry
 * outside [0, pages)) is never read or written: its tokens are lost to an
 * append and NaN to a read or an attention; the append and the attention set
 * QG_FLAG_PAGE (a read has no status word). */
#define QG_KV8_PAGE 64
#define QG_KV8_BLOCK 16

/* Quantizes rows of new keys and values into the cache.  For a block of 16
 * tokens, s_held its scale where it holds a token from before this call (else
 * 0), a = max |x| over its new tokens, in binary32:
 *   s = max(s_held, a * (1/127));  held codes q <- rint(q * (s_held / s))
 *   where s > s_held;  new codes q = clamp(rint(x / s), -127, 127), 0 for s = 0.
 * A new value that is an infinity or a NaN makes its block's scale NaN.
 * Codes after the last token of a written block are unspecified.  Writing the
 * same rows again changes nothing.  A page belongs to one sequence of a call.
 * A shorter length drops tokens, not what they did to a block that keeps others:
 * its scale and the held codes' rounding stay (NaN, too, where a dropped value was
 * none).  A caller that feeds drafted tokens and wants the cache as without the
 * rejected ones puts back, from a copy of before the append, the codes and scales of
 * the page that its last token then was in, and appends the accepted rows to that.
 *   k, v       in : bf16 [rows, hkv, d], strides as qg_qk_norm_rope
 *   lens       in : lengths with the new tokens counted
 *   max_new    in : no sequence has more new rows (a sequence's rows from
 *                   max_new on are not written)
 *   status_dev    : QG_FLAG_NONFINITE, QG_FLAG_PAGE; may be NULL
 * Errors: QG_E_NULL, QG_E_SHAPE, QG_E_HEADS, QG_E_STRIDE, QG_E_ALIGN. */
int32_t qg_kv8_append(const void *k, int64_t k_token_stride, int64_t k_head_stride, const void *v,
                      int64_t v_token_stride, int64_t v_head_stride, int64_t rows, int8_t *codes,
                      float *scales, int64_t pages, int32_t hkv, int32_t d, const int32_t *block_table,
                      int64_t table_width, const int32_t *lens, const int32_t *cu, int64_t b,
                      int64_t max_new, uint32_t *status_dev, void *stream);

/* Reads sequences back: k_out, v_out [b, max_len, hkv, d] in bf16 or fp32
 * (out_dtype); tokens at or past a sequence's length are zero. */
int32_t qg_kv8_read(const int8_t *codes, const float *scales, int64_t pages, int32_t hkv, int32_t d,
                    const int32_t *block_table, int64_t table_width, const int32_t *lens, int64_t b,
                    int64_t max_len, void *k_out, void *v_out, int32_t out_dtype, void *stream);

/* ---- qg_attn_kv8 ---------------------------------------------------------
 * Attention of every query row over its sequence in the cache:
 *   out[r, h] = sum_j softmax_j(scale * q[r, h] . k_j) v_j
 * over the tokens j <= p (the row's own token p) and, where window > 0 (up to
 * 2^30), j > p - window; head h of hq reads key/value head h / (hq / hkv).  A row
 * that sees no token (length 0, or a row before token 0) is zero.  Softmax and
 * sums are fp32; the products' operands are fp16: q scaled by a power of two
 * per row, the codes (exact), and probability times value scale, rounded once
 * to 11 bits (where it is below 2^-27 of the largest that the row itself sees: to
 * 2^-38 of that).  A key or value scale that is infinite or NaN makes the rows
 * that see its block NaN, and no others.
 *   q        in : bf16 [rows, hq, d], strides as qg_qk_norm_rope
 *   max_q    in : no sequence has more query rows (later ones are not written)
 *   max_len  in : an upper bound of lens, for the choice of the split only
 *   out      out: [rows, hq, d], bf16 or fp32 (out_dtype)
 *   splits   in : workgroups that share a sequence's pages, 1..256; 0 lets
 *                 the library choose, by the sequences' lengths where that pays
 *   ws          : qg_attn_kv8_workspace_bytes(...) bytes, NULL allowed for 0
 *   status_dev  : QG_FLAG_PAGE; may be NULL
 * Rows are query tokens of decode: 1 for a step, a few for the verification of
 * drafted tokens.  Longer chunks are right, but every 32 of a head's rows read
 * the cache anew.
 * Errors: QG_E_NULL, QG_E_SHAPE, QG_E_HEADS, QG_E_STRIDE, QG_E_ALIGN,
 * QG_E_DTYPE, QG_E_SPLIT, QG_E_BUFFER. */
int64_t qg_attn_kv8_workspace_bytes(int64_t b, int64_t rows, int32_t hq, int32_t hkv, int32_t d,
                                    int64_t max_q, int64_t max_len, int32_t window, int32_t splits);
int32_t qg_attn_kv8(const void *q, int64_t q_token_stride, int64_t q_head_stride, int64_t rows, int32_t hq,
                    const int8_t *codes, const float *scales, int64_t pages, int32_t hkv, int32_t d,
                    const int32_t *block_table, int64_t table_width, const int32_t *lens, const int32_t *cu,
                    int64_t b, int64_t max_q, int64_t max_len, int32_t window, float scale, void *out,
                    int32_t out_dtype, int32_t splits, void *ws, int64_t ws_bytes, uint32_t *status_dev,
                    void *stream);

/* ---- qg_moe_w4a16 --------------------------------------------------------
 * A whole mixture-of-experts layer for t <= 64 tokens on packed INT4 experts:
 *   l = x . router^T;  the top_k experts of a token by l (ties go to the
 *   lowest index; a NaN counts as the largest);
 *   p = softmax of l over the picked experts (renormalize not 0) or over all;
 *   y = sum over the picked e of p_e * down_e . (silu(gate_e x) * (up_e x)).
 * Each expert's products are qgemm_w4a16's on its weight; the hidden
 * activation is rounded to bf16 as the second product's operand (t <= 4: kept as
 * the sum of two bf16), all sums, logits and weights are fp32; above 4 tokens
 * the picks are added in order of rank.
 *   x        in : bf16 [t, h]          router in : bf16 [e, h]
 *   gate_up  in : e packed weights of 2 inter x h (quantize_int4_g32), one
 *                 after another: gate rows 0 .. inter - 1, then up rows
 *   down     in : e packed weights of h x inter
 *   y        out: [t, h], bf16 or fp32 (y_dtype)
 *   ws          : qg_moe_w4a16_workspace_bytes(...) bytes; contents unspecified
 * h, inter: multiples of 256; e <= 512; top_k <= 32.  t = 0 is fine.
 * Errors: QG_E_NULL, QG_E_SHAPE, QG_E_K_MULTIPLE, QG_E_M_RANGE, QG_E_BUFFER,
 * QG_E_ALIGN, QG_E_DTYPE. */
int64_t qg_moe_w4a16_workspace_bytes(int64_t t, int64_t h, int64_t e, int64_t inter, int64_t top_k);
int32_t qg_moe_w4a16(const void *x_bf16, int64_t t, int64_t h, const void *router_bf16, int64_t e,
                     const void *gate_up, int64_t gate_up_bytes, const void *down, int64_t down_bytes,
                     int64_t inter, int64_t top_k, int32_t renormalize, void *y, int32_t y_dtype, void *ws,
                     int64_t ws_bytes, void *stream);

/* ---- qg_moe_w4a16_picked -------------------------------------------------
 * The experts' part of qg_moe_w4a16 on picks and weights that come with the call
 * (qg_moe_route, or the caller's):
 *   y = sum over the picks j of weights[t][j] * down_e . (silu(gate_e x) * (up_e x)),  e = ids[t][j]
 *   ids      in : int32 [t, top_k];  weights in : fp32 [t, top_k]
 *   status_dev  : QG_FLAG_INDEX; may be NULL
 * A negative id is no pick.  One of e or more, or one that an earlier pick of the same
 * token has, counts for nothing and sets QG_FLAG_INDEX.  Other arguments, workspace
 * and errors as qg_moe_w4a16. */
int32_t qg_moe_w4a16_picked(const void *x_bf16, int64_t t, int64_t h, const int32_t *ids, const float *weights,
                            int64_t e, const void *gate_up, int64_t gate_up_bytes, const void *down,
                            int64_t down_bytes, int64_t inter, int64_t top_k, void *y, int32_t y_dtype,
                            void *ws, int64_t ws_bytes, uint32_t *status_dev, void *stream);

/* ==========================================================================
 * Operators of a serving step beside the linears.  The conventions above
 * hold, but for alignment: ids, scales, y and out of qg_lora_add, all arrays of
 * qg_moe_route, and those of qg_verify_drafts but its workspace need that of their
 * elements only; codes of qg_rms_norm_q8 8 bytes, its scales 4.
 * ======================================================================= */

/* ---- qg_rms_norm / qg_rms_norm_q8 ----------------------------------------
 * A sub-layer's output added to the residual stream, and the RMS norm of the sum:
 *   r = x + residual;   y = r * rsqrt(mean(r^2) + eps) * w
 * in binary32.  The norm takes the sum before it is rounded to the stream's type;
 * y is rounded once, to y_dtype or to the 8-bit rows of qgemm_w4a8_rows:
 *   a = max |y| of the row, or of each 32 channels where group_scales is not 0,
 *   inv = 127/a, scale = a/127, code = clamp(rint(y * inv), -127, 127)
 * with the rules of qgemm_w4a8 for spans that are zero, too small for 127/a, or
 * not finite (scale NaN).
 *   x            in : [rows, h], bf16 or fp32 (x_dtype), rows x_row_stride apart
 *   residual     in : the same shape in either type, or NULL: r = x, not stored
 *   w            in : bf16 [h], or NULL for a norm without weights
 *   residual_out out: r [rows, h], contiguous, in the residual's type; NULL without
 *                     a residual.  It may be `residual` itself (contiguous).
 *   y            out: [rows, h], bf16 or fp32 (y_dtype).  It may be x itself (contiguous,
 *                     same type).
 *   codes        out: int8 [rows, h];   scales out: fp32 [rows] or [rows, h / 32]
 * h: a multiple of 8 (group_scales: of 32) up to 32768; strides: multiples of 8;
 * rows < 2^22.  rows = 0 is fine.
 * Errors: QG_E_NULL, QG_E_SHAPE, QG_E_STRIDE, QG_E_ALIGN, QG_E_DTYPE. */
int32_t qg_rms_norm(const void *x, int32_t x_dtype, int64_t x_row_stride, const void *residual,
                    int32_t residual_dtype, int64_t residual_row_stride, int64_t rows, int64_t h,
                    const void *w, float eps, void *y, int32_t y_dtype, void *residual_out, void *stream);
int32_t qg_rms_norm_q8(const void *x, int32_t x_dtype, int64_t x_row_stride, const void *residual,
                       int32_t residual_dtype, int64_t residual_row_stride, int64_t rows, int64_t h,
                       const void *w, float eps, int8_t *codes, float *scales, int32_t group_scales,
                       void *residual_out, void *stream);

/* ---- qg_lora_add ---------------------------------------------------------
 * Low-rank adapters of many requests beside a shared projection:
 *   out[m] = y[m] + s_i * (x[m] . A_i^T) . B_i^T,   i = ids[m];   out[m] = y[m] for i < 0
 * for m <= 64 rows, as the linears take.  Sums are fp32; the inner value enters the
 * second product with 24 bits.  Every adapter that a row names is read once.
 *   x       in : bf16 [m, k]
 *   a, b    in : bf16 [adapters, r, k] and [adapters, n, r]
 *   ids     in : int32 [m]; one of `adapters` or more makes its row NaN and sets
 *                QG_FLAG_INDEX
 *   scales  in : fp32 [adapters], or NULL for 1
 *   y       in : [m, n], bf16 or fp32, rows y_row_stride elements apart
 *   out     out: [m, n], bf16 or fp32, rows out_row_stride apart; it may be y itself
 *                (same type and stride)
 *   ws         : qg_lora_add_workspace_bytes(...) bytes; contents unspecified
 *   status_dev : QG_FLAG_INDEX; may be NULL
 * r: a multiple of 8 up to 256 (lower ranks padded with zeros); k: a multiple of 8;
 * n: any; both up to 2^20.  m = 0 is fine.
 * Errors: QG_E_NULL, QG_E_SHAPE, QG_E_M_RANGE, QG_E_STRIDE, QG_E_ALIGN, QG_E_DTYPE,
 * QG_E_BUFFER. */
#define QG_LORA_MAX_RANK 256
#define QG_LORA_MAX_DIM (1 << 20)
int64_t qg_lora_add_workspace_bytes(int64_t m, int64_t k, int64_t n, int64_t r, int64_t adapters);
int32_t qg_lora_add(const void *x_bf16, int64_t m, int64_t k, const void *a_bf16, const void *b_bf16,
                    int64_t r, int64_t adapters, const int32_t *ids, const float *scales, const void *y,
                    int32_t y_dtype, int64_t y_row_stride, int64_t n, void *out, int32_t out_dtype,
                    int64_t out_row_stride, void *ws, int64_t ws_bytes, uint32_t *status_dev, void *stream);

/* ---- qg_moe_route --------------------------------------------------------
 * The choice of experts from a router's logits l [t, e]:
 *   s = softmax(l) over the experts, or 1 / (1 + exp(-l)) (sigmoid not 0)
 *   c = s + bias                     (it decides the choice and does not weigh)
 *   groups > 1: the experts fall into equal groups one after another; a group
 *   counts the sum of its group_best (1 or 2) largest c; the top_groups of them stay
 *   ids = the top_k experts of those by c, largest first
 *   weights = s of the picked, divided by their sum (renormalize not 0), times scale
 * Ties go to the lowest index; a NaN counts as the largest.  Where no bias and no sum
 * of two takes part, experts are in the order of their logits; else scores, sums
 * and comparisons are as in 64 bits, so that the choice is the exact one but for
 * differences in the 16th digit.  Weights are rounded once.  An expert with a logit
 * of -infinity has score 0 (it can be picked where too few others are left); where
 * the picked scores sum to 0, renormalized weights are 0; beside a logit of +infinity
 * a softmax is NaN.
 *   logits  in : [t, e], bf16 or fp32;   bias in : fp32 [e], or NULL
 *   ids     out: int32 [t, top_k];       weights out: fp32 [t, top_k]
 * e <= 512; top_k <= 32 and <= top_groups * e / groups; groups <= 64 divides e.
 * t <= 2^26 - 8; t = 0 is fine.  Errors: QG_E_NULL, QG_E_SHAPE, QG_E_DTYPE,
 * QG_E_ALIGN. */
int32_t qg_moe_route(const void *logits, int32_t logits_dtype, int64_t t, int64_t e, int64_t top_k,
                     int32_t sigmoid, const float *bias, int64_t groups, int64_t top_groups,
                     int32_t group_best, int32_t renormalize, float scale, int32_t *ids, float *weights,
                     void *stream);

/* ---- qg_verify_drafts ----------------------------------------------------
 * Drafted tokens against the target's probabilities, and the next token.
 * Sequence b has rows cu[b] .. cu[b + 1] - 1 of `target`: one for each of its n
 * drafted tokens and one more; and n rows of `draft`, `tokens` and `u`, which lie one
 * sequence after another, from cu[b] - b on.  Draft i, token x, is accepted while
 *   u * draft_i[x] < target_i[x]
 * (draft NULL: the drafts are certain, u < target_i[x]).  At the first that is not, the
 * next token is the first j whose running sum of max(target_i - draft_i, 0)
 * exceeds u_next times the whole sum (draft NULL: of target_i without x); that of
 * max(target_i, 0) where the whole sum is zero; and after the last draft that of the
 * last row.  All in 64 bits: sums of the 512 tokens of a piece or more in binary64, and
 * running sums in whole numbers of 2^-61 of the whole, so that a token without a share is
 * never drawn.  Rows need not add up to one; a NaN counts as 0.
 *   target     in : [rows, v], bf16 or fp32 (dtype)
 *   draft      in : [rows - b, v] in the same type, or NULL
 *   tokens, u  in : int32 and fp32 [rows - b]; u in [0, 1)
 *   u_next     in : fp32 [b], in [0, 1);   cu in : int32 [b + 1]
 *   lens       in/out: int32 [b], less the drafts that were not accepted (the
 *                   lengths that a cache is left with; for the scales of its blocks
 *                   see qg_kv8_append); may be NULL
 *   accepted, next out: int32 [b]
 *   ws            : qg_verify_drafts_workspace_bytes(...) bytes; contents unspecified;
 *                   NULL where that is 0
 *   status_dev    : may be NULL.  QG_FLAG_INDEX: a drafted token outside [0, v) (it is
 *                   rejected), or a sequence whose offsets are not in order or reach
 *                   past the rows (accepted 0, next -1, lens as it was; the others
 *                   as ever); QG_FLAG_NONFINITE: a row to draw from without a
 *                   finite sum above zero (next -1).
 * b <= 65535; b = 0 is fine.
 * Errors: QG_E_NULL, QG_E_SHAPE, QG_E_DTYPE, QG_E_ALIGN, QG_E_BUFFER. */
int64_t qg_verify_drafts_workspace_bytes(int64_t rows, int64_t b, int64_t v);
int32_t qg_verify_drafts(const void *target, const void *draft, int32_t dtype, int64_t rows, int64_t v,
                         const int32_t *tokens, const float *u, const float *u_next, const int32_t *cu,
                         int64_t b, int32_t *lens, int32_t *accepted, int32_t *next, void *ws,
                         int64_t ws_bytes, uint32_t *status_dev, void *stream);

/* ---- qg_stream_read (measurement helper, not part of the layer) ---------
 * Reads `bytes` bytes of device memory at `src` once, with one 16-byte
 * non-temporal load per lane per step over `blocks` workgroups of 256 lanes
 * (2 x 16 bytes per lane per step, grid-strided), and writes one XOR word per
 * wave to `sink` (blocks * 4 uint32).  The plain streaming-read rate of a
 * buffer, against which the GEMVs' effective bandwidth is compared.
 * bytes: a multiple of 16; src 16-byte aligned; 1 <= blocks <= 65536.
 * Errors: QG_E_NULL, QG_E_SHAPE, QG_E_ALIGN, QG_E_HIP. */
int32_t qg_stream_read(const void *src, int64_t bytes, uint32_t *sink, int32_t blocks, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* QGEMM_H */
