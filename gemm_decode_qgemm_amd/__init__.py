"""MI355X (gfx950) decode-time weight-only quantized linear layer.

y = x . dequant(W)^T (. per-row scale) for INT4 group-32 asymmetric weights
(W4A16, W4A8; fp16 group scales, or uint8 scale codes with a per-row
fp16 step as the pages store them), INT5 / INT6 group-32 weights and INT8 per-channel weights (W8A16), M = 1..64 activation rows.
Between the linears of a decoder layer: norms (rms_norm, rms_norm_q8, qk_norm_rope),
an 8-bit paged cache and its attention (kv8_*, attn_kv8), mixtures of experts
(moe_w4a16; moe_route and moe_w4a16_picked), adapters (lora_add) and the verification
of drafted tokens (verify_drafts).
The computation runs in the HIP library libqgemm.so (C ABI: include/qgemm.h);
this package only binds it.
"""
from .binding import (  # noqa: F401
    FLAG_INDEX,
    FLAG_NONFINITE,
    FLAG_OVERFLOW,
    FLAG_PAGE,
    FLAG_POSITION,
    KV8_BLOCK,
    KV8_PAGE,
    QG_BF16,
    QG_F32,
    SCRATCH_BYTES,
    QGemmError,
    attn_kv8,
    attn_kv8_workspace_bytes,
    default_split_k,
    int4_dq_packed_bytes,
    int4_packed_bytes,
    intn_packed_bytes,
    kv8_append,
    kv8_empty,
    kv8_read,
    lora_add,
    lora_add_workspace_bytes,
    moe_route,
    moe_w4a16,
    moe_w4a16_picked,
    moe_w4a16_workspace_bytes,
    qgemm_w4a8,
    qgemm_w4a8_dq,
    qgemm_w4a8_g32,
    qgemm_w4a8_g32_dq,
    qgemm_w4a8_rows,
    qgemm_w4a16,
    qgemm_w4a16_dq,
    qgemm_w4a16_noalloc,
    qgemm_w8a16,
    qgemm_wn_a16,
    qk_norm_rope,
    quantize_int4_g32,
    quantize_int4_g32_dq,
    quantize_int8_rowwise,
    quantize_intn_g32,
    rms_norm,
    rms_norm_q8,
    status_string,
    stream_read,
    verify_drafts,
    verify_drafts_workspace_bytes,
    workspace_bytes,
)
