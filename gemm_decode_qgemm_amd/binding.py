"""ctypes binding of libqgemm.so (the C ABI in include/qgemm.h).

Argument marshalling only: torch tensors supply device pointers and the
current HIP stream; every step of the computation runs in the library's
kernels.  Importing this module fails loudly if the library is not built.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# QGEMM_LIB names another build of the same library (for comparing builds).
LIB_PATH = os.environ.get("QGEMM_LIB") or os.path.join(_PKG, "libqgemm.so")

QG_BF16 = 0
QG_F32 = 1
TILE_ROWS = 64
TILE_K = 256
TILE_BYTES = 9472
GROUP = 32
MAX_M = 64
SCRATCH_BYTES = 16 * 1024 * 1024      # QG_SCRATCH_BYTES of include/qgemm.h
FLAG_NONFINITE = 1
FLAG_OVERFLOW = 2
FLAG_POSITION = 4
FLAG_PAGE = 8
KV8_PAGE = 64                         # tokens of a cache page
KV8_BLOCK = 16                        # tokens that share a scale


class QGemmError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build the HIP library first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    sigs = {
        "qg_status_string": (ctypes.c_char_p, [I32]),
        "qg_int4_packed_bytes": (I64, [I64, I64]),
        "qg_default_split_k": (I32, [I64, I64, I64]),
        "qg_default_split_k_intn": (I32, [I64, I64, I64]),
        "qg_default_split_k_g32": (I32, [I64, I64, I64]),
        "qg_workspace_bytes": (I64, [I64, I64, I64, I32]),
        "qg_int4_dq_packed_bytes": (I64, [I64, I64]),
        "qg_intn_packed_bytes": (I64, [I64, I64, I32]),
        "quantize_intn_g32": (I32, [P, I64, I64, I32, P, I64, P, P]),
        "qgemm_wn_a16": (I32, [P, I64, I64, I32, P, I64, I64, P, I32, I32, P, I64, P]),
        "quantize_int4_g32": (I32, [P, I64, I64, P, I64, P, P]),
        "quantize_int4_g32_dq": (I32, [P, I64, I64, P, I64, P, P]),
        "qgemm_w4a16_dq": (I32, [P, I64, I64, P, I64, I64, P, I32, I32, P, I64, P]),
        "quantize_int8_rowwise": (I32, [P, I64, I64, P, P, P, P]),
        "qgemm_w4a16": (I32, [P, I64, I64, P, I64, I64, P, I32, I32, P, I64, P]),
        "qgemm_w4a16_noalloc": (I32, [P, I64, I64, P, I64, I64, P, I32, I32, P]),
        "qg_stream_read": (I32, [P, I64, P, I32, P]),
        "qgemm_w8a16": (I32, [P, I64, I64, P, P, I64, P, I32, P]),
        "qgemm_w4a8": (I32, [P, I64, I64, P, I64, I64, P, I32, I32, P, I64, P]),
        "qgemm_w4a8_g32": (I32, [P, I64, I64, P, I64, I64, P, I32, I32, P, I64, P]),
        "qgemm_w4a8_dq": (I32, [P, I64, I64, P, I64, I64, P, I32, I32, P, I64, P]),
        "qgemm_w4a8_g32_dq": (I32, [P, I64, I64, P, I64, I64, P, I32, I32, P, I64, P]),
        "qg_qk_norm_rope": (I32, [P, I64, I64, P, I64, I64, I64, I32, I32, I32, P, P, P, I64, I32, I32, P,
                                  ctypes.c_float, P, P, P, P]),
        "qg_kv8_append": (I32, [P, I64, I64, P, I64, I64, I64, P, P, I64, I32, I32, P, I64, P, P, I64, I64, P, P]),
        "qg_kv8_read": (I32, [P, P, I64, I32, I32, P, I64, P, I64, I64, P, P, I32, P]),
        "qg_attn_kv8_workspace_bytes": (I64, [I64, I64, I32, I32, I32, I64, I64, I32, I32]),
        "qg_attn_kv8": (I32, [P, I64, I64, I64, I32, P, P, I64, I32, I32, P, I64, P, P, I64, I64, I64, I32,
                              ctypes.c_float, P, I32, I32, P, I64, P, P]),
        "qg_moe_w4a16_workspace_bytes": (I64, [I64, I64, I64, I64, I64]),
        "qg_moe_w4a16": (I32, [P, I64, I64, P, I64, P, I64, P, I64, I64, I64, I32, P, I32, P, I64, P]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.qg_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != 0:
        raise QGemmError(status, what)


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(index: int) -> int:
    """The current stream of a device by its index, without a Stream object (2 us less a call)."""
    return _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _dev(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA (HIP) device")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must be rank-{ndim}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def int4_packed_bytes(n: int, k: int) -> int:
    v = int(lib.qg_int4_packed_bytes(n, k))
    _check(min(v, 0), "qg_int4_packed_bytes")
    return v


def int4_dq_packed_bytes(n: int, k: int) -> int:
    v = int(lib.qg_int4_dq_packed_bytes(n, k))
    _check(min(v, 0), "qg_int4_dq_packed_bytes")
    return v


def intn_packed_bytes(n: int, k: int, bits: int) -> int:
    v = int(lib.qg_intn_packed_bytes(n, k, bits))
    _check(min(v, 0), "qg_intn_packed_bytes")
    return v


def default_split_k(m: int, n: int, k: int, bits: int = 4, group_scales: bool = False) -> int:
    """The library's split for split_k = 0: INT4 layouts (bits = 4; with
    group_scales, W4A8 with one activation scale per group of 32), or INT5 / INT6."""
    if bits != 4:
        v = int(lib.qg_default_split_k_intn(m, n, k))
    elif group_scales:
        v = int(lib.qg_default_split_k_g32(m, n, k))
    else:
        v = int(lib.qg_default_split_k(m, n, k))
    _check(min(v, 0), "qg_default_split_k")
    return v


def workspace_bytes(m: int, n: int, k: int, split_k: int = 0) -> int:
    v = int(lib.qg_workspace_bytes(m, n, k, split_k))
    _check(min(v, 0), "qg_workspace_bytes")
    return v


def quantize_int4_g32(w: torch.Tensor, status: torch.Tensor | None = None,
                      out: torch.Tensor | None = None) -> torch.Tensor:
    """bf16 [n, k] -> packed INT4 g32 weight (uint8, layout v1)."""
    _dev(w, "w", torch.bfloat16, 2)
    n, k = w.shape
    nbytes = int4_packed_bytes(n, k)
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=w.device)
    st = lib.quantize_int4_g32(w.data_ptr(), n, k, out.data_ptr(), out.numel(), _ptr(status),
                               _stream(w.device))
    _check(st, "quantize_int4_g32")
    return out


def quantize_int4_g32_dq(w: torch.Tensor, status: torch.Tensor | None = None,
                         out: torch.Tensor | None = None) -> torch.Tensor:
    """bf16 [n, k] -> packed INT4 g32 weight with scale codes (uint8, layout v2)."""
    _dev(w, "w", torch.bfloat16, 2)
    n, k = w.shape
    nbytes = int4_dq_packed_bytes(n, k)
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=w.device)
    st = lib.quantize_int4_g32_dq(w.data_ptr(), n, k, out.data_ptr(), out.numel(), _ptr(status),
                                  _stream(w.device))
    _check(st, "quantize_int4_g32_dq")
    return out


def quantize_intn_g32(w: torch.Tensor, bits: int, status: torch.Tensor | None = None,
                      out: torch.Tensor | None = None) -> torch.Tensor:
    """bf16 [n, k] -> packed INT5 / INT6 g32 weight (uint8; bits = 5 or 6)."""
    _dev(w, "w", torch.bfloat16, 2)
    n, k = w.shape
    nbytes = intn_packed_bytes(n, k, bits)
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=w.device)
    st = lib.quantize_intn_g32(w.data_ptr(), n, k, bits, out.data_ptr(), out.numel(), _ptr(status),
                               _stream(w.device))
    _check(st, "quantize_intn_g32")
    return out


def quantize_int8_rowwise(w: torch.Tensor, status: torch.Tensor | None = None,
                          out: tuple | None = None):
    """bf16 [n, k] -> (int8 [n, k], bf16 scale [n]); `out` = (q, scale) to write into."""
    _dev(w, "w", torch.bfloat16, 2)
    n, k = w.shape
    if out is None:
        q = torch.empty((n, k), dtype=torch.int8, device=w.device)
        s = torch.empty(n, dtype=torch.bfloat16, device=w.device)
    else:
        q, s = out
        _dev(q, "q", torch.int8, 2)
        if tuple(q.shape) != (n, k) or s.dtype != torch.bfloat16 or s.numel() != n or not s.is_contiguous():
            raise ValueError("out must be (int8 [n, k], contiguous bf16 [n])")
    st = lib.quantize_int8_rowwise(w.data_ptr(), n, k, q.data_ptr(), s.data_ptr(), _ptr(status),
                                   _stream(w.device))
    _check(st, "quantize_int8_rowwise")
    return q, s


def _out(m: int, n: int, out_dtype: torch.dtype, device, out: torch.Tensor | None) -> tuple:
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=device)
    else:
        _dev(out, "out", out_dtype, 2)
    return out, (QG_F32 if out_dtype == torch.float32 else QG_BF16)


def _workspace(m, n, k, split_k, device, workspace):
    need = workspace_bytes(m, n, k, split_k)
    if need == 0:
        return None, 0
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    return workspace, workspace.numel() * workspace.element_size()


def qgemm_w4a16(x: torch.Tensor, packed: torch.Tensor, n: int, *, split_k: int = 0,
                out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y[m, n] = x . dequant(W)^T for a packed INT4 g32 weight."""
    _dev(x, "x", torch.bfloat16, 2)
    m, k = x.shape
    y, yd = _out(m, n, out_dtype, x.device, out)
    ws, ws_bytes = _workspace(m, n, k, split_k, x.device, workspace)
    st = lib.qgemm_w4a16(x.data_ptr(), m, k, packed.data_ptr(), packed.numel(), n, y.data_ptr(),
                         yd, split_k, _ptr(ws), ws_bytes, _stream(x.device))
    _check(st, "qgemm_w4a16")
    return y


def qgemm_w4a16_noalloc(x: torch.Tensor, packed: torch.Tensor, n: int, *, split_k: int = 0,
                        out_dtype: torch.dtype = torch.bfloat16,
                        out: torch.Tensor | None = None) -> torch.Tensor:
    """qgemm_w4a16 with the split-K partial sums in the library's static device
    scratch (no workspace; the C call allocates nothing).  Pass `out` to keep
    the wrapper from allocating the output.  Calls that overlap on one device
    share the scratch and must not run concurrently."""
    _dev(x, "x", torch.bfloat16, 2)
    m, k = x.shape
    y, yd = _out(m, n, out_dtype, x.device, out)
    st = lib.qgemm_w4a16_noalloc(x.data_ptr(), m, k, packed.data_ptr(), packed.numel(), n, y.data_ptr(),
                                 yd, split_k, _stream(x.device))
    _check(st, "qgemm_w4a16_noalloc")
    return y


def stream_read(src: torch.Tensor, nbytes: int, sink: torch.Tensor, blocks: int = 1024) -> None:
    """qg_stream_read: read the first `nbytes` bytes of `src` once (the plain
    streaming-read rate the GEMVs are compared with); `sink` receives
    blocks * 4 XOR words (int32, at least that many elements)."""
    if not src.is_cuda or not sink.is_cuda or sink.dtype != torch.int32 or sink.numel() < 4 * blocks:
        raise ValueError("src and sink must be device tensors, sink int32 with >= 4 * blocks elements")
    if nbytes > src.numel() * src.element_size():
        raise ValueError("nbytes exceeds src")
    _check(lib.qg_stream_read(src.data_ptr(), nbytes, sink.data_ptr(), blocks, _stream(src.device)),
           "qg_stream_read")


def qgemm_w4a16_dq(x: torch.Tensor, packed: torch.Tensor, n: int, *, split_k: int = 0,
                   out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y[m, n] = x . dequant(W)^T for a packed INT4 g32 weight with scale codes (m <= 64)."""
    _dev(x, "x", torch.bfloat16, 2)
    m, k = x.shape
    y, yd = _out(m, n, out_dtype, x.device, out)
    ws, ws_bytes = _workspace(m, n, k, split_k, x.device, workspace)
    st = lib.qgemm_w4a16_dq(x.data_ptr(), m, k, packed.data_ptr(), packed.numel(), n, y.data_ptr(),
                            yd, split_k, _ptr(ws), ws_bytes, _stream(x.device))
    _check(st, "qgemm_w4a16_dq")
    return y


def qgemm_wn_a16(x: torch.Tensor, packed: torch.Tensor, n: int, bits: int, *, split_k: int = 0,
                 out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y[m, n] = x . dequant(W)^T for a packed INT5 / INT6 g32 weight (m <= 64)."""
    _dev(x, "x", torch.bfloat16, 2)
    m, k = x.shape
    y, yd = _out(m, n, out_dtype, x.device, out)
    ws, ws_bytes = _workspace(m, n, k, split_k, x.device, workspace)
    st = lib.qgemm_wn_a16(x.data_ptr(), m, k, bits, packed.data_ptr(), packed.numel(), n, y.data_ptr(),
                          yd, split_k, _ptr(ws), ws_bytes, _stream(x.device))
    _check(st, "qgemm_wn_a16")
    return y


def qgemm_w8a16(x: torch.Tensor, w: torch.Tensor, scale: torch.Tensor, *,
                out_dtype: torch.dtype = torch.bfloat16,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """y[m, n] = (x . W^T) * scale[n] for an int8 [n, k] weight."""
    _dev(x, "x", torch.bfloat16, 2)
    _dev(w, "w", torch.int8, 2)
    _dev(scale, "scale", torch.bfloat16, 1)
    m, k = x.shape
    n = w.shape[0]
    if w.shape[1] != k or scale.shape[0] != n:
        raise ValueError("w must be [n, k] and scale [n]")
    y, yd = _out(m, n, out_dtype, x.device, out)
    st = lib.qgemm_w8a16(x.data_ptr(), m, k, w.data_ptr(), scale.data_ptr(), n, y.data_ptr(), yd,
                         _stream(x.device))
    _check(st, "qgemm_w8a16")
    return y


def qgemm_w4a8(x: torch.Tensor, packed: torch.Tensor, n: int, *, split_k: int = 0,
               out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None) -> torch.Tensor:
    """W4A8: per-row int8 activations (quantized inside the call) x packed INT4 g32."""
    _dev(x, "x", torch.bfloat16, 2)
    m, k = x.shape
    y, yd = _out(m, n, out_dtype, x.device, out)
    ws, ws_bytes = _workspace(m, n, k, split_k, x.device, workspace)
    st = lib.qgemm_w4a8(x.data_ptr(), m, k, packed.data_ptr(), packed.numel(), n, y.data_ptr(),
                        yd, split_k, _ptr(ws), ws_bytes, _stream(x.device))
    _check(st, "qgemm_w4a8")
    return y


def qgemm_w4a8_g32(x: torch.Tensor, packed: torch.Tensor, n: int, *, split_k: int = 0,
                   out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None) -> torch.Tensor:
    """W4A8 with one int8 activation scale per group of 32 (quantized inside the call)."""
    _dev(x, "x", torch.bfloat16, 2)
    m, k = x.shape
    y, yd = _out(m, n, out_dtype, x.device, out)
    ws, ws_bytes = _workspace(m, n, k, split_k, x.device, workspace)
    st = lib.qgemm_w4a8_g32(x.data_ptr(), m, k, packed.data_ptr(), packed.numel(), n, y.data_ptr(),
                            yd, split_k, _ptr(ws), ws_bytes, _stream(x.device))
    _check(st, "qgemm_w4a8_g32")
    return y


def _w4a8_call(fn, name, x, packed, n, split_k, out_dtype, out, workspace):
    _dev(x, "x", torch.bfloat16, 2)
    m, k = x.shape
    y, yd = _out(m, n, out_dtype, x.device, out)
    ws, ws_bytes = _workspace(m, n, k, split_k, x.device, workspace)
    st = fn(x.data_ptr(), m, k, packed.data_ptr(), packed.numel(), n, y.data_ptr(), yd, split_k, _ptr(ws),
            ws_bytes, _stream(x.device))
    _check(st, name)
    return y


def qgemm_w4a8_dq(x: torch.Tensor, packed: torch.Tensor, n: int, *, split_k: int = 0,
                  out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None) -> torch.Tensor:
    """qgemm_w4a8 (per-row int8 activations) on a scale-code packed weight (m <= 64)."""
    return _w4a8_call(lib.qgemm_w4a8_dq, "qgemm_w4a8_dq", x, packed, n, split_k, out_dtype, out, workspace)


def qgemm_w4a8_g32_dq(x: torch.Tensor, packed: torch.Tensor, n: int, *, split_k: int = 0,
                      out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None) -> torch.Tensor:
    """qgemm_w4a8_g32 (one activation scale per group of 32) on a scale-code packed weight (m <= 64)."""
    return _w4a8_call(lib.qgemm_w4a8_g32_dq, "qgemm_w4a8_g32_dq", x, packed, n, split_k, out_dtype, out,
                      workspace)


# ---- operators of a decoder layer around the linears -------------------------
#
# A decode step's kernels run a few microseconds, so the wrappers check their
# arguments in one expression; where it fails, the _refuse function of the
# operator finds out what is wrong and raises.

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _heads(t: torch.Tensor, name: str) -> tuple:
    """[rows, heads, d] bf16 with contiguous channels, any row and head stride."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA (HIP) device")
    if t.dtype != torch.bfloat16 or t.dim() != 3:
        raise ValueError(f"{name} must be bfloat16 [rows, heads, d], got {t.dtype} of rank {t.dim()}")
    if t.shape[2] != 1 and t.stride(2) != 1:
        raise ValueError(f"{name}: the channels of a head must be contiguous")
    return t.shape


def _same_device(device: torch.device, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} must be on {device}, got {t.device}")


def _flags_ok(status: torch.Tensor | None, dev: int) -> bool:
    return status is None or (status.get_device() == dev and status.element_size() == 4 and status.numel() >= 1)


def _refuse_flags(status: torch.Tensor | None) -> None:
    if status is not None and (not status.is_cuda or status.element_size() != 4 or status.numel() < 1):
        raise ValueError("status must be a 32-bit device word")


def _refuse_norm_rope(q, k, q_weight, k_weight, cos_sin, positions, out, status) -> None:
    tokens, _, d = _heads(q, "q")
    _heads(k, "k")
    if k.shape[0] != tokens or k.shape[2] != d:
        raise ValueError("q and k must have the same tokens and channels")
    _dev(cos_sin, "cos_sin", torch.float32, 2)
    _dev(positions, "positions", torch.int32, 1)
    if positions.shape[0] != tokens:
        raise ValueError("positions must be [tokens]")
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _dev(w, name, torch.bfloat16, 1)
            if w.shape[0] != d:
                raise ValueError(f"{name} must be [d]")
    if out is not None:
        for i, (t, like) in enumerate(zip(out, (q, k))):
            _dev(t, f"out[{i}]", torch.bfloat16, 3)
            if t.shape != like.shape:
                raise ValueError("out must have the shapes of q and k")
        _same_device(q.device, q_out=out[0], k_out=out[1])
    _refuse_flags(status)
    _same_device(q.device, k=k, q_weight=q_weight, k_weight=k_weight, cos_sin=cos_sin, positions=positions,
                 status=status)
    raise ValueError("qk_norm_rope: arguments that do not fit together")


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, q_weight: torch.Tensor | None, k_weight: torch.Tensor | None,
                 cos_sin: torch.Tensor, positions: torch.Tensor, *, eps: float = 1e-6,
                 adjacent_pairs: bool = False, out: tuple | None = None,
                 status: torch.Tensor | None = None) -> tuple:
    """RMS norm of every query and key head and the rotation of its first
    cos_sin.shape[1] channels by position: (q [tokens, hq, d], k [tokens, hkv, d])
    -> the same shapes, contiguous.  q and k may be strided views of a fused
    projection; cos_sin is fp32 [max_pos, rot], the cosines of a position
    before its sines."""
    dev, qs, ks, cs = q.get_device(), q.shape, k.shape, cos_sin.shape
    if not (dev >= 0 and len(qs) == 3 and len(ks) == 3 and q.dtype is _BF16 and k.dtype is _BF16 and
            k.get_device() == dev and ks[0] == qs[0] and ks[2] == qs[2] and q.stride(2) == 1 and k.stride(2) == 1 and
            len(cs) == 2 and cos_sin.dtype is _F32 and cos_sin.get_device() == dev and cos_sin.is_contiguous() and
            positions.dtype is _I32 and positions.get_device() == dev and positions.shape == qs[:1] and
            positions.is_contiguous() and
            (q_weight is None or (q_weight.dtype is _BF16 and q_weight.get_device() == dev and
                                  q_weight.shape == qs[2:] and q_weight.is_contiguous())) and
            (k_weight is None or (k_weight.dtype is _BF16 and k_weight.get_device() == dev and
                                  k_weight.shape == qs[2:] and k_weight.is_contiguous())) and
            (out is None or (out[0].dtype is _BF16 and out[1].dtype is _BF16 and out[0].shape == qs and
                             out[1].shape == ks and out[0].is_contiguous() and out[1].is_contiguous() and
                             out[0].get_device() == dev and out[1].get_device() == dev)) and
            _flags_ok(status, dev)):
        _refuse_norm_rope(q, k, q_weight, k_weight, cos_sin, positions, out, status)
    q_out, k_out = out if out is not None else (torch.empty_like(q, memory_format=torch.contiguous_format),
                                                torch.empty_like(k, memory_format=torch.contiguous_format))
    st = lib.qg_qk_norm_rope(q.data_ptr(), q.stride(0), q.stride(1), k.data_ptr(), k.stride(0), k.stride(1), qs[0],
                             qs[1], ks[1], qs[2], _ptr(q_weight), _ptr(k_weight), cos_sin.data_ptr(), cs[0], cs[1],
                             adjacent_pairs, positions.data_ptr(), eps, q_out.data_ptr(), k_out.data_ptr(),
                             _ptr(status), _stream_of(dev))
    if st:
        _check(st, "qg_qk_norm_rope")
    return q_out, k_out


def kv8_empty(pages: int, hkv: int, d: int, device) -> tuple:
    """(codes, scales) of an empty 8-bit key/value cache of `pages` pages of 64 tokens."""
    return (torch.zeros((pages, hkv, 2, KV8_PAGE * d), dtype=torch.int8, device=device),
            torch.zeros((pages, hkv, 2, KV8_PAGE // KV8_BLOCK), dtype=torch.float32, device=device))


def _refuse_cache(codes, scales, block_table, lens) -> None:
    _dev(codes, "codes", torch.int8, 4)
    _dev(scales, "scales", torch.float32, 4)
    _dev(block_table, "block_table", torch.int32, 2)
    _dev(lens, "lens", torch.int32, 1)
    pages, hkv, two, size = codes.shape
    if two != 2 or size % KV8_PAGE != 0:
        raise ValueError("codes must be int8 [pages, hkv, 2, 64 * d]")
    if scales.shape != (pages, hkv, 2, KV8_PAGE // KV8_BLOCK):
        raise ValueError("scales must be float32 [pages, hkv, 2, 4]")
    if lens.shape[0] != block_table.shape[0] or lens.shape[0] < 1:
        raise ValueError("block_table must be [b, width] and lens [b], b >= 1")
    _same_device(codes.device, scales=scales, block_table=block_table, lens=lens)
    raise ValueError("a cache whose parts do not fit together")


def _cache(codes, scales, block_table, lens) -> tuple:
    """Checks a cache and its table; (device index, pages, hkv, d, b, table width)."""
    dev, cs, ts = codes.get_device(), codes.shape, block_table.shape
    if not (dev >= 0 and len(cs) == 4 and len(ts) == 2 and codes.dtype is torch.int8 and scales.dtype is _F32 and
            block_table.dtype is _I32 and lens.dtype is _I32 and cs[2] == 2 and cs[3] % KV8_PAGE == 0 and
            scales.shape == (cs[0], cs[1], 2, 4) and lens.shape == ts[:1] and ts[0] >= 1 and
            scales.get_device() == dev and block_table.get_device() == dev and lens.get_device() == dev and
            codes.is_contiguous() and scales.is_contiguous() and block_table.is_contiguous() and lens.is_contiguous()):
        _refuse_cache(codes, scales, block_table, lens)
    return dev, cs[0], cs[1], cs[3] // KV8_PAGE, ts[0], ts[1]


def _starts(cu: torch.Tensor | None, b: int, rows: int, most: int | None, dev: int) -> int:
    """Checks the row offsets; the bound of a sequence's rows."""
    if cu is not None:
        if cu.dtype is not _I32 or cu.shape != (b + 1,) or cu.get_device() != dev or not cu.is_contiguous():
            _dev(cu, "cu", torch.int32, 1)
            raise ValueError("cu must be [b + 1], on the cache's device")
        return rows if most is None else most
    if rows % b != 0:
        raise ValueError("without cu every sequence has the same number of rows")
    return rows // b


def kv8_append(k: torch.Tensor, v: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
               block_table: torch.Tensor, lens: torch.Tensor, *, cu: torch.Tensor | None = None,
               max_new: int | None = None, status: torch.Tensor | None = None) -> None:
    """Quantizes new keys and values [rows, hkv, d] into the cache as the last
    tokens of the sequences (lens counts them).  Rows of sequence b are
    cu[b]..cu[b + 1] (cu given), or rows / b each; with cu, max_new bounds a
    sequence's rows, and those from max_new on are not written (default: all
    rows, which launches more workgroups than needed)."""
    dev, pages, hkv, d, b, width = _cache(codes, scales, block_table, lens)
    shape = k.shape
    if not (len(shape) == 3 and shape[1] == hkv and shape[2] == d and v.shape == shape and k.dtype is _BF16 and
            v.dtype is _BF16 and k.get_device() == dev and v.get_device() == dev and k.stride(2) == 1 and
            v.stride(2) == 1 and _flags_ok(status, dev)):
        rows = _heads(k, "k")[0]
        if tuple(k.shape) != (rows, hkv, d) or tuple(_heads(v, "v")) != (rows, hkv, d):
            raise ValueError("k and v must be [rows, hkv, d] of the cache's heads")
        _refuse_flags(status)
        _same_device(codes.device, k=k, v=v, status=status)
        raise ValueError("kv8_append: arguments that do not fit together")
    rows = shape[0]
    st = lib.qg_kv8_append(k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1), rows,
                           codes.data_ptr(), scales.data_ptr(), pages, hkv, d, block_table.data_ptr(), width,
                           lens.data_ptr(), _ptr(cu), b, _starts(cu, b, rows, max_new, dev), _ptr(status),
                           _stream_of(dev))
    if st:
        _check(st, "qg_kv8_append")


def _out_type(out_dtype: torch.dtype) -> int:
    if out_dtype is _BF16:
        return QG_BF16
    if out_dtype is not _F32:
        raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
    return QG_F32


def kv8_read(codes: torch.Tensor, scales: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor,
             max_len: int, *, out_dtype: torch.dtype = torch.bfloat16, out: tuple | None = None) -> tuple:
    """The sequences' keys and values as [b, max_len, hkv, d]; zero past a length."""
    dev, pages, hkv, d, b, width = _cache(codes, scales, block_table, lens)
    od, shape = _out_type(out_dtype), (b, max_len, hkv, d)
    if out is None:
        k = torch.empty(shape, dtype=out_dtype, device=codes.device)
        v = torch.empty_like(k)
    else:
        k, v = out
        for i, t in enumerate(out):
            _dev(t, f"out[{i}]", out_dtype, 4)
            if tuple(t.shape) != shape:
                raise ValueError("out must be two [b, max_len, hkv, d]")
        _same_device(codes.device, k=k, v=v)
    st = lib.qg_kv8_read(codes.data_ptr(), scales.data_ptr(), pages, hkv, d, block_table.data_ptr(), width,
                         lens.data_ptr(), b, max_len, k.data_ptr(), v.data_ptr(), od, _stream_of(dev))
    if st:
        _check(st, "qg_kv8_read")
    return k, v


def attn_kv8_workspace_bytes(b: int, rows: int, hq: int, hkv: int, d: int, max_q: int, max_len: int, *,
                             window: int = 0, splits: int = 0) -> int:
    v = int(lib.qg_attn_kv8_workspace_bytes(b, rows, hq, hkv, d, max_q, max_len, window, splits))
    _check(min(v, 0), "qg_attn_kv8_workspace_bytes")
    return v


def attn_kv8(q: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, block_table: torch.Tensor,
             lens: torch.Tensor, *, cu: torch.Tensor | None = None, max_q: int | None = None,
             max_len: int | None = None, window: int = 0, scale: float | None = None, splits: int = 0,
             out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
             workspace: torch.Tensor | None = None, status: torch.Tensor | None = None) -> torch.Tensor:
    """Causal attention of query rows [rows, hq, d] (a sequence's last tokens)
    over the cache -> [rows, hq, d].  scale defaults to d ** -0.5, max_len (an
    upper bound of lens, for the choice of the split) to the table's width.
    Rows that no sequence of cu has, and a sequence's rows from max_q on, are
    not written: give an `out` where that can happen."""
    dev, pages, hkv, d, b, width = _cache(codes, scales, block_table, lens)
    shape, od = q.shape, _out_type(out_dtype)
    if not (len(shape) == 3 and shape[2] == d and q.dtype is _BF16 and q.get_device() == dev and q.stride(2) == 1 and
            (out is None or (out.dtype is out_dtype and out.shape == shape and out.get_device() == dev and
                             out.is_contiguous())) and
            (workspace is None or (workspace.get_device() == dev and workspace.is_contiguous())) and
            _flags_ok(status, dev)):
        if _heads(q, "q")[2] != d:
            raise ValueError("q must have the cache's channels")
        if out is not None:
            _dev(out, "out", out_dtype, 3)
            if out.shape != shape:
                raise ValueError("out must have the shape of q")
        _refuse_flags(status)
        _same_device(codes.device, q=q, out=out, workspace=workspace, status=status)
        raise ValueError("attn_kv8: arguments that do not fit together")
    rows, hq = shape[0], shape[1]
    most = _starts(cu, b, rows, max_q, dev)
    if max_len is None:
        max_len = min(width * KV8_PAGE, 2**31 - 1)
    if out is None:
        out = torch.empty_like(q, dtype=out_dtype, memory_format=torch.contiguous_format)
    if rows == 0:
        return out
    ws_bytes = 0
    if workspace is None:
        ws_bytes = lib.qg_attn_kv8_workspace_bytes(b, rows, hq, hkv, d, most, max_len, window, splits)
        if ws_bytes > 0:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
        elif ws_bytes < 0:
            _check(ws_bytes, "qg_attn_kv8")
    else:
        ws_bytes = workspace.numel() * workspace.element_size()
    st = lib.qg_attn_kv8(q.data_ptr(), q.stride(0), q.stride(1), rows, hq, codes.data_ptr(), scales.data_ptr(), pages,
                         hkv, d, block_table.data_ptr(), width, lens.data_ptr(), _ptr(cu), b, most, max_len, window,
                         d ** -0.5 if scale is None else scale, out.data_ptr(), od, splits, _ptr(workspace), ws_bytes,
                         _ptr(status), _stream_of(dev))
    if st:
        _check(st, "qg_attn_kv8")
    return out


def moe_w4a16_workspace_bytes(t: int, h: int, e: int, inter: int, top_k: int) -> int:
    v = int(lib.qg_moe_w4a16_workspace_bytes(t, h, e, inter, top_k))
    _check(min(v, 0), "qg_moe_w4a16_workspace_bytes")
    return v


def _refuse_moe(x, router, gate_up, down, inter, out, out_dtype, workspace) -> None:
    _dev(x, "x", torch.bfloat16, 2)
    _dev(router, "router", torch.bfloat16, 2)
    _dev(gate_up, "gate_up", torch.uint8, 2)
    _dev(down, "down", torch.uint8, 2)
    e, h = router.shape[0], x.shape[1]
    if router.shape[1] != h or gate_up.shape[0] != e or down.shape[0] != e:
        raise ValueError("router must be [e, h], gate_up and down [e, bytes]")
    if gate_up.shape[1] != int4_packed_bytes(2 * inter, h) or down.shape[1] != int4_packed_bytes(h, inter):
        raise ValueError("gate_up must hold packed 2 inter x h weights and down packed h x inter ones")
    if out is not None:
        _dev(out, "out", out_dtype, 2)
        if out.shape != x.shape:
            raise ValueError("out must be [t, h]")
    _same_device(x.device, router=router, gate_up=gate_up, down=down, out=out, workspace=workspace)
    raise ValueError("moe_w4a16: arguments that do not fit together")


def moe_w4a16(x: torch.Tensor, router: torch.Tensor, gate_up: torch.Tensor, down: torch.Tensor, inter: int,
              top_k: int, *, renormalize: bool = True, out_dtype: torch.dtype = torch.bfloat16,
              out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """A mixture-of-experts layer for up to 64 tokens: x [t, h], router [e, h]
    (bf16), gate_up and down uint8 [e, bytes] of quantize_int4_g32 weights
    (2 inter x h, gate rows first; h x inter) -> y [t, h]."""
    dev, xs, rs, gs, ds = x.get_device(), x.shape, router.shape, gate_up.shape, down.shape
    od = _out_type(out_dtype)
    if not (dev >= 0 and len(xs) == 2 and len(rs) == 2 and len(gs) == 2 and len(ds) == 2 and x.dtype is _BF16 and
            router.dtype is _BF16 and gate_up.dtype is torch.uint8 and down.dtype is torch.uint8 and
            rs[1] == xs[1] and gs[0] == rs[0] and ds[0] == rs[0] and inter > 0 and
            gs[1] == 2 * inter // TILE_ROWS * (xs[1] // TILE_K) * TILE_BYTES and
            ds[1] == xs[1] // TILE_ROWS * (inter // TILE_K) * TILE_BYTES and
            router.get_device() == dev and gate_up.get_device() == dev and down.get_device() == dev and
            x.is_contiguous() and router.is_contiguous() and gate_up.is_contiguous() and down.is_contiguous() and
            (out is None or (out.dtype is out_dtype and out.shape == xs and out.get_device() == dev and
                             out.is_contiguous())) and
            (workspace is None or (workspace.get_device() == dev and workspace.is_contiguous()))):
        if dev >= 0:
            moe_w4a16_workspace_bytes(xs[0], xs[-1], rs[0], inter, top_k)   # sizes that no call takes
        _refuse_moe(x, router, gate_up, down, inter, out, out_dtype, workspace)
    t, h, e = xs[0], xs[1], rs[0]
    if workspace is None:
        ws_bytes = lib.qg_moe_w4a16_workspace_bytes(t, h, e, inter, top_k)
        if ws_bytes < 0:
            _check(ws_bytes, "qg_moe_w4a16")
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
    else:
        ws_bytes = workspace.numel() * workspace.element_size()
    if out is None:
        out = torch.empty_like(x, dtype=out_dtype)
    st = lib.qg_moe_w4a16(x.data_ptr(), t, h, router.data_ptr(), e, gate_up.data_ptr(), gate_up.numel(), down.data_ptr(),
                          down.numel(), inter, top_k, renormalize, out.data_ptr(), od, workspace.data_ptr(), ws_bytes,
                          _stream_of(dev))
    if st:
        _check(st, "qg_moe_w4a16")
    return out
