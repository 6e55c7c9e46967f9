"""The decoder-layer entry points on the host: every bad argument is refused
before anything is launched.  No call here reaches a kernel (each carries a
definite argument error, or has nothing to do), so these run without a GPU."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

import gemm_decode_qgemm_amd as qg
from gemm_decode_qgemm_amd.binding import lib

A, U = 0x10000, 0x10008          # a 16-byte aligned and an 8-byte aligned fake address, never dereferenced
OK, E_NULL, E_SHAPE, E_SPLIT, E_BUF, E_ALIGN, E_DTYPE, E_HEADS, E_STRIDE = 0, -1, -2, -5, -6, -7, -8, -12, -13


def norm_rope(**kw):
    a = dict(q=A, qts=5120, qhs=128, k=A, kts=5120, khs=128, tokens=3, hq=32, hkv=8, d=128, qw=A, kw=A, cs=A,
             max_pos=100, rot=128, pairs=0, pos=A, eps=1e-6, qo=A, ko=A, status=None, stream=None)
    assert set(kw) <= set(a)
    return lib.qg_qk_norm_rope(*(a | kw).values())


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), E_NULL), (dict(k=None), E_NULL), (dict(qo=None), E_NULL), (dict(ko=None), E_NULL), (dict(pos=None), E_NULL),
    (dict(cs=None), E_NULL), (dict(tokens=-1), E_SHAPE), (dict(tokens=1 << 31), E_SHAPE), (dict(tokens=(1 << 26) - 3), E_SHAPE), (dict(max_pos=0), E_SHAPE),
    (dict(eps=-1.0), E_SHAPE), (dict(eps=float("nan")), E_SHAPE), (dict(eps=float("inf")), E_SHAPE),
    (dict(hq=-1), E_HEADS), (dict(hq=0, hkv=0), E_HEADS), (dict(hq=5000), E_HEADS), (dict(d=120), E_HEADS), (dict(d=0), E_HEADS),
    (dict(d=528), E_HEADS), (dict(rot=24), E_HEADS), (dict(rot=144), E_HEADS), (dict(rot=-16), E_HEADS),
    (dict(qts=5121), E_STRIDE), (dict(qhs=4), E_STRIDE), (dict(qhs=120), E_STRIDE), (dict(kts=64), E_STRIDE), (dict(kts=-8), E_STRIDE),
    (dict(q=U), E_ALIGN), (dict(k=U), E_ALIGN), (dict(qw=U), E_ALIGN), (dict(kw=U), E_ALIGN), (dict(cs=U), E_ALIGN),
    (dict(pos=A + 2), E_ALIGN), (dict(qo=U), E_ALIGN), (dict(ko=U), E_ALIGN), (dict(status=A + 1), E_ALIGN), (dict(tokens=0), OK)])
def test_norm_rope_refusals(kw, want):
    assert norm_rope(**kw) == want


CACHE = dict(codes=A, scales=A, pages=10, hkv=2, d=128, table=A, width=4, lens=A)


def append(**kw):
    a = dict(k=A, kts=256, khs=128, v=A, vts=256, vhs=128, rows=4) | CACHE | dict(cu=None, b=2, max_new=2, status=None, stream=None)
    assert set(kw) <= set(a)
    return lib.qg_kv8_append(*(a | kw).values())


def read(**kw):
    a = CACHE | dict(b=2, max_len=9, k=A, v=A, dt=0, stream=None)
    assert set(kw) <= set(a)
    return lib.qg_kv8_read(*(a | kw).values())


def attn(**kw):
    a = dict(q=A, qts=1024, qhs=128, rows=4, hq=8) | CACHE | dict(cu=None, b=2, max_q=2, max_len=200, window=0, scale=0.1, out=A,
                                                                  dt=0, splits=1, ws=None, ws_bytes=0, status=None, stream=None)
    assert set(kw) <= set(a)
    return lib.qg_attn_kv8(*(a | kw).values())


@pytest.mark.parametrize("call", [append, read, attn])
@pytest.mark.parametrize("kw,want", [
    (dict(codes=None), E_NULL), (dict(scales=None), E_NULL), (dict(table=None), E_NULL), (dict(lens=None), E_NULL),
    (dict(pages=0), E_SHAPE), (dict(pages=1 << 31), E_SHAPE), (dict(width=0), E_SHAPE), (dict(b=0), E_SHAPE), (dict(b=1 << 16), E_SHAPE),
    (dict(b=65535, hkv=257), E_SHAPE), (dict(hkv=0), E_HEADS), (dict(d=96), E_HEADS), (dict(d=320), E_HEADS),
    (dict(codes=U), E_ALIGN), (dict(scales=U), E_ALIGN), (dict(table=A + 2), E_ALIGN), (dict(lens=A + 1), E_ALIGN)])
def test_cache_refusals(call, kw, want):
    assert call(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), E_NULL), (dict(v=None), E_NULL), (dict(rows=-1), E_SHAPE), (dict(rows=3), E_SHAPE), (dict(max_new=-1), E_SHAPE),
    (dict(max_new=1 << 40), E_SHAPE), (dict(kts=64), E_STRIDE), (dict(vhs=64), E_STRIDE), (dict(kts=260), E_STRIDE),
    (dict(k=U), E_ALIGN), (dict(v=U), E_ALIGN), (dict(cu=A + 2), E_ALIGN), (dict(status=A + 2), E_ALIGN),
    (dict(rows=0, k=None, v=None), OK), (dict(max_new=0), OK)])
def test_append_refusals(kw, want):
    assert append(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), E_NULL), (dict(v=None), E_NULL), (dict(max_len=-1), E_SHAPE), (dict(max_len=1 << 30), E_SHAPE),
    (dict(dt=2), E_DTYPE), (dict(k=U), E_ALIGN), (dict(v=U), E_ALIGN), (dict(max_len=0), OK)])
def test_read_refusals(kw, want):
    assert read(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), E_NULL), (dict(out=None), E_NULL), (dict(rows=5), E_SHAPE), (dict(max_q=0), E_SHAPE), (dict(max_q=70000), E_SHAPE),
    (dict(max_len=-1), E_SHAPE), (dict(window=-1), E_SHAPE), (dict(window=(1 << 30) + 1), E_SHAPE), (dict(scale=float("nan")), E_SHAPE), (dict(scale=float("inf")), E_SHAPE),
    (dict(hq=7), E_HEADS), (dict(hq=0), E_HEADS), (dict(dt=7), E_DTYPE), (dict(splits=-1), E_SPLIT), (dict(splits=257), E_SPLIT),
    (dict(splits=2), E_NULL), (dict(splits=2, ws=A, ws_bytes=2 * 4 * 8 * 130 * 4 - 1), E_BUF), (dict(ws=U), E_ALIGN),
    (dict(qts=64), E_STRIDE), (dict(qhs=12), E_STRIDE), (dict(q=U), E_ALIGN), (dict(out=U), E_ALIGN), (dict(status=A + 2), E_ALIGN),
    (dict(rows=0), OK)])
def test_attn_refusals(kw, want):
    assert attn(**kw) == want


def test_attn_workspace():
    assert qg.attn_kv8_workspace_bytes(2, 4, 8, 2, 128, 2, 200, splits=1) == 0
    assert qg.attn_kv8_workspace_bytes(2, 4, 8, 2, 128, 2, 200, splits=3) == 3 * 4 * 8 * 130 * 4
    assert qg.attn_kv8_workspace_bytes(1, 1, 32, 1, 128, 1, 64) == 0                  # one page: nothing to split
    assert qg.attn_kv8_workspace_bytes(1, 1, 32, 1, 128, 1, 131072) > 0
    assert qg.attn_kv8_workspace_bytes(1, 1, 32, 1, 128, 1, 131072, window=64) == 0
    with pytest.raises(qg.QGemmError):
        qg.attn_kv8_workspace_bytes(2, 4, 8, 3, 128, 2, 200)
    for status in (E_HEADS, E_STRIDE):
        assert "unknown" not in qg.status_string(status)


def moe(**kw):
    a = dict(x=A, t=3, h=512, router=A, e=8, gu=A, gu_bytes=8 * 2 * 256 // 64 * 2 * 9472, dn=A, dn_bytes=8 * 8 * 9472, inter=256, k=2,
             renorm=1, y=A, dt=0, ws=A, ws_bytes=1 << 30, stream=None)
    assert set(kw) <= set(a)
    return lib.qg_moe_w4a16(*(a | kw).values())


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), E_NULL), (dict(router=None), E_NULL), (dict(gu=None), E_NULL), (dict(dn=None), E_NULL), (dict(y=None), E_NULL),
    (dict(ws=None), E_NULL), (dict(t=-1), E_SHAPE), (dict(t=65), -4), (dict(h=0), E_SHAPE), (dict(h=500), -3), (dict(inter=128), -3),
    (dict(inter=0), E_SHAPE), (dict(e=0), E_SHAPE), (dict(e=513), E_SHAPE), (dict(k=0), E_SHAPE), (dict(k=9), E_SHAPE),
    (dict(e=64, k=33), E_SHAPE), (dict(dt=3), E_DTYPE), (dict(gu_bytes=8 * 8 * 2 * 9472 - 1), E_BUF), (dict(dn_bytes=8 * 8 * 9472 - 1), E_BUF),
    (dict(ws_bytes=100), E_BUF), (dict(x=U), E_ALIGN), (dict(router=U), E_ALIGN), (dict(gu=U), E_ALIGN), (dict(dn=U), E_ALIGN),
    (dict(y=U), E_ALIGN), (dict(ws=U), E_ALIGN), (dict(t=0), OK)])
def test_moe_refusals(kw, want):
    assert moe(**kw) == want
    with pytest.raises(qg.QGemmError):
        qg.moe_w4a16_workspace_bytes(65, 512, 8, 256, 2)


def test_wrappers_refuse_host_tensors_and_wrong_types():
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        qg.qk_norm_rope(x, x, None, None, torch.zeros(4, 64), torch.zeros(2, dtype=torch.int32))
    codes, scales = qg.kv8_empty(3, 4, 64, "cpu")
    assert codes.shape == (3, 4, 2, 4096) and scales.shape == (3, 4, 2, 4)
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        qg.kv8_append(x, x, codes, scales, table, lens)
    with pytest.raises(ValueError, match="device"):
        qg.kv8_read(codes, scales, table, lens, 4)
    with pytest.raises(ValueError, match="device"):
        qg.attn_kv8(x, codes, scales, table, lens)


def test_attn_workspace_of_shared_out_splits():
    # 16 sequences on 8 heads, tables of 8192 tokens: 96 partial results a row and 8 bytes a sequence
    assert qg.attn_kv8_workspace_bytes(16, 16, 32, 8, 128, 1, 8192) == 96 * 32 * 130 * 4 + 16 * 8
    assert qg.attn_kv8_workspace_bytes(16, 16, 32, 8, 128, 1, 8192, splits=2) == 2 * 16 * 32 * 130 * 4
    # few pages a split, or rows so ragged that their bound says little: equal splits
    for args, one in (((16, 16, 32, 8, 128, 1, 2048), 16 * 32 * 130 * 4), ((16, 17, 32, 8, 128, 4, 8192), 17 * 32 * 130 * 4)):
        need = qg.attn_kv8_workspace_bytes(*args)
        assert need > one and need % one == 0
    for n in (0, 1, 63, 64, 65, 257):
        assert qg.attn_kv8_workspace_bytes(3, 3, 8, 2, 64, 1, n) >= 0
        assert qg.attn_kv8_workspace_bytes(3, 3, 8, 2, 256, 1, n) >= 0


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_layer.py")
    spec = importlib.util.spec_from_file_location("decoder_layer_example", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("batch", [0, 65, 1000])
def test_the_example_refuses_batches_that_no_step_takes(batch):
    """Before any weight is made, not in the middle of a prompt."""
    with pytest.raises(ValueError, match="1 to 64"):
        example().DecoderLayer(batch, 100, device="cpu")


def test_the_example_takes_short_prompts():
    lengths = example().prompt_lengths
    assert lengths(100, 7) == [100, 97, 94, 91, 88, 100, 97]
    assert lengths(1, 6) == [1] * 6 and lengths(7, 5) == [7, 4, 1, 1, 1]
    with pytest.raises(ValueError):
        lengths(0, 3)
