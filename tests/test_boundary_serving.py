"""The serving-step entry points on the host: every bad argument is refused before
anything is launched.  No call here reaches a kernel, so these run without a GPU."""
from __future__ import annotations

import pytest
import torch

import gemm_decode_qgemm_amd as qg
from gemm_decode_qgemm_amd.binding import lib

A, U = 0x10000, 0x10008          # a 16-byte aligned and an 8-byte aligned fake address, never dereferenced
OK, E_NULL, E_SHAPE, E_M, E_BUF, E_ALIGN, E_DTYPE, E_STRIDE = 0, -1, -2, -4, -6, -7, -8, -13
NAN, INF = float("nan"), float("inf")


def norm(**kw):
    a = dict(x=A, xt=0, xs=512, res=A, rt=1, rs=512, rows=3, h=512, w=A, eps=1e-6, y=A, yt=0, ro=A, stream=None)
    assert set(kw) <= set(a)
    return lib.qg_rms_norm(*(a | kw).values())


def norm_q8(**kw):
    a = dict(x=A, xt=0, xs=512, res=A, rt=1, rs=512, rows=3, h=512, w=A, eps=1e-6, codes=A, scales=A, group=1, ro=A, stream=None)
    assert set(kw) <= set(a)
    return lib.qg_rms_norm_q8(*(a | kw).values())


@pytest.mark.parametrize("call", [norm, norm_q8])
@pytest.mark.parametrize("kw,want", [
    (dict(x=None), E_NULL), (dict(ro=None), E_NULL), (dict(res=None), E_NULL), (dict(rows=-1), E_SHAPE), (dict(rows=1 << 22), E_SHAPE),
    (dict(h=0), E_SHAPE), (dict(h=-8), E_SHAPE), (dict(h=516), E_SHAPE), (dict(h=32776, xs=40000, rs=40000), E_SHAPE), (dict(eps=-1.0), E_SHAPE),
    (dict(eps=NAN), E_SHAPE), (dict(eps=INF), E_SHAPE), (dict(xt=2), E_DTYPE), (dict(rt=-1), E_DTYPE), (dict(xs=504), E_STRIDE), (dict(xs=516), E_STRIDE),
    (dict(rs=8), E_STRIDE), (dict(rs=-512), E_STRIDE), (dict(xs=1 << 41), E_STRIDE), (dict(x=U), E_ALIGN), (dict(res=U), E_ALIGN), (dict(w=U), E_ALIGN),
    (dict(ro=U), E_ALIGN), (dict(rows=0), OK), (dict(rows=0, x=None, res=None, ro=None), OK)])
def test_norm_refusals(call, kw, want):
    assert call(**kw) == want


@pytest.mark.parametrize("kw,want", [(dict(y=None), E_NULL), (dict(y=U), E_ALIGN), (dict(yt=5), E_DTYPE)])
def test_norm_output_refusals(kw, want):
    assert norm(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(codes=None), E_NULL), (dict(scales=None), E_NULL), (dict(codes=A + 4), E_ALIGN), (dict(scales=A + 2), E_ALIGN),
    (dict(h=520, xs=520, rs=520), E_SHAPE)])
def test_norm_q8_output_refusals(kw, want):
    assert norm_q8(**kw) == want


def lora(**kw):
    a = dict(x=A, m=3, k=512, a=A, b=A, r=16, adapters=5, ids=A, scales=None, y=A, yt=0, ys=300, n=300, out=A, ot=0, os=300, ws=A, ws_bytes=1 << 30,
             status=None, stream=None)
    assert set(kw) <= set(a)
    return lib.qg_lora_add(*(a | kw).values())


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), E_NULL), (dict(a=None), E_NULL), (dict(b=None), E_NULL), (dict(ids=None), E_NULL), (dict(y=None), E_NULL), (dict(out=None), E_NULL),
    (dict(ws=None), E_NULL), (dict(m=-1), E_SHAPE), (dict(m=65), E_M), (dict(k=0), E_SHAPE), (dict(k=516), E_SHAPE), (dict(k=(1 << 20) + 8), E_SHAPE),
    (dict(n=0), E_SHAPE), (dict(n=(1 << 20) + 1), E_SHAPE), (dict(r=0), E_SHAPE), (dict(r=12), E_SHAPE), (dict(r=264), E_SHAPE), (dict(adapters=0), E_SHAPE),
    (dict(adapters=1 << 31), E_SHAPE), (dict(yt=2), E_DTYPE), (dict(ot=2), E_DTYPE), (dict(ys=299), E_STRIDE), (dict(os=0), E_STRIDE),
    (dict(ys=1 << 41), E_STRIDE), (dict(ws_bytes=3 * 16 * 4 - 1), E_BUF), (dict(x=U), E_ALIGN), (dict(a=U), E_ALIGN), (dict(b=U), E_ALIGN),
    (dict(ids=A + 2), E_ALIGN), (dict(scales=A + 2), E_ALIGN), (dict(y=A + 1), E_ALIGN), (dict(yt=1, y=A + 2), E_ALIGN), (dict(out=A + 1), E_ALIGN),
    (dict(ws=U), E_ALIGN), (dict(status=A + 1), E_ALIGN), (dict(m=0), OK), (dict(m=0, x=None, ids=None, y=None, out=None, ws=None), OK)])
def test_lora_refusals(kw, want):
    assert lora(**kw) == want


def test_lora_workspace():
    assert qg.lora_add_workspace_bytes(0, 512, 300, 16, 5) == 0
    n = qg.lora_add_workspace_bytes(3, 512, 300, 16, 5)
    assert n > 0 and n % (3 * 16 * 4) == 0
    for args in ((65, 512, 300, 16, 5), (3, 512, 300, 12, 5), (3, 511, 300, 16, 5)):
        with pytest.raises(qg.QGemmError):
            qg.lora_add_workspace_bytes(*args)


def route(**kw):
    a = dict(l=A, lt=1, t=3, e=256, k=8, sigmoid=1, bias=None, groups=8, top=4, best=2, renorm=1, scale=2.5, ids=A, w=A, stream=None)
    assert set(kw) <= set(a)
    return lib.qg_moe_route(*(a | kw).values())


@pytest.mark.parametrize("kw,want", [
    (dict(l=None), E_NULL), (dict(ids=None), E_NULL), (dict(w=None), E_NULL), (dict(t=-1), E_SHAPE), (dict(t=1 << 26), E_SHAPE), (dict(e=0), E_SHAPE),
    (dict(e=520), E_SHAPE), (dict(k=0), E_SHAPE), (dict(k=33), E_SHAPE), (dict(groups=0), E_SHAPE), (dict(groups=7), E_SHAPE), (dict(groups=128), E_SHAPE),
    (dict(top=0), E_SHAPE), (dict(top=9), E_SHAPE), (dict(best=0), E_SHAPE), (dict(best=3), E_SHAPE), (dict(e=8, groups=8, k=4), E_SHAPE),
    (dict(e=16, k=9), E_SHAPE), (dict(scale=NAN), E_SHAPE), (dict(scale=INF), E_SHAPE), (dict(lt=3), E_DTYPE), (dict(l=A + 2), E_ALIGN),
    (dict(bias=A + 2), E_ALIGN), (dict(ids=A + 2), E_ALIGN), (dict(w=A + 1), E_ALIGN), (dict(t=0), OK)])
def test_route_refusals(kw, want):
    assert route(**kw) == want


def verify(**kw):
    a = dict(p=A, q=A, dt=1, rows=9, v=131071, tokens=A, u=A, u_next=A, cu=A, b=3, lens=None, acc=A, nxt=A, ws=A, ws_bytes=1 << 20, status=None, stream=None)
    assert set(kw) <= set(a)
    return lib.qg_verify_drafts(*(a | kw).values())


@pytest.mark.parametrize("kw,want", [
    (dict(p=None), E_NULL), (dict(tokens=None), E_NULL), (dict(u=None), E_NULL), (dict(u_next=None), E_NULL), (dict(cu=None), E_NULL),
    (dict(acc=None), E_NULL), (dict(nxt=None), E_NULL), (dict(ws=None), E_NULL), (dict(b=-1), E_SHAPE), (dict(b=65536, rows=70000), E_SHAPE),
    (dict(rows=2), E_SHAPE), (dict(rows=1 << 31), E_SHAPE), (dict(v=0), E_SHAPE), (dict(v=1 << 31), E_SHAPE), (dict(dt=2), E_DTYPE), (dict(ws_bytes=3 * 256 * 8 - 1), E_BUF),
    (dict(p=A + 2), E_ALIGN), (dict(dt=0, q=A + 1), E_ALIGN), (dict(tokens=A + 2), E_ALIGN), (dict(u=A + 1), E_ALIGN), (dict(u_next=A + 2), E_ALIGN),
    (dict(cu=A + 2), E_ALIGN), (dict(lens=A + 2), E_ALIGN), (dict(acc=A + 2), E_ALIGN), (dict(nxt=A + 1), E_ALIGN), (dict(ws=U), E_ALIGN),
    (dict(status=A + 2), E_ALIGN), (dict(b=0), OK), (dict(b=0, rows=0, p=None, ws=None, cu=None), OK)])
def test_verify_refusals(kw, want):
    assert verify(**kw) == want


def test_verify_workspace():
    assert qg.verify_drafts_workspace_bytes(9, 3, 1000) == 0              # a workgroup a sequence keeps its sums
    assert qg.verify_drafts_workspace_bytes(9, 3, 131071) == 3 * 256 * 8
    assert qg.verify_drafts_workspace_bytes(0, 0, 1000) == 0
    assert 512 * 8 < qg.verify_drafts_workspace_bytes(1, 1, 2 ** 31 - 1) <= 1024 * 8
    assert verify(v=1000, ws=None, ws_bytes=0, p=None) == E_NULL
    with pytest.raises(qg.QGemmError):
        qg.verify_drafts_workspace_bytes(2, 3, 1000)


def rows(**kw):
    a = dict(xq=A, scales=A, group=0, m=3, k=512, packed=A, bytes=2 * 2 * 9472, codes=0, n=128, y=A, dt=0, split=0, ws=A, ws_bytes=1 << 20, stream=None)
    assert set(kw) <= set(a)
    return lib.qgemm_w4a8_rows(*(a | kw).values())


@pytest.mark.parametrize("kw,want", [
    (dict(xq=None), E_NULL), (dict(scales=None), E_NULL), (dict(packed=None), E_NULL), (dict(y=None), E_NULL), (dict(m=0), E_SHAPE), (dict(m=65), E_M),
    (dict(n=0), E_SHAPE), (dict(k=500), -3), (dict(split=3), -5), (dict(split=4), -5), (dict(dt=2), E_DTYPE), (dict(bytes=2 * 2 * 9472 - 1), E_BUF),
    (dict(codes=1, bytes=2 * (128 + 2 * 8960) - 1), E_BUF), (dict(split=2, ws=None), E_NULL), (dict(split=2, ws_bytes=2 * 3 * 128 * 4 - 1), E_BUF),
    (dict(m=9, split=1, ws=None), E_NULL), (dict(m=9, split=1, ws_bytes=9 * 512 * 2), E_BUF), (dict(xq=U), E_ALIGN), (dict(packed=U), E_ALIGN),
    (dict(y=U), E_ALIGN), (dict(ws=U), E_ALIGN), (dict(scales=A + 2), E_ALIGN)])
def test_w4a8_rows_refusals(kw, want):
    assert rows(**kw) == want


def picked(**kw):
    a = dict(x=A, t=3, h=512, ids=A, weights=A, e=8, gu=A, gu_bytes=8 * 2 * 256 // 64 * 2 * 9472, dn=A, dn_bytes=8 * 8 * 9472, inter=256, k=2,
             y=A, dt=0, ws=A, ws_bytes=1 << 30, status=None, stream=None)
    assert set(kw) <= set(a)
    return lib.qg_moe_w4a16_picked(*(a | kw).values())


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), E_NULL), (dict(ids=None), E_NULL), (dict(weights=None), E_NULL), (dict(gu=None), E_NULL), (dict(dn=None), E_NULL), (dict(y=None), E_NULL),
    (dict(ws=None), E_NULL), (dict(t=-1), E_SHAPE), (dict(t=65), E_M), (dict(h=500), -3), (dict(inter=128), -3), (dict(e=513), E_SHAPE), (dict(k=9), E_SHAPE),
    (dict(dt=3), E_DTYPE), (dict(gu_bytes=8 * 8 * 2 * 9472 - 1), E_BUF), (dict(dn_bytes=8 * 8 * 9472 - 1), E_BUF), (dict(ws_bytes=100), E_BUF),
    (dict(x=U), E_ALIGN), (dict(ids=A + 2), E_ALIGN), (dict(weights=A + 1), E_ALIGN), (dict(gu=U), E_ALIGN), (dict(dn=U), E_ALIGN), (dict(y=U), E_ALIGN),
    (dict(ws=U), E_ALIGN), (dict(status=A + 2), E_ALIGN), (dict(t=0), OK)])
def test_moe_picked_refusals(kw, want):
    assert picked(**kw) == want


def test_wrappers_refuse_host_tensors_and_wrong_types():
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        qg.rms_norm(x, w)
    with pytest.raises(ValueError, match="device"):
        qg.rms_norm_q8(x, w, residual=x)
    ids = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        qg.lora_add(x, x, x[None], x[None], ids)
    with pytest.raises(ValueError, match="device"):
        qg.moe_route(x, 4)
    with pytest.raises(ValueError, match="device"):
        qg.qgemm_w4a8_rows(torch.zeros(2, 256, dtype=torch.int8), torch.zeros(2), torch.zeros(9472, dtype=torch.uint8), 64)
    f = torch.zeros(2)
    with pytest.raises(ValueError, match="device"):
        qg.verify_drafts(x, None, ids, f, f, ids)


@pytest.mark.parametrize("kw", [dict(), dict(e=6, groups=1, top=1, best=1, k=2), dict(k=32), dict(e=512)])
def test_route_refuses_more_tokens_than_its_grids_hold(kw):
    """2^23 workgroups of 512 threads and eight tokens each would be 2^32 threads."""
    for t in ((1 << 26) - 7, (1 << 26) - 4, 1 << 40):
        assert route(t=t, **kw) == E_SHAPE


class OnDevice:
    """What a wrapper's checks see of a device tensor."""

    def __init__(self, shape, dtype, contiguous=True):
        self.shape, self.dtype, self._contiguous, self.is_cuda = torch.Size(shape), dtype, contiguous, True
        self.device = torch.device("cuda:0")

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return self._contiguous


def test_linears_refuse_an_out_or_workspace_that_they_would_write_past():
    from gemm_decode_qgemm_amd import binding
    bf16, u8 = torch.bfloat16, torch.uint8
    for shape in ((4, 99), (3, 100), (0, 100), (1, 1)):
        with pytest.raises(ValueError, match="out"):
            binding._out(4, 100, bf16, None, OnDevice(shape, bf16))
    for shape in ((4, 100), (64, 100)):
        assert binding._out(4, 100, bf16, None, OnDevice(shape, bf16))[0].shape == shape
    need = binding.workspace_bytes(1, 128, 512, 2)
    assert need > 0
    with pytest.raises(ValueError, match="workspace"):
        binding._workspace(1, 128, 512, 2, None, OnDevice((need,), u8, contiguous=False))
    assert binding._workspace(1, 128, 512, 2, None, OnDevice((need,), u8))[1] == need


def test_quantized_rows_refuse_a_weight_or_out_of_another_kind():
    bf16, u8, f32 = torch.bfloat16, torch.uint8, torch.float32
    codes, scales, packed = OnDevice((4, 256), torch.int8), OnDevice((4,), f32), OnDevice((9472 * 2,), u8)
    for kw, name in ((dict(packed=OnDevice((9472 * 2,), torch.int32)), "packed"), (dict(packed=OnDevice((9472 * 2,), u8, False)), "packed"),
                     (dict(out=OnDevice((4, 127), bf16)), "out"), (dict(out=OnDevice((3, 128), bf16)), "out"),
                     (dict(out=OnDevice((4, 256), bf16)), "out"), (dict(out=OnDevice((128, 4), bf16)), "out"), (dict(out=OnDevice((4, 128), f32)), "out")):
        a = dict(codes=codes, scales=scales, packed=packed, n=128, out=None) | kw
        with pytest.raises(ValueError, match=name):
            qg.qgemm_w4a8_rows(**a)
