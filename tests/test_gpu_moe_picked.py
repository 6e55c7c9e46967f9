"""qg.moe_w4a16_picked against the experts in 64 bits on the oracle's quantization.

Tolerance per output as for the whole layer: with B = the sum over picks of |w| |W2|
|silu(g) u| in 64 bits, the hidden activation is rounded to bf16 (2^-8 of each term
at most), the fp32 sums add less than 2^-10 of the terms at these sizes, and cancelled
gate or up sums 2^-16 of the largest B of the row; half a bf16 step for bf16 output."""
from __future__ import annotations

import functools

import numpy as np
import pytest
import torch

import oracle
import synthetic_inputs as si
import serving_reference as ref

import gemm_decode_qgemm_amd as qg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


@functools.lru_cache(maxsize=4)
def experts(e, h, inter):
    """(packed gate_up, packed down, their values in 64 bits)."""
    g = torch.Generator().manual_seed(e + h + inter)
    out = []
    for n, k in ((2 * inter, h), (h, inter)):
        packed, values = [], []
        for _ in range(e):
            w = (torch.randn(n, k, generator=g) * k ** -0.5).bfloat16()
            codes, scales, zeros, _ = oracle.quantize_int4_g32(si.bf16_bits(w))
            packed.append(torch.from_numpy(oracle.pack_int4(codes, scales, zeros)))
            q = codes.reshape(n, k // 32, 32).astype(np.float64) - zeros.reshape(n, k // 32, 1)
            values.append((q * scales.reshape(n, k // 32, 1).view(np.float16).astype(np.float64)).reshape(n, k))
        out.append((torch.stack(packed), values))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def plain(x, ids, weights, gate_up, down, inter):
    y, bound = np.zeros_like(x), np.zeros_like(x)
    for t in range(x.shape[0]):
        seen = set()
        for e, w in zip(ids[t].tolist(), weights[t]):
            if not 0 <= e < len(down) or e in seen:
                continue
            seen.add(e)
            gu = gate_up[e] @ x[t]
            g, u = gu[:inter], gu[inter:]
            a = g / (1 + np.exp(-g)) * u
            y[t] += w * (down[e] @ a)
            bound[t] += abs(w) * (np.abs(down[e]) @ np.abs(a))
    return y, bound


def check(y, want, bound):
    got = ref.f64(y)
    tol = bound * (2.0 ** -8 + 2.0 ** -10) + bound.max(-1, keepdims=True) * 2.0 ** -16
    if y.dtype == torch.bfloat16:
        tol = tol + ref.half_step(np.abs(want) + tol, 8)
    assert np.all(np.abs(got - want) <= tol), np.argwhere(~(np.abs(got - want) <= tol))[:3]


def inputs(t, e, k, h, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(t, h, generator=g).bfloat16()
    ids = torch.stack([torch.randperm(e, generator=g)[:k] for _ in range(t)]).to(torch.int32)
    return x, ids, torch.randn(t, k, generator=g)          # weights of either sign, summing to anything


def run(dev, x, ids, w, e, inter, **kw):
    gu, dn, gu_v, dn_v = experts(e, x.shape[1], inter)
    y = qg.moe_w4a16_picked(x.to(dev), ids.to(dev), w.to(dev), gu.to(dev), dn.to(dev), inter, **kw)
    return y, plain(ref.f64(x), ids.numpy(), ref.f64(w), gu_v, dn_v, inter)


@pytest.mark.parametrize("t", [1, 2, 3, 4, 5, 8, 9, 17, 33, 64])
@pytest.mark.parametrize("e,k,h,inter", [(8, 2, 512, 256), (16, 4, 256, 768), (70, 6, 256, 256)])
def test_every_token_count(dev, t, e, k, h, inter):
    x, ids, w = inputs(t, e, k, h, t + e)
    for dt in (torch.float32, torch.bfloat16):
        y, (want, bound) = run(dev, x, ids, w, e, inter, out_dtype=dt)
        assert y.dtype == dt and y.shape == (t, h)
        check(y, want, bound)


@pytest.mark.parametrize("t", [1, 2, 4, 5, 8, 20, 64])
@pytest.mark.parametrize("e,k", [(8, 3), (40, 8)])
def test_picks_that_count_for_nothing(dev, t, e, k):
    """None, past the experts, a second time; tokens without any pick among them."""
    x, ids, w = inputs(t, e, k, 256, 3 * t + e)
    for m in range(t):
        if m % 4 == 0:
            ids[m, 0] = -1
        if m % 4 == 1:
            ids[m, 1], ids[m, 2] = ids[m, 0], e
        if m % 4 == 2:
            ids[m] = -7
        if m % 4 == 3:
            ids[m, 1:] = ids[m, 0]
    ids[0, 1] = 2 ** 31 - 1
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    ws = torch.full((qg.moe_w4a16_workspace_bytes(t, 256, e, 256, k),), 0xff, dtype=torch.uint8, device=dev)   # NaN patterns
    y, (want, bound) = run(dev, x, ids, w, e, 256, out_dtype=torch.float32, status=status, workspace=ws)
    check(y, want, bound)
    assert status.item() == qg.FLAG_INDEX
    if t > 2:
        assert not bool(y[2].any())
    status.zero_()
    x, ids, w = inputs(t, e, k, 256, 3)
    ids[t - 1] = -1
    run(dev, x, ids, w, e, 256, status=status)
    assert status.item() == 0


def test_all_tokens_on_the_same_experts(dev):
    x, ids, w = inputs(64, 16, 4, 256, 9)
    ids[:] = torch.tensor([3, 15, 0, 7], dtype=torch.int32)
    y, (want, bound) = run(dev, x, ids, w, 16, 256, out_dtype=torch.float32)
    check(y, want, bound)


def test_the_whole_layer_is_the_route_and_the_experts(dev):
    """moe_route on the logits of moe_w4a16's router, then the picked experts."""
    for t in (1, 3, 7, 30):
        gu, dn, _, _ = experts(16, 256, 768)
        g = torch.Generator().manual_seed(t)
        x, router = torch.randn(t, 256, generator=g).bfloat16().to(dev), (torch.randn(16, 256, generator=g) / 8).bfloat16().to(dev)
        for renorm in (True, False):
            want = qg.moe_w4a16(x, router, gu.to(dev), dn.to(dev), 768, 4, renormalize=renorm, out_dtype=torch.float32)
            ids, w = qg.moe_route(x.float() @ router.float().t(), 4, renormalize=renorm)
            got = qg.moe_w4a16_picked(x, ids, w, gu.to(dev), dn.to(dev), 768, out_dtype=torch.float32)
            # the same products; the weights' last bits differ
            assert float((got - want).norm()) <= 1e-5 * float(want.norm())


def test_captured_and_replayed(dev):
    for t in (1, 4, 12):
        gu, dn, _, _ = experts(8, 512, 256)
        gu, dn = gu.to(dev), dn.to(dev)
        x, ids, w = (v.to(dev) for v in inputs(t, 8, 2, 512, t))
        ws = torch.empty(qg.moe_w4a16_workspace_bytes(t, 512, 8, 256, 2), dtype=torch.uint8, device=dev)
        out = torch.empty_like(x)
        qg.moe_w4a16_picked(x, ids, w, gu, dn, 256, out=out, workspace=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            qg.moe_w4a16_picked(x, ids, w, gu, dn, 256, out=out, workspace=ws)
        for k in range(3):
            nx, nids, nw = inputs(t, 8, 2, 512, 100 + k)
            x.copy_(nx), ids.copy_(nids), w.copy_(nw)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, qg.moe_w4a16_picked(x, ids, w, gu, dn, 256)), (t, k)
    assert qg.moe_w4a16_picked(x[:0], ids[:0], w[:0], gu, dn, 256).shape == (0, 512)
