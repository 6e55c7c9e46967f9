"""qg_qk_norm_rope against the 64-bit form.

Tolerance: the result is computed in binary32 (a few 2^-23 of the pair's
magnitude, which the rotation may cancel) and rounded once to bf16: half a
unit in the last place of the reference, plus 2^-19 of the head's largest
channel."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import layer_reference as ref

import gemm_decode_qgemm_amd as qg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


def table(most, rot):
    a = torch.arange(most, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    return torch.cat([a.cos(), a.sin()], 1).float()


def check(y, x, w, cs, pos, eps, pairs):
    r = ref.norm_rope(ref.f64(x), None if w is None else ref.f64(w), ref.f64(cs), pos.cpu().numpy(), eps, pairs)
    err = np.abs(ref.f64(y) - r)
    tol = ref.half_ulp_bf16(r) + np.abs(r).max(-1, keepdims=True) * 2.0 ** -19 + 1e-30
    assert np.isfinite(ref.f64(y)).all()
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("tokens", [1, 3, 70])
@pytest.mark.parametrize("hq,hkv,d,rot,pairs", [
    (32, 8, 128, 128, False), (32, 8, 128, 64, True), (5, 1, 64, 64, False), (3, 3, 80, 80, False), (3, 1, 96, 32, True),
    (7, 2, 192, 192, False), (16, 2, 256, 64, True), (2, 1, 512, 512, False), (4, 4, 16, 16, False), (4, 2, 32, 0, False),
    (1, 1, 48, 16, False)])
def test_against_64_bits(dev, tokens, hq, hkv, d, rot, pairs):
    torch.manual_seed(tokens * 1000 + d + rot)
    qkv = torch.randn(tokens, (hq + 2 * hkv) * d).bfloat16()
    w = (1 + torch.randn(2, d) * 0.3).bfloat16()
    cs, pos = table(97, rot), torch.randint(0, 97, (tokens,), dtype=torch.int32)
    q = qkv[:, :hq * d].unflatten(1, (hq, d))
    k = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    qkv_d = qkv.to(dev)
    qd = qkv_d[:, :hq * d].unflatten(1, (hq, d))
    kd = qkv_d[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    yq, yk = qg.qk_norm_rope(qd, kd, w[0].to(dev), w[1].to(dev), cs.to(dev), pos.to(dev), adjacent_pairs=pairs)
    assert yq.shape == (tokens, hq, d) and yk.shape == (tokens, hkv, d)
    check(yq, q, w[0], cs, pos, 1e-6, pairs)
    check(yk, k, w[1], cs, pos, 1e-6, pairs)


def test_many_tokens_take_whole_tokens_per_wave(dev):
    """Above 16 waves per CU a wave walks all heads of a token; the same bits as a call per part."""
    torch.manual_seed(1)
    t, hq, hkv, d = 4999, 9, 3, 128
    q, k = torch.randn(t, hq, d, device=dev).bfloat16(), torch.randn(t, hkv, d, device=dev).bfloat16()
    cs, pos = table(8192, d).to(dev), torch.arange(t, device=dev, dtype=torch.int32)
    yq, yk = qg.qk_norm_rope(q, k, None, None, cs, pos)
    for lo in (0, 1234, t - 57):
        pq, pk = qg.qk_norm_rope(q[lo:lo + 57], k[lo:lo + 57], None, None, cs, pos[lo:lo + 57].contiguous())
        assert torch.equal(pq, yq[lo:lo + 57]) and torch.equal(pk, yk[lo:lo + 57])
    check(yq[-3:], q[-3:], None, cs, pos[-3:], 1e-6, False)


@pytest.mark.parametrize("t,hq,d,rot,pairs", [(200001, 1, 64, 64, False), (70000, 2, 80, 32, True)])
def test_more_tokens_than_a_long_prompt(dev, t, hq, d, rot, pairs):
    torch.manual_seed(t)
    q, k = torch.randn(t, hq, d, device=dev).bfloat16(), torch.randn(t, 1, d, device=dev).bfloat16()
    w = (1 + torch.randn(d) * 0.3).bfloat16()
    cs, pos = table(4096, rot), torch.arange(t, device=dev, dtype=torch.int32) % 4096
    yq, yk = qg.qk_norm_rope(q, k, w.to(dev), None, cs.to(dev), pos, adjacent_pairs=pairs)
    assert yq.isfinite().all() and yk.isfinite().all()
    for lo in (0, 32700, 65500, t - 100):
        part = slice(lo, lo + 100)
        check(yq[part], q[part], w, cs, pos[part], 1e-6, pairs)
        check(yk[part], k[part], None, cs, pos[part], 1e-6, pairs)


def test_no_weights_eps_zero_rows_and_extremes(dev):
    d = 64
    q = torch.zeros(4, 2, d, dtype=torch.bfloat16, device=dev)
    q[1] = 1e-20
    q[2, 0] = 3e18          # the sum of squares stays finite
    q[2, 1, 5] = -2e15
    q[3] = torch.randn(2, d, device=dev).bfloat16()
    k = q[:, :1].contiguous()
    cs, pos = table(5, d).to(dev), torch.tensor([4, 0, 3, 1], dtype=torch.int32, device=dev)
    for eps in (1e-6, 1e-3):
        yq, yk = qg.qk_norm_rope(q, k, None, None, cs, pos, eps=eps)
        check(yq, q, None, cs, pos, eps, False)
        assert torch.equal(yk, yq[:, :1])


def test_position_outside_the_table_is_nan_and_flagged(dev):
    q = torch.randn(5, 2, 64, device=dev).bfloat16()
    k = torch.randn(5, 1, 64, device=dev).bfloat16()
    cs = table(10, 64).to(dev)
    pos = torch.tensor([0, 10, 9, -1, 2**31 - 1], dtype=torch.int32, device=dev)
    flag = torch.zeros(1, dtype=torch.int32, device=dev)
    yq, yk = qg.qk_norm_rope(q, k, None, None, cs, pos, status=flag)
    bad = torch.tensor([False, True, False, True, True], device=dev)
    assert torch.equal(yq.isnan().all(2).all(1), bad) and torch.equal(yq.isnan().any(2).any(1), bad)
    assert torch.equal(yk.isnan().any(2).any(1), bad)
    assert flag.item() == qg.FLAG_POSITION


def test_nan_stays_in_its_head(dev):
    q = torch.randn(2, 4, 128, device=dev).bfloat16()
    q[1, 2, 7] = float("nan")
    k = torch.randn(2, 1, 128, device=dev).bfloat16()
    yq, yk = qg.qk_norm_rope(q, k, None, None, table(4, 128).to(dev), torch.tensor([1, 2], dtype=torch.int32, device=dev))
    bad = yq.isnan().any(2)
    assert bad.sum() == 1 and bool(bad[1, 2]) and not yk.isnan().any()


def test_side_stream_graph_and_empty_call(dev):
    torch.manual_seed(3)
    q, k = torch.randn(33, 8, 128, device=dev).bfloat16(), torch.randn(33, 2, 128, device=dev).bfloat16()
    cs, pos = table(64, 128).to(dev), torch.arange(33, device=dev, dtype=torch.int32)
    want = qg.qk_norm_rope(q, k, None, None, cs, pos)
    out = (torch.empty_like(want[0]), torch.empty_like(want[1]))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        qg.qk_norm_rope(q, k, None, None, cs, pos, out=out)
    s.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qg.qk_norm_rope(q, k, None, None, cs, pos, out=out)
    for _ in range(3):
        out[0].zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    e = qg.qk_norm_rope(q[:0], k[:0], None, None, cs, pos[:0])
    assert e[0].shape == (0, 8, 128)


@pytest.mark.parametrize("d", [64, 128, 512])
def test_channels_whose_squares_leave_binary32(dev, d):
    """Heads of one magnitude from bf16's smallest normal numbers to its largest: the norm makes all of them
    of size one.  Without eps where the channels are small, as any eps would be larger than they are."""
    torch.manual_seed(d)
    cs, pos = table(5, d), torch.tensor([0, 4, 2, 3], dtype=torch.int32, device=dev)
    for size in (1e-37, 1e-30, 1e-24, 1e-20, 1e-18, 1e-10, 1.0, 1e10, 1e18, 3e18, 1e19, 1e30, 8e37):
        q = (torch.randn(4, 3, d).clamp(-4, 4) * size).bfloat16()
        for eps in ((0.0,) if size < 1e-9 else (0.0, 1e-6)):
            yq, yk = qg.qk_norm_rope(q.to(dev), q[:, :1].contiguous().to(dev), None, None, cs.to(dev), pos, eps=eps)
            check(yq, q, None, cs, pos, eps, False)
            assert torch.equal(yk, yq[:, :1])
    # one channel at the largest value of bf16 beside ordinary ones, in one head of three
    q = torch.randn(4, 3, d).bfloat16()
    q[:, 1, 3] = torch.finfo(torch.bfloat16).max
    yq, _ = qg.qk_norm_rope(q.to(dev), q[:, :1].contiguous().to(dev), None, None, cs.to(dev), pos)
    check(yq, q, None, cs, pos, 1e-6, False)


def test_small_heads_beside_a_small_eps(dev):
    """eps of the size of the mean square: both count."""
    torch.manual_seed(9)
    d = 128
    cs, pos = table(3, d), torch.tensor([2, 1], dtype=torch.int32, device=dev)
    for size, eps in ((1e-20, 1e-40), (1e-19, 1e-38), (1e-17, 1e-34), (1e-17, 0.0), (1e-14, 1e-28)):
        q = (torch.randn(2, 2, d) * size).bfloat16()
        yq, _ = qg.qk_norm_rope(q.to(dev), q[:, :1].contiguous().to(dev), None, None, cs.to(dev), pos, eps=eps)
        e = float(torch.tensor(eps, dtype=torch.float32))        # as the call takes it
        check(yq, q, None, cs, pos, e, False)
