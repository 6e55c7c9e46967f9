"""qg.rms_norm and qg.rms_norm_q8 against 64 bits.

Tolerances: a thread sums up to 32 squares one after another, then trees of at
most 10 steps and 16 partial sums join them, so the mean square is off by at most
(32 + 10 + 16) 2^-24 of itself and the norm by half of that; with the handful of
single roundings around it y is off by less than 2^-18 of itself before its own
rounding: to nearest, half a step.  The sum x + residual is rounded once to
32 bits (2^-24) and once to the stream's type."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gemm_decode_qgemm_amd as qg
import serving_reference as ref

pytestmark = pytest.mark.gpu
BITS = {torch.bfloat16: 8, torch.float32: 24}
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


def check(y, want, dtype, rel=2.0 ** -18):
    got = ref.f64(y)
    assert y.dtype == dtype and got.shape == want.shape
    near = ref.half_step(want * (1 + rel), BITS[dtype]) + rel * np.abs(want)
    bad = ~(np.abs(got - want) <= near)
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])


def inputs(t, h, xt, rt, seed=0):
    g = torch.Generator().manual_seed(1000 * t + h + seed)
    x = torch.randn(t, h, generator=g)
    x[:, 5 % h] *= 30
    res = None if rt is None else (3 * torch.randn(t, h, generator=g)).to(rt)
    w = (1 + 0.3 * torch.randn(h, generator=g)).bfloat16()
    return x.to(xt), res, w


def put(t, dev):
    return None if t is None else t.to(dev)


SIZES = [(1, 8), (3, 64), (5, 512), (2, 520), (7, 1024), (4, 1032), (9, 2048), (3, 2056), (2, 4096), (3, 4104), (2, 6656),
         (1, 8192), (3, 8200), (2, 16384), (2, 16392), (1, 32768), (301, 96), (1025, 256)]


@pytest.mark.parametrize("t,h", SIZES)
@pytest.mark.parametrize("xt,rt,ot", [(BF16, None, BF16), (BF16, BF16, BF16), (BF16, F32, F32), (F32, BF16, BF16), (F32, F32, F32),
                                      (F32, None, BF16)])
def test_norm(dev, t, h, xt, rt, ot):
    x, res, w = inputs(t, h, xt, rt)
    got = qg.rms_norm(x.to(dev), w.to(dev), residual=put(res, dev), out_dtype=ot)
    want, r = ref.rms_norm(ref.f64(x), None if res is None else ref.f64(res), ref.f64(w), 1e-6)
    if rt is None:
        check(got, want, ot)
    else:
        check(got[0], want, ot)
        check(got[1], r, rt, rel=2.0 ** -24 if rt is BF16 else 0.0)


def check_q8(codes, scales, want, group):
    c, s = ref.f64(codes), ref.f64(scales)
    t, h = want.shape
    wide = want.reshape(t, -1, group or h)
    a = np.abs(wide).max(2)
    assert s.shape == ((t, h // 32) if group else (t,)) and codes.dtype == torch.int8
    s = s.reshape(t, -1)
    assert np.all(np.abs(s - a / 127) <= 2.0 ** -17 * a / 127)
    c = c.reshape(wide.shape)
    assert np.abs(c).max() <= 127
    # off by half a step, and by what y and its scale are off where that crosses a tie
    exact = wide / np.maximum(a, 1e-300)[..., None] * 127
    assert np.all(np.abs(c - exact) <= 0.5 + 127 * 2.0 ** -16)


@pytest.mark.parametrize("t,h", [(1, 32), (3, 64), (5, 512), (2, 544), (7, 1024), (4, 1056), (9, 2048), (2, 2080), (3, 4096), (2, 6656), (1, 8224),
                                 (2, 16384), (2, 19968), (1, 32768), (515, 96)])
@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("xt,rt", [(BF16, BF16), (F32, F32), (BF16, None), (F32, None)])
def test_norm_q8(dev, t, h, group, xt, rt):
    x, res, w = inputs(t, h, xt, rt, seed=1)
    codes, scales, *r = qg.rms_norm_q8(x.to(dev), w.to(dev), residual=put(res, dev), group_scales=bool(group))
    want, sums = ref.rms_norm(ref.f64(x), None if res is None else ref.f64(res), ref.f64(w), 1e-6)
    check_q8(codes, scales, want, group)
    if rt is not None:
        check(r[0], sums, rt, rel=2.0 ** -24 if rt is BF16 else 0.0)


def test_rows_of_eight_channels_in_8_bits(dev):
    """Row scales need no whole groups."""
    x, _, w = inputs(3, 40, BF16, None)
    codes, scales = qg.rms_norm_q8(x.to(dev), w.to(dev))
    check_q8(codes, scales, ref.rms_norm(ref.f64(x), None, ref.f64(w), 1e-6)[0], 0)


@pytest.mark.parametrize("h", [128, 4096, 16384])
def test_views_in_place_and_no_weight(dev, h):
    t = 5
    x, res, w = inputs(t, h, BF16, BF16)
    big = torch.full((t, 3 * h + 8), 7.0, dtype=BF16, device=dev)
    big[:, h:2 * h], big[:, 2 * h + 8:] = x.to(dev), res.to(dev)
    y, r = qg.rms_norm(big[:, h:2 * h], None, residual=big[:, 2 * h + 8:], eps=0.25)
    want, sums = ref.rms_norm(ref.f64(x), ref.f64(res), None, 0.25)
    check(y, want, BF16)
    check(r, sums, BF16, rel=2.0 ** -24)
    stream = res.to(dev)
    y2, r2 = qg.rms_norm(x.to(dev), None, residual=stream, residual_out=stream, eps=0.25)
    assert r2.data_ptr() == stream.data_ptr() and torch.equal(r2, r) and torch.equal(y2, y)
    assert bool((big[:, :h] == 7).all())
    one = big[2:3, h:2 * h].as_strided((1, h), (h + 3, 1), big[2:3, h:2 * h].storage_offset())   # one row: any stride
    assert torch.equal(qg.rms_norm(one, None, eps=0.25), qg.rms_norm(x[2:3].to(dev), None, eps=0.25))


def test_channels_whose_squares_leave_binary32(dev):
    for h in (96, 4096, 20000):
        for size in (1e-38, 1e-30, 1e-24, 1e-20, 1e-18, 1e-10, 1.0, 1e10, 1e18, 3e18, 1e19, 1e30, 8e37):
            x = torch.randn(2, h).clamp(-4, 4) * size
            for eps in ((0.0,) if size < 1e-9 else (0.0, 1e-6)):
                want, _ = ref.rms_norm(ref.f64(x), None, None, eps)
                check(qg.rms_norm(x.to(dev), eps=eps, out_dtype=F32), want, F32)
    x = torch.full((1, 512), 1e-42)            # denormal numbers
    check(qg.rms_norm(x.to(dev), eps=0.0, out_dtype=F32), np.ones((1, 512)), F32)
    e = float(torch.tensor(1e-40))
    x = torch.randn(2, 256) * 1e-20
    check(qg.rms_norm(x.to(dev), eps=e, out_dtype=F32), ref.rms_norm(ref.f64(x), None, None, e)[0], F32)


def test_rows_that_are_zero_or_not_finite(dev):
    x = torch.randn(4, 512).bfloat16()
    x[0] = 0
    x[1, 77] = float("inf")
    x[2, 100] = float("nan")
    y = ref.f64(qg.rms_norm(x.to(dev)))
    assert np.all(y[0] == 0) and np.isnan(y[1, 77]) and np.isnan(y[2]).all() and np.isfinite(y[3]).all()
    assert np.all(np.delete(y[1], 77) == 0)    # the others over an infinite norm
    codes, scales = qg.rms_norm_q8(x.to(dev))
    s = ref.f64(scales)
    assert s[0] == 0 and np.isnan(s[1]) and np.isnan(s[2]) and s[3] > 0 and not codes[0].any()
    codes, scales = qg.rms_norm_q8(x.to(dev), group_scales=True)
    s = ref.f64(scales)
    assert np.all(s[0] == 0) and np.isnan(s[1, 77 // 32]) and np.isnan(s[2]).all() and np.isfinite(np.delete(s[1], 77 // 32)).all()


def test_graph_streams_empty_and_repeats(dev):
    x, res, w = (t.to(dev) for t in inputs(33, 6656, BF16, F32))
    want = qg.rms_norm_q8(x, w, residual=res)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = qg.rms_norm_q8(x, w, residual=res)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    outs = (torch.zeros_like(want[0]), torch.zeros_like(want[1]))
    stream = torch.zeros_like(res)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qg.rms_norm_q8(x, w, residual=res, out=outs, residual_out=stream)
    for k in range(3):
        x.copy_(torch.randn(33, 6656, device=dev))
        graph.replay()
        torch.cuda.synchronize()
        want = qg.rms_norm_q8(x, w, residual=res)
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]) and torch.equal(stream, want[2]), k
    e = qg.rms_norm(x[:0], w, residual=res[:0])
    assert e[0].shape == (0, 6656) and e[1].dtype == F32


def test_a_device_that_is_not_the_current_one(dev, monkeypatch):
    """The wrapper makes the tensors' device current for the launch."""
    x = torch.randn(2, 64, device=dev)
    want = qg.rms_norm(x)
    monkeypatch.setattr(qg.binding, "_current", lambda: -1)
    assert torch.equal(qg.rms_norm(x), want)


@pytest.mark.parametrize("h", [128, 2056, 6656, 20000])
def test_over_its_own_input(dev, h):
    """y over x, and the sum over the residual, in one call."""
    x, res, w = (t.to(dev) for t in inputs(9, h, BF16, BF16))
    y, r = qg.rms_norm(x, w, residual=res)
    got = qg.rms_norm(x, w, residual=res, out=x, residual_out=res)
    assert got[0].data_ptr() == x.data_ptr() and torch.equal(got[0], y) and torch.equal(got[1], r)


def test_rows_past_two_to_the_31_elements(dev):
    t, h = 2 ** 19 + 3, 4096
    x = torch.zeros(t, h, dtype=BF16, device=dev)
    x[-5:] = torch.randn(5, h, device=dev)
    y = qg.rms_norm(x)
    codes, scales = qg.rms_norm_q8(x, group_scales=True)
    few = x[-5:].clone()
    assert torch.equal(y[-5:], qg.rms_norm(few)) and not bool(y[-6].any())
    want = qg.rms_norm_q8(few, group_scales=True)
    assert torch.equal(codes[-5:], want[0]) and torch.equal(scales[-5:], want[1]) and not bool(scales[-6].any())
