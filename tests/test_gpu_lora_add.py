"""qg.lora_add against 64 bits.

Tolerance: the inner value v is a sum of k exact products of bf16 in fp32, in
chains of at most k / 128 matrix instructions of 32 products (counted as 32
additions each, of which the partial sums' magnitude is at most the sum of the
products' magnitudes), 4 waves and 16 splits: off by at most (k / 4 + 20) 2^-24
times sum |a x|.  It enters the second product with 24 bits (2^-23 with the
scale's rounding), whose 3 r terms are summed in fp32: (3 r + 3) 2^-24 times
sum |b v|; then one addition and the rounding to the output's type."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gemm_decode_qgemm_amd as qg
import serving_reference as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
BITS = {BF16: 8, F32: 24}


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


def make(m, k, n, r, adapters, yt=BF16, seed=0):
    g = torch.Generator().manual_seed(seed + m + 7 * k + 11 * n + 13 * r)
    x = torch.randn(m, k, generator=g).bfloat16()
    a = (torch.randn(adapters, r, k, generator=g) * k ** -0.5).bfloat16()
    b = (torch.randn(adapters, n, r, generator=g) * r ** -0.5).bfloat16()
    y = torch.randn(m, n, generator=g).to(yt)
    scales = 0.2 + torch.rand(adapters, generator=g)
    ids = torch.randint(-1, adapters, (m,), generator=g).to(torch.int32)
    return y, x, a, b, ids, scales


def check(out, y, x, a, b, ids, scales):
    y, x, a, b = (ref.f64(t) for t in (y, x, a, b))
    s = np.ones(a.shape[0]) if scales is None else ref.f64(scales)
    k, r = x.shape[1], a.shape[1]
    got, eps = ref.f64(out), 2.0 ** -24
    for m, i in enumerate(ids.tolist()):
        if i < 0:
            want, tol = y[m], 0.0
        else:
            v = s[i] * (a[i] @ x[m])
            dv = s[i] * (np.abs(a[i]) @ np.abs(x[m])) * (k / 4 + 20) * eps
            want = y[m] + b[i] @ v
            tol = np.abs(b[i]) @ (dv + np.abs(v) * (3 * r + 5) * eps) + np.abs(want) * 2 * eps
        tol = tol + ref.half_step(np.abs(want) + tol, BITS[out.dtype]) * (i >= 0 or out.dtype == BF16)
        bad = ~(np.abs(got[m] - want) <= tol)
        assert not bad.any(), (m, i, np.argwhere(bad)[:3].ravel(), got[m][bad][:3], want[bad][:3])


@pytest.mark.parametrize("yt", [BF16, F32])
@pytest.mark.parametrize("m,k,n,r,adapters", [(64, 64, 16385, 8, 64), (40, 64, 30001, 16, 64), (64, 72, 131072, 16, 8), (64, 64, 131075, 8, 9),
                                               (33, 512, 700, 8, 3), (50, 512, 700, 16, 6), (64, 128, 4099, 24, 64)])
def test_low_ranks_beside_wide_projections(dev, m, k, n, r, adapters, yt):
    args = make(m, k, n, r, adapters, yt)
    y, x, a, b, ids, scales = (t.to(dev) for t in args)
    check(qg.lora_add(y, x, a, b, ids, scales=scales), *args)
    check(qg.lora_add(y, x, a, b, ids, out_dtype=F32 if yt is BF16 else BF16), *args[:5], None)


@pytest.mark.parametrize("m,k,n,r,adapters", [
    (1, 8, 1, 8, 1), (1, 256, 256, 16, 4), (2, 264, 33, 24, 1), (3, 1000, 257, 16, 3), (5, 512, 1000, 32, 2), (16, 1024, 64, 40, 1),
    (17, 768, 129, 64, 1), (33, 520, 300, 16, 2), (64, 256, 70, 8, 1), (64, 1280, 513, 64, 64), (64, 2048, 130, 128, 3),
    (40, 512, 200, 256, 1), (64, 256, 65, 248, 2), (64, 6656, 256, 16, 7), (9, 19968, 100, 72, 20), (31, 4096, 2000, 16, 100)])
@pytest.mark.parametrize("yt", [BF16, F32])
def test_against_64_bits(dev, m, k, n, r, adapters, yt):
    args = make(m, k, n, r, adapters, yt)
    y, x, a, b, ids, scales = (t.to(dev) for t in args)
    check(qg.lora_add(y, x, a, b, ids, scales=scales), *args)
    check(qg.lora_add(y, x, a, b, ids, out_dtype=F32 if yt is BF16 else BF16), *args[:5], None)


def test_every_row_has_its_own_result_whatever_the_batch(dev):
    """The rows that share an adapter, and their order, change nothing."""
    y, x, a, b, ids, scales = (t.to(dev) for t in make(64, 1024, 300, 16, 9))
    want = qg.lora_add(y, x, a, b, ids, scales=scales)
    order = torch.randperm(64, device=dev)
    got = qg.lora_add(y[order].contiguous(), x[order].contiguous(), a, b, ids[order].contiguous(), scales=scales)
    assert torch.equal(got, want[order])
    same = torch.full_like(ids, 3)
    all_of_one = qg.lora_add(y, x, a, b, same, scales=scales)
    assert torch.equal(all_of_one[ids == 3], want[ids == 3])


def test_in_place_views_and_rows_without_adapter(dev):
    args = make(7, 512, 200, 16, 5)
    y, x, a, b, ids, scales = (t.to(dev) for t in args)
    ids[2] = ids[5] = -1
    ids[3] = -(2 ** 31)
    big = torch.full((7, 701), 3.0, dtype=BF16, device=dev)
    view = big[:, 101:301]
    view.copy_(y)
    out = qg.lora_add(view, x, a, b, ids, scales=scales, out=view)
    assert out.data_ptr() == view.data_ptr()
    check(out, *args[:4], ids, args[5])
    assert torch.equal(out[2], y[2]) and torch.equal(out[3], y[3])
    assert bool((big[:, :101] == 3).all()) and bool((big[:, 301:] == 3).all())
    none = torch.full_like(ids, -1)
    assert torch.equal(qg.lora_add(y, x, a, b, none, scales=scales), y)
    other = torch.full((7, 400), 3.0, dtype=F32, device=dev)
    assert torch.equal(qg.lora_add(y, x, a, b, none, out=other[:, 100:300]), y.float()) and bool((other[:, :100] == 3).all())


def test_adapters_outside_those_held(dev):
    y, x, a, b, ids, scales = (t.to(dev) for t in make(6, 256, 70, 8, 3))
    ids = torch.tensor([0, 3, -1, 2 ** 31 - 1, 2, 1], dtype=torch.int32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    out = qg.lora_add(y, x, a, b, ids, scales=scales, status=status)
    assert status.item() == qg.FLAG_INDEX
    assert bool(out[[1, 3]].isnan().all()) and bool(out[[0, 2, 4, 5]].isfinite().all()) and torch.equal(out[2], y[2])
    status.zero_()
    qg.lora_add(y, x, a, b, ids.clamp(-1, 2), scales=scales, status=status)
    assert status.item() == 0
    assert torch.equal(qg.lora_add(y[:2], x[:2], a, b, ids[:2]).isnan().all(1).cpu(), torch.tensor([False, True]))   # by rows


def test_values_that_are_not_finite_stay_with_their_rows(dev):
    y, x, a, b, ids, scales = (t.to(dev) for t in make(4, 256, 70, 8, 2))
    ids = torch.tensor([0, 1, 1, -1], dtype=torch.int32, device=dev)
    x[1, 9] = float("nan")
    scales[0] = float("inf")
    out = qg.lora_add(y, x, a, b, ids, scales=scales)
    assert not bool(out[0].isfinite().any()) and bool(out[1].isnan().all()) and bool(out[2:].isfinite().all())


def test_graphs_that_share_a_workspace_and_streams(dev):
    m, k, n, r, adapters = 19, 2048, 777, 32, 6
    y, x, a, b, ids, scales = (t.to(dev) for t in make(m, k, n, r, adapters))
    ws = torch.empty(qg.lora_add_workspace_bytes(m, k, n, r, adapters), dtype=torch.uint8, device=dev)
    outs = [torch.empty_like(y), torch.empty_like(y)]
    other = ids.flip(0).contiguous()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    qg.lora_add(y, x, a, b, ids, scales=scales, out=outs[0], workspace=ws)
    for g, i, o in zip(graphs, (ids, other), outs):
        with torch.cuda.graph(g):
            qg.lora_add(y, x, a, b, i, scales=scales, out=o, workspace=ws)
    for k_ in range(3):
        x.copy_(torch.randn(m, k, device=dev))
        want = [qg.lora_add(y, x, a, b, i, scales=scales) for i in (ids, other)]
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]), k_
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = qg.lora_add(y, x, a, b, ids, scales=scales)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want[0])
    assert qg.lora_add(y[:0], x[:0], a, b, ids[:0]).shape == (0, n)


def test_the_largest_widths(dev):
    """Offsets of an adapter past 2^31 elements."""
    k, r, n = 2 ** 20, 64, 128
    adapters = 34                               # 34 * 64 * 2^20 elements of A: 4.25 GiB
    a = torch.zeros(adapters, r, k, dtype=BF16, device=dev)
    a[33] = (torch.randn(r, k, device=dev) * k ** -0.5).bfloat16()
    b = torch.randn(adapters, n, r, device=dev).bfloat16()
    x = torch.randn(2, k, device=dev).bfloat16()
    y = torch.randn(2, n, device=dev)
    ids = torch.tensor([33, 0], dtype=torch.int32, device=dev)
    out = qg.lora_add(y, x, a, b, ids)
    v = torch.matmul(a[33].double(), x[0].double())
    want = y[0].double() + torch.matmul(b[33].double(), v)
    # the chain of 2^20 / 128 additions of positive and negative terms, far under its bound of (k / 4) 2^-24
    assert float((out[0].double() - want).abs().max()) <= 1e-2 and torch.equal(out[1], y[1])


def test_adapters_and_rows_that_no_one_names_are_not_read(dev):
    y, x, a, b, ids, scales = (t.to(dev) for t in make(24, 520, 130, 24, 5))
    ids = torch.tensor([0, 2, -1, 4] * 6, dtype=torch.int32, device=dev)
    want = qg.lora_add(y, x, a, b, ids, scales=scales)
    x[2::4] = float("nan")
    for i in (1, 3):
        a[i], b[i], scales[i] = float("nan"), float("nan"), float("nan")
    assert torch.equal(qg.lora_add(y, x, a, b, ids, scales=scales), want)
    few = slice(0, 4)                          # fewer rows than adapters
    assert torch.equal(qg.lora_add(y[few], x[few], a, b, ids[few].contiguous(), scales=scales), want[few])


def test_two_streams_at_once(dev):
    """Calls that overlap, each with a workspace of its own."""
    args = [tuple(t.to(dev) for t in make(33, 2048, 5000, 64, 20, seed=s)) for s in (0, 1)]
    want = [qg.lora_add(*c[:5], scales=c[5]) for c in args]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(qg.lora_add(*args[i][:5], scales=args[i][5]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in (0, 1) for o in got[i])


@pytest.mark.parametrize("r", [8, 16, 24, 64])
@pytest.mark.parametrize("n,adapters", [(300, 5), (20000, 64)])
def test_weights_that_are_not_finite_stay_with_their_columns(dev, r, n, adapters):
    """Infinities and NaN in B reach the columns that they weigh, of the rows with that adapter, and no other; an inner
    value that is infinite is taken as it is."""
    y, x, a, b, ids, scales = (t.to(dev) for t in make(64, 128, n, r, adapters))
    ids = (torch.arange(64, device=dev) % 5).to(torch.int32)
    want = qg.lora_add(y, x, a, b, ids, scales=scales)
    inf, nan = float("inf"), float("nan")
    b[1, 17, 3], b[1, 100, r - 1], b[3, 40, 0], b[3, 299, 5] = nan, inf, -inf, nan
    got = qg.lora_add(y, x, a, b, ids, scales=scales)
    bad = torch.zeros(64, n, dtype=torch.bool, device=dev)
    bad[1::5, 17] = bad[1::5, 100] = bad[3::5, 40] = bad[3::5, 299] = True
    assert torch.equal(got[~bad], want[~bad])
    inner = [scales[i].double() * (x[i::5].double() @ a[i].double().t()) for i in (1, 3)]
    assert bool(got[1::5, 17].isnan().all()) and bool(got[3::5, 299].isnan().all())
    assert torch.equal(got[1::5, 100].double(), inner[0][:, r - 1] * inf) and torch.equal(got[3::5, 40].double(), inner[1][:, 0] * -inf)
    scales[0] = inf                            # an inner value's sign times a weight's: infinite or, where they differ, NaN
    ref_ = y.double()[0] + (scales[0].double() * (a[0].double() @ x[0].double())) @ b[0].double().t()
    got = qg.lora_add(y, x, a, b, ids, scales=scales, out_dtype=F32)[0]
    assert torch.equal(got.isnan(), ref_.isnan()) and torch.equal(got.isinf(), ref_.isinf())


@pytest.mark.parametrize("r", [8, 16, 24, 40, 64, 72, 136])
@pytest.mark.parametrize("m", [1, 9])
def test_an_infinite_scale_reaches_the_ranks_that_there_are(dev, m, r):
    """Ranks that fill up a matrix operand are no part of the sums: positive products times an infinite scale are infinite."""
    k, n = 72, 301
    g = torch.Generator().manual_seed(r)
    x, a, b = (0.5 + torch.rand(s, generator=g).bfloat16().to(dev) for s in ((m, k), (2, r, k), (2, n, r)))
    y = torch.randn(m, n, generator=g).to(dev)
    ids = torch.ones(m, dtype=torch.int32, device=dev)
    for s in (float("inf"), -float("inf")):
        out = qg.lora_add(y, x, a, b, ids, scales=torch.tensor([1.0, s], device=dev))
        assert bool((out == s).all())


@pytest.mark.parametrize("r", [8, 16, 40])
def test_inner_values_next_to_the_largest_binary32(dev, r):
    """An inner value keeps its 24 bits up to the largest binary32 number, where bf16 rounds to infinity.

    One product a rank, exact in fp32: v = s c with c a power of two.  It enters the second product as a sum of three bf16,
    which hold its 24 bits, b = 2^-20 is exact, and r equal terms are summed in fp32: off by (3 r + 2) 2^-24 at most."""
    k, n = 8, 70
    x = torch.zeros(3, k, dtype=BF16, device=dev)
    x[:, 3] = 1.0
    a = torch.zeros(3, r, k, dtype=BF16, device=dev)
    a[:, :, 3] = 2.0 ** 100
    b = torch.full((3, n, r), 2.0 ** -20, dtype=BF16, device=dev)
    scales = torch.tensor([2.0 ** 28 * (1 - 2.0 ** -24), 2.0 ** 27 * (1 + 2.0 ** -12 + 2.0 ** -23), -(2.0 ** 28) * (1 - 2.0 ** -10 + 2.0 ** -24)],
                          device=dev)
    ids = torch.arange(3, dtype=torch.int32, device=dev)
    out = qg.lora_add(torch.zeros(3, n, device=dev), x, a, b, ids, scales=scales)
    want = r * 2.0 ** 80 * ref.f64(scales)[:, None]
    assert np.all(np.abs(ref.f64(out) - want) <= (3 * r + 2) * 2.0 ** -24 * np.abs(want))
