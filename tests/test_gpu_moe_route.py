"""qg.moe_route against 64 bits: the same experts in the same order, weights within
half a step of fp32 (plus the 64-bit errors of a sum over 512 scores: 2^-40)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gemm_decode_qgemm_amd as qg
import serving_reference as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


def check(dev, l, k, sigmoid=False, bias=None, groups=1, top_groups=1, best=1, renorm=True, scale=1.0):
    ids, w = qg.moe_route(l.to(dev), k, sigmoid=sigmoid, bias=None if bias is None else bias.to(dev), groups=groups,
                          top_groups=top_groups, group_best=best, renormalize=renorm, scale=scale)
    want, weights = ref.route(ref.f64(l), k, sigmoid, None if bias is None else ref.f64(bias), groups, top_groups, best, renorm,
                              float(torch.tensor(scale)))
    assert ids.dtype == torch.int32 and w.dtype == F32
    assert np.array_equal(ids.cpu().numpy(), want), np.argwhere(ids.cpu().numpy() != want)[:3]
    tol = ref.half_step(np.abs(weights) * (1 + 2.0 ** -30), 24) + 2.0 ** -40 * np.abs(weights)
    got = ref.f64(w)
    bad = ~((np.abs(got - weights) <= tol) | (np.isnan(got) & np.isnan(weights)))
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], weights[bad][:3])
    return ids, w


@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (3, 2, 2), (5, 8, 2), (7, 16, 16), (9, 60, 6), (4, 64, 8), (130, 65, 3), (61, 128, 8), (33, 160, 6),
                                   (17, 256, 8), (5, 257, 32), (11, 384, 10), (3, 512, 32), (1000, 64, 4)])
@pytest.mark.parametrize("sigmoid,bias,renorm", [(False, False, True), (False, True, False), (True, True, True), (True, False, False)])
@pytest.mark.parametrize("half", [False, True])
def test_choice(dev, t, e, k, sigmoid, bias, renorm, half):
    torch.manual_seed(t + e)
    l = 2 * torch.randn(t, e)
    check(dev, l.bfloat16() if half else l, k, sigmoid, 0.2 * torch.randn(e) if bias else None, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("e,groups,top,k", [(256, 8, 4, 8), (256, 8, 1, 8), (64, 64, 7, 5), (160, 8, 3, 6), (512, 4, 2, 32), (384, 8, 8, 9), (66, 6, 2, 11),
                                            (128, 2, 1, 32)])
@pytest.mark.parametrize("sigmoid,bias", [(False, False), (True, True), (True, False), (False, True)])
def test_groups(dev, e, groups, top, k, sigmoid, bias):
    torch.manual_seed(e + groups)
    l = 2 * torch.randn(53, e)
    for best in (1, 2) if e > groups else (1,):
        check(dev, l, k, sigmoid, 0.2 * torch.randn(e) if bias else None, groups, top, best, renorm=best == 2)
        check(dev, l.bfloat16(), k, sigmoid, 0.2 * torch.randn(e).bfloat16().float() if bias else None, groups, top, best)


def test_ties_go_to_the_lowest_index(dev):
    l = torch.zeros(3, 256)
    l[1, 200:] = 1.0
    l[2] = torch.arange(256) % 4
    for sigmoid in (False, True):
        for bias in (None, torch.zeros(256), torch.full((256,), 0.5)):
            check(dev, l, 8, sigmoid, bias)
            check(dev, l, 8, sigmoid, bias, 8, 3, 2)
            check(dev, l, 8, sigmoid, bias, 8, 3, 1)
    # an expert's bias makes up exactly for another's score
    check(dev, torch.zeros(1, 4), 2, True, torch.tensor([0.25, 0.5, 0.25, 0.5]))


def test_near_ties_that_32_bits_do_not_tell_apart(dev):
    """Scores of logits that differ in the last bits, biased so that the scores' first digits are lost in 32 bits."""
    torch.manual_seed(4)
    l = (1 + torch.arange(512).flip(0) * 2.0 ** -23)[torch.randperm(512)].repeat(5, 1)
    bias = torch.full((512,), 8.0)
    check(dev, l, 16, True, bias)
    check(dev, l, 16, False, bias)
    check(dev, l, 16, True, bias, 8, 3, 2)
    check(dev, l, 16, True, None)
    # far along the sigmoid, where 32 bits hold a one
    check(dev, 20 + 0.01 * torch.randn(9, 256), 8, True, torch.zeros(256))


def test_masked_experts_and_rows_without_any(dev):
    inf = float("inf")
    l = torch.randn(6, 64)
    l[0, 3:] = -inf                        # three experts left for four picks
    l[1] = -inf
    l[2, ::2] = torch.finfo(F32).min
    l[3] = torch.finfo(F32).min
    l[4, 10] = 80.0
    l[5, 20] = torch.finfo(F32).max
    for sigmoid in (False, True):
        for renorm in (False, True):
            for groups in (1, 8):
                check(dev, l, 4, sigmoid, None, groups, 1 if groups == 1 else 4, renorm=renorm)
    bias = torch.zeros(64)
    bias[5] = -inf                         # an expert that the bias takes out
    ids, _ = check(dev, l[2:5], 8, True, bias)
    assert not bool((ids == 5).any())
    ids, w = qg.moe_route(l[1:2].to(dev), 4)
    assert ids.tolist() == [[0, 1, 2, 3]] and not bool(w.any())


def test_nan_counts_as_the_largest(dev):
    l = torch.randn(2, 128)
    l[0, 77] = float("nan")
    for kw in (dict(), dict(sigmoid=True, bias=torch.zeros(128, device=dev)), dict(sigmoid=True, groups=4, top_groups=1, group_best=2)):
        ids, w = qg.moe_route(l.to(dev), 4, **kw)
        assert ids[0, 0] == 77 and bool(w[1].isfinite().all()) and bool(w[0, 0].isnan())


def test_long_prompts_graph_and_out(dev):
    l = torch.randn(70001, 64, device=dev)
    ids, w = qg.moe_route(l, 6, sigmoid=True, scale=0.5)
    top = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :6]
    assert torch.equal(ids.long(), top)
    l = torch.randn(37, 256, device=dev)
    bias = 0.1 * torch.randn(256, device=dev)
    kw = dict(sigmoid=True, bias=bias, groups=8, top_groups=4, group_best=2)
    out = (torch.zeros(37, 8, dtype=torch.int32, device=dev), torch.zeros(37, 8, device=dev))
    graph = torch.cuda.CUDAGraph()
    qg.moe_route(l, 8, **kw)
    with torch.cuda.graph(graph):
        qg.moe_route(l, 8, **kw, out=out)
    for k in range(3):
        l.copy_(torch.randn(37, 256, device=dev))
        graph.replay()
        torch.cuda.synchronize()
        want = qg.moe_route(l, 8, **kw)
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]), k
    e = qg.moe_route(l[:0], 8, **kw)
    assert e[0].shape == (0, 8) and e[1].shape == (0, 8)


# ---- many tokens: four of them a wave, up to 256 experts and 8 picks ------------------

def check_many(dev, l, k, **kw):
    """A few hundred tokens, each many times over in any order, as many as that takes; the reference takes each once."""
    n = l.shape[0]
    order = torch.randint(0, n, (16387,), generator=torch.Generator().manual_seed(n))
    order[:n] = torch.arange(n)
    bias = kw.get("bias")
    ids, w = qg.moe_route(l[order].to(dev), k, sigmoid=kw.get("sigmoid", False), bias=None if bias is None else bias.to(dev),
                          groups=kw.get("groups", 1), top_groups=kw.get("top_groups", 1), group_best=kw.get("best", 1),
                          renormalize=kw.get("renorm", True), scale=kw.get("scale", 1.0))
    once = check(dev, l, k, **kw)
    assert torch.equal(ids, once[0][order.to(dev)])
    again = once[1][order.to(dev)]
    # both within half a step of the same number, and a hair more: a step of the last place apart at most
    assert bool(((w - again).abs() <= 2.0 ** -23 * again.abs()).logical_or(w.isnan() & again.isnan()).all())


@pytest.mark.parametrize("e,k", [(4, 1), (8, 2), (60, 6), (64, 8), (72, 5), (100, 4), (128, 8), (256, 8), (144, 6), (512, 8), (8, 8), (256, 1)])
@pytest.mark.parametrize("sigmoid,bias,renorm", [(False, False, True), (False, True, False), (True, True, True), (True, False, False)])
@pytest.mark.parametrize("half", [False, True])
def test_many_tokens(dev, e, k, sigmoid, bias, renorm, half):
    torch.manual_seed(e + k)
    l = 2 * torch.randn(203, e)
    check_many(dev, l.bfloat16() if half else l, k, sigmoid=sigmoid, bias=0.2 * torch.randn(e) if bias else None, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("e,groups,top,k", [(128, 8, 4, 8), (128, 16, 1, 8), (64, 16, 7, 5), (64, 8, 3, 6), (96, 4, 2, 8), (32, 2, 1, 8), (256, 8, 4, 8),
                                            (128, 2, 1, 8), (96, 6, 2, 4), (256, 2, 1, 8), (192, 4, 2, 8), (256, 16, 2, 5)])
@pytest.mark.parametrize("sigmoid,bias", [(False, False), (True, True), (True, False), (False, True)])
@pytest.mark.parametrize("half", [False, True])
def test_many_tokens_in_groups(dev, e, groups, top, k, sigmoid, bias, half):
    torch.manual_seed(e + groups)
    l = 2 * torch.randn(150, e)
    for best in (1, 2):
        check_many(dev, l.bfloat16() if half else l, k, sigmoid=sigmoid, bias=0.2 * torch.randn(e) if bias else None, groups=groups,
                   top_groups=top, best=best, renorm=best == 2)


@pytest.mark.parametrize("e", [64, 128, 256])
def test_many_tokens_with_ties_clusters_masks_and_nan(dev, e):
    """Equal logits, the best experts side by side, experts masked out, tokens with nothing left, and NaN: token by token
    beside ordinary ones."""
    inf = float("inf")
    torch.manual_seed(e)
    l = torch.randn(160, e)
    l[::8] = 0.0
    l[1::8, 5:16] += 20.0
    l[2::8] = torch.randint(0, 3, (20, e)).float()
    l[3::8, 9:] = -inf
    l[4::8] = -inf
    l[5::16, e // 2] = torch.finfo(F32).max
    l[6::8, 1::2] = torch.finfo(F32).min
    l[7::8] = 1 + torch.arange(e).flip(0) * 2.0 ** -23
    for sigmoid, bias in ((False, None), (True, None), (True, torch.zeros(e)), (False, torch.zeros(e)), (True, torch.full((e,), 8.0))):
        for groups in (1, 4):
            for half in (False, True):
                check_many(dev, l.bfloat16() if half else l, 8, sigmoid=sigmoid, bias=bias, groups=groups, top_groups=max(1, groups // 2),
                           best=1 if sigmoid or groups == 1 else 2)
    l[13, 33] = float("nan")
    l = l.repeat(103, 1)
    for kw in (dict(), dict(sigmoid=True, bias=torch.zeros(e, device=dev)), dict(sigmoid=True, groups=4, top_groups=1, group_best=2)):
        for x in (l, l.bfloat16()):
            ids, w = qg.moe_route(x.to(dev), 4, **kw)
            # (the largest binary32 number is an infinity in bf16, beside which a softmax has no scores)
            others = (x < inf).all(1) | torch.tensor("sigmoid" in kw)
            others[13::160] = False
            assert bool((ids[13::160, 0] == 33).all()) and bool(w[13::160, 0].isnan().all()) and bool(w[others.to(dev)].isfinite().all())


def test_many_tokens_at_addresses_that_are_not_aligned(dev):
    """Logits and bias 4 bytes off: the other way, with the same result."""
    torch.manual_seed(8)
    l, bias = torch.randn(17000, 128), 0.1 * torch.randn(128)
    want = qg.moe_route(l.to(dev), 8, sigmoid=True, bias=bias.to(dev))
    room = torch.empty(17000 * 128 + 1, device=dev)
    room[1:] = l.flatten().to(dev)
    room_b = torch.empty(129, device=dev)
    room_b[1:] = bias.to(dev)
    got = qg.moe_route(room[1:].view(17000, 128), 8, sigmoid=True, bias=room_b[1:])
    assert torch.equal(got[0], want[0]) and bool(((got[1] - want[1]).abs() <= 2.0 ** -23 * want[1]).all())


@pytest.mark.parametrize("e", [64, 512])           # four tokens a wave; one
def test_logits_past_two_to_the_31_elements(dev, e):
    t = 2 ** 31 // e + 5
    l = torch.zeros(t, e, dtype=BF16, device=dev)
    l[-7:] = torch.randn(7, e, device=dev)
    ids, w = qg.moe_route(l, 6, sigmoid=True)
    want = qg.moe_route(l[-7:].clone(), 6, sigmoid=True)
    assert torch.equal(ids[-7:], want[0]) and bool(((w[-7:] - want[1]).abs() <= 2.0 ** -23 * want[1]).all())
    assert torch.equal(ids[-8], torch.arange(6, dtype=torch.int32, device=dev))


def test_sigmoid_scores_that_are_all_one(dev):
    """Nothing is added to the scores, so the logits decide, also where 64 bits hold a one; infinite ones are equal."""
    l = torch.zeros(2, 16)
    l[0, 3], l[0, 9], l[0, 12] = 50.0, 60.0, 55.0
    l[1, 7] = l[1, 5] = float("inf")
    ids, w = qg.moe_route(l.to(dev), 3, sigmoid=True, renormalize=False)
    assert ids.tolist() == [[9, 12, 3], [5, 7, 0]] and w.tolist() == [[1.0, 1.0, 1.0], [1.0, 1.0, 0.5]]


@pytest.mark.parametrize("best", [8, 9, 12, 16])
def test_many_tokens_whose_best_are_side_by_side(dev, best):
    """Up to 16 experts of one lane ahead of all others, equal or a hair apart from the eighth on."""
    torch.manual_seed(best)
    l = torch.randn(120, 256)
    l[:, 16:16 + best] = 6 + torch.rand(120, best)
    l[::3, 16:16 + best] = 6.0
    l[1::3, 16:16 + best] = 6 + 2.0 ** -21 * torch.randint(0, 3, (40, best)).float()
    for kw in (dict(), dict(sigmoid=True, bias=torch.zeros(256)), dict(sigmoid=True, bias=0.01 * torch.randn(256), groups=8, top_groups=4, best=2),
               dict(bias=torch.zeros(256))):
        check_many(dev, l, 8, **kw)
        check_many(dev, l.bfloat16(), 8, **kw)


@pytest.mark.parametrize("e,groups", [(64, 4), (128, 4), (256, 8)])
def test_many_tokens_with_whole_groups_masked(dev, e, groups):
    """Fewer experts left than picks, in one group: the rest of the picks are that group's, or the first group's beside it."""
    l = torch.full((40, e), -float("inf"))
    per = e // groups
    for i in range(40):
        at = (i % groups) * per
        l[i, at + i % 3:at + 2 + i % 5] = torch.randn(2 + i % 5 - i % 3)
    for top in (1, 2):
        for sigmoid in (False, True):
            for best in (1, 2):
                check_many(dev, l, 8, sigmoid=sigmoid, groups=groups, top_groups=top, best=best)
                check_many(dev, l.bfloat16(), 8, sigmoid=sigmoid, groups=groups, top_groups=top, best=best)
                check(dev, l.bfloat16(), 8, sigmoid, None, groups, top, best)
