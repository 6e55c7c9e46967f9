"""qg.verify_drafts against 64 bits: the same tokens.  The random numbers of these
tests stay away from the borders between tokens by more than the 64-bit running
sums are off (2^-53 a step), which the reference checks for itself by chance only:
a border is hit with probability 1e-11 a draw."""
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


def make(counts, v, dtype=F32, sure=False, cut=False, seed=0, agree=1.0):
    g = torch.Generator().manual_seed(seed + v + sum(counts))
    b, n = len(counts), sum(counts)
    cu = [0]
    for c in counts:
        cu.append(cu[-1] + c + 1)
    z = 2 * torch.randn(n + b, v, generator=g)
    row = [cu[i] + j for i, c in enumerate(counts) for j in range(c)]
    p, q = torch.softmax(z, 1), torch.softmax(z[row] + agree * torch.randn(n, v, generator=g), 1)
    if cut:
        p, q = (torch.where(t > 0.5 / v, t, 0.0) for t in (p, q))
    tokens = torch.multinomial(q, 1, generator=g)[:, 0] if n else torch.zeros(0, dtype=torch.int64)
    return dict(target=p.to(dtype), draft=None if sure else q.to(dtype), tokens=tokens.to(torch.int32), u=torch.rand(n, generator=g),
                u_next=torch.rand(b, generator=g), cu=torch.tensor(cu, dtype=torch.int32))


def run(dev, c, **kw):
    return qg.verify_drafts(*(None if c[n] is None else c[n].to(dev) for n in ("target", "draft", "tokens", "u", "u_next", "cu")), **kw)


def want(c):
    return ref.verify(ref.f64(c["target"]), None if c["draft"] is None else ref.f64(c["draft"]), c["tokens"].tolist(), ref.f64(c["u"]),
                      ref.f64(c["u_next"]), c["cu"].tolist())


def check(dev, c):
    accepted, following = run(dev, c)
    assert accepted.dtype == torch.int32 and following.dtype == torch.int32
    w = want(c)
    assert accepted.tolist() == w[0] and following.tolist() == w[1], (accepted.tolist(), w[0], following.tolist(), w[1])
    return w


@pytest.mark.parametrize("counts", [[0], [1], [3], [0, 0, 0], [2, 0, 5, 1, 0, 7], [70], [4] * 33], ids=lambda c: f"{len(c)}x{max(c)}")
@pytest.mark.parametrize("v", [1, 2, 63, 1000, 2048, 2049, 32000])
@pytest.mark.parametrize("dtype,sure,cut", [(F32, False, False), (BF16, False, True), (F32, True, True), (BF16, True, False)])
def test_against_64_bits(dev, counts, v, dtype, sure, cut):
    for seed in range(3):
        check(dev, make(counts, v, dtype, sure, cut, seed))


def test_large_and_odd_vocabularies(dev):
    for v in (131071, 262143, 300000):
        taken = check(dev, make([2, 0, 4], v))[0]
        assert len(taken) == 3


def test_all_accepted_and_all_rejected(dev):
    c = make([3, 4], 500)
    c["draft"] = c["target"][[0, 1, 2, 4, 5, 6, 7]].clone()
    assert check(dev, c)[0] == [3, 4]                  # u < 1 against p / q = 1
    c["u"].zero_()
    check(dev, c)
    c["target"].scatter_(1, torch.tensor([[c["tokens"][i]] for i in (0, 1, 2, 0, 3, 4, 5, 6, 0)]).long(), 0.0)
    assert check(dev, c)[0] == [0, 0]                  # p = 0 is never accepted, not even at u = 0


def test_no_token_left_over(dev):
    """p below q everywhere (rows that add up to less): the token comes from p."""
    c = make([1, 1], 300)
    c["draft"] = c["target"][[0, 2]].clone()
    c["target"] *= 0.5
    c["u"].fill_(0.75)
    assert check(dev, c)[0] == [0, 0]
    # one certain draft that holds all the target's probability, rejected by rounding alone: 0.999 < u
    p = torch.zeros(2, 10)
    p[:, 4] = 0.5
    c = dict(target=p, draft=None, tokens=torch.tensor([4], dtype=torch.int32), u=torch.tensor([0.75]), u_next=torch.tensor([0.3]),
             cu=torch.tensor([0, 2], dtype=torch.int32))
    assert check(dev, c) == ([0], [4])


@pytest.mark.parametrize("v", [7, 2048, 5000])
def test_borders_between_tokens(dev, v):
    """Equal shares that 64 bits add up exactly: u' on a border takes the token after it."""
    n = 1 << (v.bit_length() - 1)
    p = torch.zeros(9, v)
    p[:, v - n:] = 1.0 / n
    u = torch.tensor([0.0, 1 / n, 0.5, 0.5 - 2.0 ** -24, 1 - 1 / n, 1 - 2.0 ** -24, 0.25, 0.75, 0.25 + 1 / n])
    c = dict(target=p, draft=None, tokens=torch.zeros(0, dtype=torch.int32), u=torch.zeros(0), u_next=u, cu=torch.arange(10, dtype=torch.int32))
    w = check(dev, c)[1]
    assert w[0] == v - n and w[2] == v - n // 2 and w[3] == v - n // 2 - 1 and w[5] == v - 1


def test_tiny_shares_and_u_of_one(dev):
    """The first token with any share at u' = 0, the last one at u' of 1 (outside [0, 1), but not lost)."""
    p = torch.zeros(4, 6000)
    p[:, 100], p[:, 3000], p[:, 5900] = 1e-38, 1.0, 1e-38
    c = dict(target=p, draft=None, tokens=torch.zeros(0, dtype=torch.int32), u=torch.zeros(0), u_next=torch.tensor([0.0, 0.5, 1.0, 1.5]),
             cu=torch.arange(5, dtype=torch.int32))
    assert run(dev, c)[1].tolist() == [100, 3000, 5900, 5900]
    p *= 1e-6                                          # denormal numbers beside 1e-6
    assert run(dev, c | dict(target=p))[1].tolist()[1] == 3000
    p = torch.full((1, 5000), 1e-45)                   # a row of denormal numbers alone
    c = dict(target=p, draft=None, tokens=torch.zeros(0, dtype=torch.int32), u=torch.zeros(0), u_next=torch.tensor([0.5]),
             cu=torch.arange(2, dtype=torch.int32))
    assert run(dev, c)[1].tolist() == [2500]


def test_rows_that_cannot_be_drawn_from(dev):
    c = make([1, 1, 1, 1], 400)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    c["u"].fill_(0.999999)
    c["draft"].scatter_(1, c["tokens"].long()[:, None], 1.0)     # rejected, most likely
    c["target"][0] = 0.0
    c["target"][2, 7] = float("inf")
    c["target"][4, 9] = float("nan")
    accepted, following = run(dev, c, status=status)
    w = want(c)
    assert accepted.tolist() == w[0] and following.tolist() == w[1] and w[1][:2] == [-1, -1] and w[1][2] >= 0
    assert status.item() == qg.FLAG_NONFINITE
    status.zero_()
    run(dev, make([1, 1], 400), status=status)
    assert status.item() == 0


def test_tokens_and_offsets_outside_what_there_is(dev):
    c = make([2, 3, 1], 300)
    c["tokens"][0], c["tokens"][3], c["tokens"][5] = 300, -1, 2 ** 31 - 1
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    accepted, following = run(dev, c, status=status)
    w = want(c)
    assert accepted.tolist() == w[0] and following.tolist() == w[1] and status.item() == qg.FLAG_INDEX
    sure = c | dict(draft=None)
    accepted, following = run(dev, sure)
    assert accepted.tolist() == want(sure)[0] and following.tolist() == want(sure)[1]
    # the right offsets: 0 3 7 9
    good = make([2, 3, 1], 300)
    for cu in ([0, 3, 2, 9], [0, 3, 700, 9], [0, -5, 7, 9], [4, 3, 7, 9], [0, 3, 3, 9], [2 ** 31 - 1, 3, 7, 9]):
        status.zero_()
        lens = torch.full((3,), 50, dtype=torch.int32, device=dev)
        c = good | dict(cu=torch.tensor(cu, dtype=torch.int32))
        accepted, following = run(dev, c, status=status, lens=lens)
        assert status.item() & qg.FLAG_INDEX and bool((following < 300).all()) and bool((following >= -1).all())
        assert bool(((accepted == 0) | (following >= 0)).all())


def test_lengths_streams_and_graphs(dev):
    c = {k: t.to(dev) for k, t in make([4, 0, 6, 3, 2], 33000).items()}
    lens = torch.tensor([100, 20, 300, 50, 7], dtype=torch.int32, device=dev)
    before = lens.clone()
    accepted, following = qg.verify_drafts(*c.values(), lens=lens)
    n = c["cu"][1:] - c["cu"][:-1] - 1
    assert torch.equal(lens, before - (n - accepted))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = qg.verify_drafts(*c.values())
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other[0], accepted) and torch.equal(other[1], following)
    ws = torch.empty(qg.verify_drafts_workspace_bytes(c["target"].shape[0], 5, 33000), dtype=torch.uint8, device=dev)
    out = (torch.zeros_like(accepted), torch.zeros_like(accepted))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qg.verify_drafts(*c.values(), out=out, workspace=ws)
    for k in range(4):
        c["u"].uniform_()
        c["u_next"].uniform_()
        graph.replay()
        torch.cuda.synchronize()
        want_ = qg.verify_drafts(*c.values())
        assert torch.equal(out[0], want_[0]) and torch.equal(out[1], want_[1]), k
    e = qg.verify_drafts(c["target"][:0], c["draft"][:0], c["tokens"][:0], c["u"][:0], c["u_next"][:0], c["cu"][:1])
    assert e[0].shape == (0,) and e[1].shape == (0,)


def test_draws_follow_the_target(dev):
    """What is emitted at a place is distributed as the target, whatever the draft: the first tokens of 20000 sequences
    with one draft each, compared with the target's probabilities (10 tokens; the deviation of a count is below
    sqrt(20000) / 2 = 71, six of which are allowed)."""
    b, v = 20000, 10
    torch.manual_seed(3)
    p, q = torch.softmax(torch.randn(v), 0), torch.softmax(torch.randn(v), 0)
    tokens = torch.multinomial(q, b, replacement=True).to(torch.int32)
    c = dict(target=p.repeat(2 * b, 1), draft=q.repeat(b, 1), tokens=tokens, u=torch.rand(b), u_next=torch.rand(b),
             cu=2 * torch.arange(b + 1, dtype=torch.int32))
    accepted, following = run(dev, c)
    first = torch.where(accepted.cpu() > 0, tokens, following.cpu())
    count = torch.bincount(first.long(), minlength=v)
    assert float((count - b * p).abs().max()) <= 6 * 71


# ---- vocabularies whose sums are a launch of their own, and wide batches ----------------

@pytest.mark.parametrize("v", [40008, 50001, 600001])       # whole rows of 16 bytes; odd; pieces of more than 512
@pytest.mark.parametrize("dtype,sure,cut", [(F32, False, False), (BF16, False, True), (F32, True, True), (BF16, True, False)])
def test_wide_vocabularies(dev, v, dtype, sure, cut):
    check(dev, make([2, 0, 3, 1, 0], v, dtype, sure, cut))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_wide_batches_of_wide_vocabularies(dev, dtype):
    """130 sequences of 60001: one workgroup each; the same outcome as 13 at a time."""
    g = torch.Generator(device=dev).manual_seed(1)
    b, v = 130, 60001
    p = torch.softmax(2 * torch.randn(2 * b, v, generator=g, device=dev), 1).to(dtype)
    q = torch.softmax(2 * torch.randn(b, v, generator=g, device=dev), 1).to(dtype)
    tokens = torch.randint(0, v, (b,), generator=g, device=dev, dtype=torch.int32)
    u, u_next = torch.rand(b, generator=g, device=dev), torch.rand(b, generator=g, device=dev)
    got = qg.verify_drafts(p, q, tokens, u, u_next, 2 * torch.arange(b + 1, device=dev, dtype=torch.int32))
    cu = 2 * torch.arange(14, device=dev, dtype=torch.int32)
    for i in range(0, b, 13):
        s = slice(i, i + 13)
        part = qg.verify_drafts(p[2 * i:2 * i + 26], q[s], tokens[s], u[s], u_next[s], cu)
        assert torch.equal(got[0][s], part[0]) and torch.equal(got[1][s], part[1]), i


def test_wide_vocabularies_at_their_edges(dev):
    """Nothing left over, nothing to draw from, tokens and offsets outside, lengths and flags: as for small ones."""
    v = 50000
    c = make([1, 1], v)
    c["draft"] = c["target"][[0, 2]].clone()
    c["target"] *= 0.5
    c["u"].fill_(0.75)
    assert check(dev, c)[0] == [0, 0]
    c = make([1, 1, 1, 1], v)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    c["u"].fill_(0.999999)
    c["draft"].scatter_(1, c["tokens"].long()[:, None], 1.0)
    c["target"][0] = 0.0
    c["target"][2, 7] = float("inf")
    c["target"][4, 9] = float("nan")
    accepted, following = run(dev, c, status=status)
    w = want(c)
    assert accepted.tolist() == w[0] and following.tolist() == w[1] and w[1][:2] == [-1, -1] and w[1][2] >= 0
    assert status.item() == qg.FLAG_NONFINITE
    c = make([2, 3, 1], v)
    c["tokens"][0], c["tokens"][3] = v, -1
    status.zero_()
    accepted, following = run(dev, c, status=status)
    assert accepted.tolist() == want(c)[0] and following.tolist() == want(c)[1] and status.item() == qg.FLAG_INDEX
    status.zero_()
    lens = torch.full((3,), 50, dtype=torch.int32, device=dev)
    accepted, following = run(dev, make([2, 3, 1], v) | dict(cu=torch.tensor([0, 3, 2, 9], dtype=torch.int32)), status=status, lens=lens)
    assert status.item() & qg.FLAG_INDEX and accepted[1].item() == 0 and following[1].item() == -1 and lens[1].item() == 50


def test_captured_graphs_of_wide_vocabularies_share_a_workspace(dev):
    first, second = ({k: t.to(dev) for k, t in make([4, 0, 6, 3, 2], 50001, seed=s).items()} for s in (0, 1))
    ws = torch.empty(qg.verify_drafts_workspace_bytes(first["target"].shape[0], 5, 50001), dtype=torch.uint8, device=dev)
    assert ws.numel() > 0
    graphs, outs = [], []
    for c in (first, second):
        outs.append((torch.zeros(5, dtype=torch.int32, device=dev), torch.zeros(5, dtype=torch.int32, device=dev)))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            qg.verify_drafts(*c.values(), out=outs[-1], workspace=ws)
    for k in range(3):
        for c in (first, second):
            c["u"].uniform_()
            c["u_next"].uniform_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for c, out in zip((first, second), outs):
            want_ = qg.verify_drafts(*c.values())
            assert torch.equal(out[0], want_[0]) and torch.equal(out[1], want_[1]), k


def test_rows_past_two_to_the_31_elements(dev):
    v, b = 131072, 16385                       # 2^31 elements and a row, 4 GiB
    target = torch.zeros(b, v, dtype=BF16, device=dev)
    hit = torch.arange(b, device=dev) * 7919 % v
    target.scatter_(1, hit[:, None], 1.0)
    none = torch.zeros(0, device=dev)
    accepted, following = qg.verify_drafts(target, None, none.to(torch.int32), none, torch.rand(b, device=dev),
                                           torch.arange(b + 1, dtype=torch.int32, device=dev))
    assert not bool(accepted.any()) and torch.equal(following.long(), hit)


@pytest.mark.parametrize("v", [300, 50000])        # one launch; the sums in one of their own
@pytest.mark.parametrize("cu,bad", [([0, 3, 7, 10], 2), ([0, 3, 7, 700], 2), ([0, 3, 7, 2 ** 31 - 1], 2), ([-1, 3, 7, 9], 0), ([-5, 3, 7, 9], 0),
                                    ([-2 ** 31, 3, 7, 9], 0), ([0, 3, 7, -1], 2)])
def test_offsets_that_reach_past_the_rows(dev, v, cu, bad):
    """The one sequence whose rows are not all there accepts nothing and draws nothing, its length stays, and the flag says so; the
    others are as they are with the right offsets, 0 3 7 9."""
    c = make([2, 3, 1], v)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    lens = torch.full((3,), 50, dtype=torch.int32, device=dev)
    right = [t.tolist() for t in run(dev, c, lens=lens, status=status)]
    want_lens = lens.tolist()
    assert status.item() == 0
    lens.fill_(50)
    accepted, following = run(dev, c | dict(cu=torch.tensor(cu, dtype=torch.int32)), lens=lens, status=status)
    right[0][bad], right[1][bad], want_lens[bad] = 0, -1, 50
    assert accepted.tolist() == right[0] and following.tolist() == right[1] and lens.tolist() == want_lens
    assert status.item() == qg.FLAG_INDEX
