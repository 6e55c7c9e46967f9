"""qg_moe_w4a16 against the layer in 64 bits on the oracle's own quantization.

Tolerance per output, with B = sum over picks of p |W2| |silu(g) u| in 64 bits:
the hidden activation is rounded to bf16 (2^-8 of each term at most), the fp32
sums and the routing weights add less than 2^-11 of the terms at these sizes
(sums of at most 2048 products; a cancelled gate or up sum enters B with its own
terms' rounding, covered by 2^-16 of the largest row of |W| |x|), so
|err| <= (2^-8 + 2^-10) B + 2^-16 max B, plus half a bf16 unit for bf16 output."""
from __future__ import annotations

import functools

import numpy as np
import pytest
import torch

import layer_reference as ref
import oracle
import synthetic_inputs as si

import gemm_decode_qgemm_amd as qg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


@functools.lru_cache(maxsize=4)
def experts(e, h, inter, seed):
    """(packed gate_up, packed down, their values in 64 bits)."""
    g = torch.Generator().manual_seed(seed)
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


def check(y, want, bound):
    got = ref.f64(y)
    assert np.isfinite(got).all()
    tol = bound * (2.0 ** -8 + 2.0 ** -10) + bound.max(-1, keepdims=True) * 2.0 ** -16
    if y.dtype == torch.bfloat16:
        tol = tol + ref.half_ulp_bf16(np.abs(want) + tol)
    err = np.abs(got - want)
    assert (err <= tol).all(), float((err / tol).max())


def case(dev, t, e, k, h, inter, renorm, seed, dtypes=(torch.float32, torch.bfloat16), x=None, router=None):
    gu, dn, gu_v, dn_v = experts(e, h, inter, e + h + inter)
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(t, h, generator=g).bfloat16() if x is None else x
    router = (torch.randn(e, h, generator=g) * 2 * h ** -0.5).bfloat16() if router is None else router
    want, bound = ref.moe(ref.f64(x), ref.f64(router), gu_v, dn_v, inter, k, renorm)
    args = (x.to(dev), router.to(dev), gu.to(dev), dn.to(dev), inter, k)
    for dt in dtypes:
        y = qg.moe_w4a16(*args, renormalize=renorm, out_dtype=dt)
        assert y.shape == (t, h) and y.dtype == dt
        check(y, want, bound)
    return args, want


@pytest.mark.parametrize("t", [1, 2, 3, 4, 5, 16, 17, 33, 64])
@pytest.mark.parametrize("e,k,h,inter,renorm", [(8, 2, 512, 256, True), (16, 4, 256, 768, False)])
def test_every_token_count(dev, t, e, k, h, inter, renorm):
    case(dev, t, e, k, h, inter, renorm, 100 * t + e)


@pytest.mark.parametrize("t,e,k,h,inter", [
    (1, 1, 1, 256, 256), (7, 1, 1, 256, 256), (64, 2, 2, 256, 256), (3, 5, 5, 256, 512), (2, 64, 6, 256, 256), (9, 70, 3, 256, 256),
    (20, 128, 8, 256, 256), (1, 160, 32, 256, 256), (30, 3, 1, 2048, 1280)])
@pytest.mark.parametrize("renorm", [True, False])
def test_expert_counts_and_sizes(dev, t, e, k, h, inter, renorm):
    case(dev, t, e, k, h, inter, renorm, t + e + k, (torch.bfloat16,))


def test_all_tokens_on_the_same_experts(dev):
    """64 tokens on two experts of eight: units of 64 tokens next to empty ones."""
    e, h = 8, 512
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(64, h, generator=g) * 0.2 + 1).bfloat16()
    router = torch.zeros(e, h).bfloat16()
    router[5], router[2] = 0.02, 0.01
    case(dev, 64, e, 2, h, 256, True, 0, x=x, router=router)
    case(dev, 3, e, 2, h, 256, False, 0, x=x[:3], router=router)
    for t in (5, 6, 8, 9):
        case(dev, t, e, 2, h, 256, False, 0, x=x[:t], router=router)


@pytest.mark.parametrize("t,k,same", [(17, 3, False), (64, 4, False), (64, 2, True), (60, 2, True), (5, 10, False)])
def test_many_row_blocks_and_experts(dev, t, k, same):
    """50 experts with 8 pairs of row blocks each in the down product: more than
    the workgroups that halves of K are for; 64 tokens of one expert among them."""
    e, h, inter = 50, 1024, 256
    g = torch.Generator().manual_seed(t)
    x = (torch.randn(t, h, generator=g) * 0.2 + 1).bfloat16() if same else None
    router = None
    if same:
        router = torch.zeros(e, h).bfloat16()
        router[31], router[7] = 0.02, 0.01
    case(dev, t, e, k, h, inter, True, t, x=x, router=router)


@pytest.mark.parametrize("t,k", [(2, 30), (3, 17), (4, 16), (4, 20), (5, 10), (7, 11), (8, 7), (8, 32)])
def test_few_tokens_on_many_workgroups(dev, t, k):
    """Up to 8 tokens with more gate and up workgroups than run at once."""
    case(dev, t, 50, k, 256, 768, t & 1 == 0, t + k, (torch.bfloat16,))


@pytest.mark.parametrize("e,k", [(512, 32), (300, 5), (65, 3)])
@pytest.mark.parametrize("t", [2, 8, 63])
def test_tokens_of_many_experts(dev, t, e, k):
    """Routing alone: every expert one tile, its weights those of expert e % 8."""
    h = inter = 256
    gu, dn, gu_v, dn_v = experts(8, h, inter, 77)
    which = [i % 8 for i in range(e)]
    g = torch.Generator().manual_seed(e + t)
    x = torch.randn(t, h, generator=g).bfloat16()
    router = (torch.randn(e, h, generator=g) * 2 * h ** -0.5).bfloat16()
    want, bound = ref.moe(ref.f64(x), ref.f64(router), [gu_v[i] for i in which], [dn_v[i] for i in which], inter, k, True)
    y = qg.moe_w4a16(x.to(dev), router.to(dev), gu[which].to(dev), dn[which].to(dev), inter, k, out_dtype=torch.float32)
    check(y, want, bound)


def test_ties_go_to_the_lowest_index(dev):
    """Equal logits everywhere: the first k experts, with equal weights."""
    e, h = 16, 256
    x = torch.randn(6, h, generator=torch.Generator().manual_seed(5)).bfloat16()
    router = torch.zeros(e, h).bfloat16()
    for t in (1, 2, 6):
        case(dev, t, e, 4, h, 768, True, 0, x=x[:t], router=router)
    router[3:9] = torch.randn(h, generator=torch.Generator().manual_seed(6)).bfloat16() * 0.05   # six equal rows
    case(dev, 6, e, 4, h, 768, False, 0, x=x, router=router)


def test_wide_logits_and_zero_tokens(dev):
    e, h = 8, 512
    g = torch.Generator().manual_seed(7)
    x = torch.randn(5, h, generator=g).bfloat16()
    x[2] = 0.0
    router = (torch.randn(e, h, generator=g) * 30).bfloat16()      # one expert has all the weight
    case(dev, 5, e, 2, h, 256, True, 0, x=x, router=router)
    case(dev, 5, e, 2, h, 256, False, 0, x=x, router=router)


def test_a_nan_token_leaves_the_others_alone(dev):
    args, want = case(dev, 20, 8, 2, 512, 256, True, 11, (torch.float32,))
    clean = qg.moe_w4a16(*args, out_dtype=torch.float32)
    x = args[0].clone()
    x[7, 100] = float("nan")
    y = qg.moe_w4a16(x, *args[1:], out_dtype=torch.float32)
    assert y[7].isnan().all()
    keep = [t for t in range(20) if t != 7]
    assert not y[keep].isnan().any()
    assert torch.allclose(y[keep], clean[keep], rtol=1e-4, atol=1e-5)


def test_repeats_streams_graphs_and_stale_workspace(dev):
    for t in (1, 3, 17, 40):
        args, _ = case(dev, t, 16, 4, 256, 768, False, 13 + t, (torch.bfloat16,))
        want = qg.moe_w4a16(*args, renormalize=False)
        ws = torch.full((qg.moe_w4a16_workspace_bytes(t, 256, 16, 768, 4),), 255, dtype=torch.uint8, device=dev)
        out = torch.empty_like(want)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            qg.moe_w4a16(*args, renormalize=False, out=out, workspace=ws)
        s.synchronize()
        assert torch.equal(out, want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qg.moe_w4a16(*args, renormalize=False, out=out, workspace=ws)
        for _ in range(3):
            out.fill_(5.0)
            ws.fill_(255)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)


def test_packed_weights_of_the_library_and_the_linear_layer(dev):
    """One expert with weight one is two qgemm_w4a16 calls with silu between."""
    h, inter, t = 512, 256, 6
    torch.manual_seed(17)
    w1, w2 = (torch.randn(2 * inter, h) * 0.05).bfloat16().to(dev), (torch.randn(h, inter) * 0.05).bfloat16().to(dev)
    gu, dn = qg.quantize_int4_g32(w1), qg.quantize_int4_g32(w2)
    x = torch.randn(t, h).bfloat16().to(dev)
    y = qg.moe_w4a16(x, torch.zeros(1, h, dtype=torch.bfloat16, device=dev), gu[None], dn[None], inter, 1, out_dtype=torch.float32)
    z = qg.qgemm_w4a16(x, gu, 2 * inter, out_dtype=torch.float32)
    a = (torch.nn.functional.silu(z[:, :inter]) * z[:, inter:]).bfloat16()
    want = qg.qgemm_w4a16(a, dn, h, out_dtype=torch.float32)
    # a hidden value may round the other way where silu differs in its last bits: 2^-8 of one term in 256
    assert (y - want).abs().max() <= 2.0 ** -8 * want.abs().max()


def test_experts_past_4_gib(dev):
    """Offsets of the last experts need 64 bits."""
    e, h, inter = 512, 2048, 4096
    n1, n2 = qg.int4_packed_bytes(2 * inter, h), qg.int4_packed_bytes(h, inter)
    assert (e - 1) * n1 > 1 << 32
    gu = torch.zeros(e, n1, dtype=torch.uint8, device=dev)
    dn = torch.zeros(e, n2, dtype=torch.uint8, device=dev)
    torch.manual_seed(19)
    one = [qg.quantize_int4_g32((torch.randn(n, k, device=dev) * 0.02).bfloat16()) for n, k in ((2 * inter, h), (h, inter))]
    gu[-1], dn[-1] = one
    x = torch.randn(2, h, device=dev).bfloat16()
    router = torch.zeros(e, h, dtype=torch.bfloat16, device=dev)
    router[-1] = x[0] * 0.01
    y = qg.moe_w4a16(x[:1], router, gu, dn, inter, 1)
    z = qg.moe_w4a16(x[:1], router[-1:], one[0][None], one[1][None], inter, 1)
    assert torch.equal(y, z) and y.any()


def one_term_weights(n, k, rows, cols, seed):
    """A packed n x k weight whose row r has one value that is not zero, at cols[r] (rows alone), and its values
    in 64 bits.  Codes of 8 with zero points of 8 are zeros; the others are 4 to 7 steps away from it."""
    g = np.random.default_rng(seed)
    codes, zeros = np.full((n, k), 8, np.uint8), np.full((n, k // 32), 8, np.uint8)
    scales = (0.1 + 0.2 * g.random((n, k // 32))).astype(np.float16)
    codes[rows, cols] = 8 + g.choice([-7, -6, -5, -4, 4, 5, 6, 7], len(rows))
    values = (codes.astype(np.float64) - 8) * np.repeat(scales.astype(np.float64), 32, 1)
    return torch.from_numpy(oracle.pack_int4(codes, scales.view(np.uint16), zeros)), values


def bf16(a):
    return torch.from_numpy(np.asarray(a)).float().bfloat16().double().numpy()


@pytest.mark.parametrize("t", [1, 2, 3, 4])
@pytest.mark.parametrize("e,k", [(2, 1), (2, 2), (5, 3)])
def test_up_to_four_tokens_keep_the_hidden_values_as_two_bf16(dev, t, e, k):
    """Weights with one term a row and one hidden value an expert, so that no sum rounds and what is left is
    the rounding of the hidden value to the sum of two bf16 (2^-18 of it), silu in binary32 (its
    exponential's argument of up to 16 carries 2^-20) and the last product (2^-24 of 272 / 4 of the term, from
    the bias of 128 + 8 on a code at least 4 away from it): below 2^-15 of the terms in all.  The same
    hidden values as one bf16 are outside it."""
    h, inter, hot = 256, 256, 7 + 32 * ((t + e) % 8)
    ks = 32 * np.arange(8) + 5                        # channels of x that are not zero
    g = np.random.default_rng(10 * t + e)
    gu, dn, gu_v, dn_v = [], [], [], []
    for i in range(e):
        w, v = one_term_weights(2 * inter, h, np.array([hot, inter + hot]), g.choice(ks, 2), 31 * i + e)
        gu.append(w), gu_v.append(v)
        w, v = one_term_weights(h, inter, np.arange(h), np.full(h, hot), 37 * i + e)
        dn.append(w), dn_v.append(v)
    x = torch.zeros(t, h, dtype=torch.bfloat16)
    x[:, ks] = torch.from_numpy(1.5 * g.standard_normal((t, 8))).clamp(-4, 4).bfloat16()
    router = torch.zeros(e, h, dtype=torch.bfloat16)
    want, bound = ref.moe(ref.f64(x), ref.f64(router), gu_v, dn_v, inter, k, True)
    y = qg.moe_w4a16(x.to(dev), router.to(dev), torch.stack(gu).to(dev), torch.stack(dn).to(dev), inter, k, out_dtype=torch.float32)
    tol = bound * 2.0 ** -15 + 1e-30
    assert (np.abs(ref.f64(y) - want) <= tol).all(), float((np.abs(ref.f64(y) - want) / tol).max())
    once = np.zeros_like(want)                        # the first k experts, equal weights
    for i in range(k):
        gate, up = ref.f64(x) @ gu_v[i][:inter].T, ref.f64(x) @ gu_v[i][inter:].T
        once += bf16(gate / (1 + np.exp(-gate)) * up) @ dn_v[i].T / k
    assert (np.abs(once - want) > tol).any()
