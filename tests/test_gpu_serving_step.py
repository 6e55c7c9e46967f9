"""The serving-step operators together, as examples/decoder_layer.py runs them: a layer
with adapters, grouped experts and 8-bit rows against the same layer in plain 64-bit
form on the dequantized weights, and steps that verify drafted tokens.

Tolerance of the layer: as for the layer without them, about eight roundings to
bf16, an 8-bit cache and a softmax over scores that carry those errors: 2 % of the
whole output; 8-bit rows (half a step of 1 / 127 of a group's largest channel, about
0.4 % of each channel's size, averaged over a product's terms) leave it there."""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest
import torch

import layer_reference as lref
import serving_reference as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import decoder_layer
    finally:
        sys.path.pop(0)
    return decoder_layer


def dequantized(qg, packed, n, k):
    rows = [qg.qgemm_w4a16(torch.eye(k, device="cuda")[i:i + 64].bfloat16(), packed, n, out_dtype=torch.float32)
            for i in range(0, k, 64)]
    return ref.f64(torch.cat(rows)).T


class Plain:
    """One sequence of a layer in 64 bits."""

    def __init__(self, layer, qg, sequence):
        h, d = layer.hidden, layer.d
        self.l, self.qkv = layer, dequantized(qg, layer.qkv, (layer.hq + 2 * layer.hkv) * d, h)
        self.o = dequantized(qg, layer.o, h, layer.hq * d)
        self.gu = [dequantized(qg, w, 2 * layer.inter, h) for w in layer.gate_up]
        self.dn = [dequantized(qg, w, h, layer.inter) for w in layer.down]
        self.id = -1 if layer.ids is None else int(layer.ids[sequence])
        self.k, self.v = [], []

    def adapted(self, name, y, x):
        if self.id < 0:
            return y
        a, b = (ref.f64(t) for t in self.l.lora[name])
        return ref.lora(y, x, a, b, [self.id] * len(x), ref.f64(self.l.lora_scales))

    def experts(self, x):
        l = self.l
        ids, w = ref.route(x @ ref.f64(l.router).T, l.top_k, True, ref.f64(l.bias), l.groups, l.groups // 2, 2, True, 1.0)
        y = np.zeros_like(x)
        for t in range(len(x)):
            for e, p in zip(ids[t], w[t]):
                gu = self.gu[e] @ x[t]
                g, u = gu[:l.inter], gu[l.inter:]
                y[t] += p * (self.dn[e] @ (g / (1 + np.exp(-g)) * u))
        return y

    def feed(self, x):
        l, n0 = self.l, len(self.k)
        pos, cs = np.arange(n0, n0 + len(x)), ref.f64(l.cos_sin)
        normed = ref.rms_norm(x, None, None, 1e-6)[0]
        qkv = self.adapted("qkv", normed @ self.qkv.T, normed).reshape(len(x), -1, l.d)
        q = lref.norm_rope(qkv[:, :l.hq], ref.f64(l.q_norm), cs, pos, 1e-6, False)
        k = lref.norm_rope(qkv[:, l.hq:l.hq + l.hkv], ref.f64(l.k_norm), cs, pos, 1e-6, False)
        self.k += list(k)
        self.v += list(qkv[:, l.hq + l.hkv:])
        a, _ = lref.attention(q, np.stack(self.k), np.stack(self.v), len(self.k), l.d ** -0.5, 0)
        a = a.reshape(len(x), -1)
        normed, x = ref.rms_norm(self.adapted("o", a @ self.o.T, a), x, None, 1e-6)
        return x + self.experts(normed)


@pytest.mark.parametrize("act8", [False, True])
def test_adapters_grouped_experts_and_8_bit_rows(example, act8):
    qg = example.qg
    layer = example.DecoderLayer(4, 120, hidden=256, hq=4, hkv=2, d=64, experts=8, top_k=2, inter=256, adapters=2, groups=4,
                                 act8=act8)
    assert layer.ids.tolist() == [-1, 0, 1, -1]
    g = torch.Generator().manual_seed(5)
    prompts = [torch.randn(n, 256, generator=g).bfloat16() for n in (40, 1, 33, 7)]
    last = layer.prompts([p.cuda() for p in prompts])
    plain = [Plain(layer, qg, b) for b in range(4)]
    for b, p in enumerate(prompts):
        want = plain[b].feed(ref.f64(p))[-1]
        got = ref.f64(last[b])
        assert np.linalg.norm(got - want) <= 0.02 * np.linalg.norm(want), (b, np.linalg.norm(got - want) / np.linalg.norm(want))
    x = torch.randn(12, 256, generator=g).bfloat16()       # three rows a sequence, as a verification's
    y = layer.forward(x.cuda(), torch.full((4,), 3, dtype=torch.int32, device="cuda"), None, 3)
    for b in range(4):
        want = plain[b].feed(ref.f64(x[3 * b:3 * b + 3]))
        got = ref.f64(y[3 * b:3 * b + 3])
        assert np.linalg.norm(got - want) <= 0.02 * np.linalg.norm(want)


def test_verified_steps_keep_the_accepted_tokens(example):
    """Every step's outcome is the reference's on the same probabilities, and lengths lose what was rejected."""
    qg = example.qg
    layer = example.DecoderLayer(6, 200, hidden=256, hq=4, hkv=2, d=64, experts=8, top_k=2, inter=256, adapters=2)
    layer.prompts([torch.randn(n, 256).bfloat16().cuda() for n in (9, 3, 30, 1, 17, 5)])
    s = example.Speculator(layer, vocabulary=512)
    seen = {}
    probabilities, verify = s.probabilities, qg.verify_drafts
    s.probabilities = lambda y: seen.setdefault("p", probabilities(y).clone())

    def spied(p, q, tokens, u, u_next, cu, lens=None):
        seen.update(q=q, tokens=tokens, u=u, u_next=u_next, cu=cu)
        return verify(p, q, tokens, u, u_next, cu, lens=lens)

    example.qg.verify_drafts = spied
    try:
        last = torch.zeros(6, dtype=torch.int32, device="cuda")
        for _ in range(5):
            seen.clear()
            before = layer.lens.clone()
            accepted, last = s.step(last, 4)
            want = ref.verify(ref.f64(seen["p"]), ref.f64(seen["q"]), seen["tokens"].tolist(), ref.f64(seen["u"]),
                              ref.f64(seen["u_next"]), seen["cu"].tolist())
            assert accepted.tolist() == want[0] and last.tolist() == want[1]
            assert torch.equal(layer.lens, before + 1 + accepted)
    finally:
        example.qg.verify_drafts = verify


def test_a_captured_step_with_all_of_them(example):
    """Norm in 8 bits, adapters, choice of experts and the experts, captured once: replays equal eager steps."""
    def start():
        layer = example.DecoderLayer(5, 100, hidden=512, hq=8, hkv=2, d=128, experts=16, top_k=4, inter=256, adapters=3, groups=4,
                                     act8=True)
        g = torch.Generator().manual_seed(3)
        x = layer.prompts([torch.randn(n, 512, generator=g).bfloat16().cuda() for n in (40, 17, 64, 5, 20)])
        return layer, x, torch.ones(5, dtype=torch.int32, device="cuda")

    layer, x, one = start()
    outs = []
    for _ in range(4):
        x.copy_(example.rms(layer.forward(x, one, None, 1)))
        outs.append(x.clone())
    eager = layer
    layer, x, one = start()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x.copy_(example.rms(layer.forward(x, one, None, 1)))
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(x, outs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.copy_(example.rms(layer.forward(x, one, None, 1)))
    for i in range(1, 4):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, outs[i]), i
    assert torch.equal(layer.codes, eager.codes) and torch.equal(layer.lens, eager.lens)


def small_layer(example):
    """Blocks that are empty, partly held and full, and one whose next tokens lie in two pages."""
    layer = example.DecoderLayer(6, 200, hidden=256, hq=4, hkv=2, d=64, experts=8, top_k=2, inter=256)
    g = torch.Generator().manual_seed(11)
    layer.prompts([torch.randn(n, 256, generator=g).bfloat16().cuda() for n in (9, 3, 30, 16, 17, 61)])
    return layer


def state_and_next(example, layer):
    """Lengths, the cache's tokens as they are read back, and the same after a further token, with its output."""
    def held():
        return example.qg.kv8_read(layer.codes, layer.scales, layer.table, layer.lens, layer.max_len, out_dtype=torch.float32)

    x = torch.randn(6, 256, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    return [layer.lens.clone(), *held(), layer.forward(x, torch.ones_like(layer.lens), None, 1), *held()]


@pytest.mark.parametrize("infinite", [False, True])
def test_rejected_drafts_leave_nothing_in_the_cache(example, monkeypatch, infinite):
    """Steps with the same last tokens whose drafts, other ones each, are all rejected: the same cache, and the same output of
    the next token."""
    def rejected(p, q, tokens, u, u_next, cu, lens=None):
        drafts.append(tokens.clone())
        lens -= cu[1:] - cu[:-1] - 1
        return torch.zeros_like(lens), torch.zeros_like(lens)

    drafts, seen = [], []
    monkeypatch.setattr(example.qg, "verify_drafts", rejected)
    for seed in (1, 2):
        layer = small_layer(example)
        s = example.Speculator(layer, vocabulary=512)
        s.g.manual_seed(seed)
        if infinite and seed == 2:
            s.embedding[1:, 5] = float("inf")      # all tokens but the last ones
        s.step(torch.zeros(6, dtype=torch.int32, device="cuda"), 4)
        seen.append(state_and_next(example, layer))
    assert not torch.equal(*drafts) and seen[0][0].tolist() == [10, 4, 31, 17, 18, 62]
    assert all(torch.equal(a, b) for a, b in zip(*seen)) and bool(seen[1][3].isfinite().all())


@pytest.mark.parametrize("rest", [1.0, 100.0, float("inf")])
def test_the_cache_keeps_the_accepted_rows_alone(example, rest):
    """Two layers whose steps agree in the accepted rows, from the last token alone to all, and not in the others."""
    kept = torch.tensor([1, 2, 3, 4, 5, 4], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(4)
    x = torch.randn(6, 5, 256, generator=g).bfloat16().cuda()
    gone = torch.arange(5, device="cuda") >= kept[:, None]
    seen = []
    for size in (1.0, rest):
        layer = small_layer(example)
        x[gone] = torch.randn(int(gone.sum()), 256, generator=g).bfloat16().cuda()
        x[..., 7] = torch.where(gone, size, x[..., 7])
        layer.forward(x.view(30, 256), torch.full_like(layer.lens, 5), None, 5, drafted=True)
        layer.lens -= 5 - kept
        layer.keep_only(kept)
        seen.append(state_and_next(example, layer))
    assert seen[0][0].tolist() == [10, 5, 33, 20, 22, 65]
    assert all(torch.equal(a, b) for a, b in zip(*seen)) and bool(seen[1][3].isfinite().all())


@pytest.mark.parametrize("args", [["--drafts", "15", "--batch", "4"], ["--batch", "3"], ["--batch", "3", "--graph"]], ids=lambda a: a[0][2:] + a[-1][2:])
def test_the_longest_sequences_have_room(example, monkeypatch, capsys, args):
    """The program with every draft accepted: no token past the table of positions or the pages, so outputs are finite."""
    layers, outs = [], []

    class Layer(example.DecoderLayer):
        def __init__(self, *a, **kw):
            super().__init__(*a, **kw)
            layers.append(self)

        def forward(self, *a, **kw):
            outs.append(super().forward(*a, **kw))
            return outs[-1]

    def accepted(p, q, tokens, u, u_next, cu, lens=None):
        return cu[1:] - cu[:-1] - 1, torch.zeros_like(lens)

    monkeypatch.setattr(example, "DecoderLayer", Layer)
    monkeypatch.setattr(example.qg, "verify_drafts", accepted)
    monkeypatch.setattr(sys, "argv", ["decoder_layer.py", "--prompt", "5", "--steps", "2", *args])
    example.main()
    assert "us a step" in capsys.readouterr().out
    layer, = layers
    assert int(layer.lens.max()) <= layer.max_len == layer.cos_sin.shape[0] <= layer.table.shape[1] * example.qg.KV8_PAGE
    assert all(bool(y.isfinite().all()) for y in outs)
