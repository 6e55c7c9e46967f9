"""The decoder layer of examples/decoder_layer.py: prompts in chunks and decode
steps against the same layer in plain 64-bit form on the dequantized weights.

Tolerance: the layer's outputs pass through about eight roundings to bf16 (2^-9
of their values each on average), an 8-bit cache (half a step of 2 / 254 of a
block's largest value per key and value, averaged over the attended tokens) and
a softmax over scores that carry those errors; the relative error of the whole
output is held to 2 %, ten times a bf16 rounding."""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest
import torch

import layer_reference as ref

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
    """The values of a packed weight: its product with the identity."""
    rows = [qg.qgemm_w4a16(torch.eye(k, device="cuda")[i:i + 64].bfloat16(), packed, n, out_dtype=torch.float32)
            for i in range(0, k, 64)]
    return ref.f64(torch.cat(rows)).T


def rms(x):
    return x / np.sqrt(np.mean(x * x, -1, keepdims=True) + 1e-6)


class Plain:
    def __init__(self, layer, qg):
        h, d = layer.hidden, layer.d
        self.l, self.qkv = layer, dequantized(qg, layer.qkv, (layer.hq + 2 * layer.hkv) * d, h)
        self.o = dequantized(qg, layer.o, h, layer.hq * d)
        self.gu = [dequantized(qg, w, 2 * layer.inter, h) for w in layer.gate_up]
        self.dn = [dequantized(qg, w, h, layer.inter) for w in layer.down]
        self.k, self.v = [], []

    def feed(self, x):
        """Rows of one sequence after those fed before."""
        l, n0 = self.l, len(self.k)
        pos = np.arange(n0, n0 + x.shape[0])
        qkv = (rms(x) @ self.qkv.T).reshape(x.shape[0], -1, l.d)
        cs = ref.f64(l.cos_sin)
        q = ref.norm_rope(qkv[:, :l.hq], ref.f64(l.q_norm), cs, pos, 1e-6, False)
        k = ref.norm_rope(qkv[:, l.hq:l.hq + l.hkv], ref.f64(l.k_norm), cs, pos, 1e-6, False)
        self.k += list(k)
        self.v += list(qkv[:, l.hq + l.hkv:])
        a, _ = ref.attention(q, np.stack(self.k), np.stack(self.v), len(self.k), l.d ** -0.5, 0)
        x = x + a.reshape(x.shape[0], -1) @ self.o.T
        y, _ = ref.moe(rms(x), ref.f64(l.router), self.gu, self.dn, l.inter, l.top_k, True)
        return x + y


def test_prompts_and_decode_steps(example):
    qg = example.qg
    layer = example.DecoderLayer(3, 120, hidden=256, hq=4, hkv=2, d=64, experts=8, top_k=2, inter=256)
    g = torch.Generator().manual_seed(2)
    prompts = [torch.randn(n, 256, generator=g).bfloat16() for n in (70, 1, 33)]
    last = layer.prompts([p.cuda() for p in prompts])
    plain = Plain(layer, qg)
    state = []
    for b, p in enumerate(prompts):
        plain.k, plain.v = [], []
        want = plain.feed(ref.f64(p))[-1]
        state.append((plain.k, plain.v))
        got = ref.f64(last[b])
        assert np.linalg.norm(got - want) <= 0.02 * np.linalg.norm(want), np.linalg.norm(got - want) / np.linalg.norm(want)
    one = torch.ones(3, dtype=torch.int32, device="cuda")
    for step in range(3):
        x = torch.randn(3, 256, generator=g).bfloat16()
        y = layer.forward(x.cuda(), one, None, 1)
        for b in range(3):
            plain.k, plain.v = state[b]
            want = plain.feed(ref.f64(x[b:b + 1]))[0]
            got = ref.f64(y[b])
            assert np.linalg.norm(got - want) <= 0.02 * np.linalg.norm(want)
    assert layer.lens.tolist() == [73, 4, 36]


def test_graph_replays_equal_eager_steps(example):
    """The captured decode step, replayed, writes the same outputs and cache."""
    def start():
        layer = example.DecoderLayer(4, 100, hidden=512, hq=8, hkv=2, d=128, experts=16, top_k=4, inter=256)
        g = torch.Generator().manual_seed(3)
        x = layer.prompts([torch.randn(n, 512, generator=g).bfloat16().cuda() for n in (40, 17, 64, 5)])
        return layer, x, torch.ones(4, dtype=torch.int32, device="cuda")

    layer, x, one = start()
    outs = []
    for _ in range(5):
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
    for i in range(1, 5):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, outs[i]), i
    assert torch.equal(layer.codes, eager.codes) and torch.equal(layer.scales, eager.scales)
    assert torch.equal(layer.lens, eager.lens)
