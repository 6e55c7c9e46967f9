"""One decoder layer of quantized linears, from prompt to decode.

    python examples/decoder_layer.py [--batch 8] [--prompt 100] [--steps 16] [--graph]

Every step runs on this library: the INT4 linears around attention
(qgemm_w4a16), the norm and rotation of query and key heads (qk_norm_rope), the
8-bit paged cache and attention over it (kv8_append, attn_kv8), and an INT4
mixture of experts (moe_w4a16).  Prompts are fed in chunks of at most 64 rows,
then one token per sequence and step; with --graph the decode step is captured
once and replayed.  Weights are random.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gemm_decode_qgemm_amd as qg  # noqa: E402


def rms(x: torch.Tensor, eps: float = 1e-6) -> torch.Tensor:
    x = x.float()
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)).bfloat16()


def rotation_table(positions: int, rot: int, device) -> torch.Tensor:
    angle = torch.arange(positions, device=device)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, device=device) / rot)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


class DecoderLayer:
    """Weights, cache and buffers of one layer for `batch` sequences of up to `max_len` tokens."""

    def __init__(self, batch, max_len, *, hidden=1024, hq=16, hkv=4, d=64, experts=16, top_k=4, inter=512, seed=0,
                 device="cuda"):
        if not 1 <= batch <= qg.binding.MAX_M:
            raise ValueError(f"a step has a row for every sequence and the linears take 1 to {qg.binding.MAX_M}, got {batch}")
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(n, k):
            return (torch.randn(n, k, generator=g, device=device) * k ** -0.5).bfloat16()

        self.hidden, self.hq, self.hkv, self.d, self.top_k, self.inter = hidden, hq, hkv, d, top_k, inter
        self.dense = {"qkv": weight((hq + 2 * hkv) * d, hidden), "o": weight(hidden, hq * d),
                      "gate_up": [weight(2 * inter, hidden) for _ in range(experts)],
                      "down": [weight(hidden, inter) for _ in range(experts)]}
        self.qkv, self.o = qg.quantize_int4_g32(self.dense["qkv"]), qg.quantize_int4_g32(self.dense["o"])
        self.gate_up = torch.stack([qg.quantize_int4_g32(w) for w in self.dense["gate_up"]])
        self.down = torch.stack([qg.quantize_int4_g32(w) for w in self.dense["down"]])
        self.router = weight(experts, hidden)
        self.q_norm = (1 + 0.1 * torch.randn(d, generator=g, device=device)).bfloat16()
        self.k_norm = (1 + 0.1 * torch.randn(d, generator=g, device=device)).bfloat16()
        self.cos_sin = rotation_table(max_len, d, device)
        width = -(-max_len // qg.KV8_PAGE)
        self.codes, self.scales = qg.kv8_empty(batch * width, hkv, d, device)
        self.table = torch.randperm(batch * width, generator=g, device=device).to(torch.int32).view(batch, width)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.max_len = max_len

    def forward(self, x: torch.Tensor, counts: torch.Tensor, cu: torch.Tensor | None, max_rows: int) -> torch.Tensor:
        """x [rows, hidden]: the next counts[b] tokens of every sequence, row offsets cu
        (None: the same number each)."""
        batch = self.lens.shape[0]
        before = self.lens.clone()
        self.lens += counts
        rows = x.shape[0]
        if cu is None:
            positions = (before[:, None] + torch.arange(rows // batch, device=x.device)).flatten().to(torch.int32)
        else:
            seq = torch.repeat_interleave(torch.arange(batch, device=x.device), counts.long(), output_size=rows)
            positions = (torch.arange(rows, device=x.device) - cu[seq] + before[seq]).to(torch.int32)
        qkv = qg.qgemm_w4a16(rms(x), self.qkv, (self.hq + 2 * self.hkv) * self.d).unflatten(1, (-1, self.d))
        q, k, v = qkv.split((self.hq, self.hkv, self.hkv), 1)
        q, k = qg.qk_norm_rope(q, k, self.q_norm, self.k_norm, self.cos_sin, positions)
        qg.kv8_append(k, v, self.codes, self.scales, self.table, self.lens, cu=cu, max_new=max_rows)
        a = qg.attn_kv8(q, self.codes, self.scales, self.table, self.lens, cu=cu, max_q=max_rows, max_len=self.max_len)
        x = x + qg.qgemm_w4a16(a.flatten(1), self.o, self.hidden)
        return x + qg.moe_w4a16(rms(x), self.router, self.gate_up, self.down, self.inter, self.top_k)

    def prompts(self, x: list) -> torch.Tensor:
        """Feeds prompts [n_b, hidden] in chunks of at most 64 rows in all; the last output row of each."""
        batch, at, last = len(x), [0] * len(x), [None] * len(x)
        share = max(1, qg.binding.MAX_M // batch)
        while any(at[b] < x[b].shape[0] for b in range(batch)):
            n = [min(share, x[b].shape[0] - at[b]) for b in range(batch)]
            rows = torch.cat([x[b][at[b]:at[b] + n[b]] for b in range(batch)])
            cu = [0]
            for c in n:
                cu.append(cu[-1] + c)
            y = self.forward(rows, torch.tensor(n, dtype=torch.int32, device=rows.device),
                             torch.tensor(cu, dtype=torch.int32, device=rows.device), max(n))
            for b in range(batch):
                at[b] += n[b]
                if n[b]:
                    last[b] = y[cu[b + 1] - 1]
        return torch.stack(last)


def prompt_lengths(longest: int, batch: int) -> list:
    """Ragged prompts of at least one token."""
    if longest < 1:
        raise ValueError("a prompt has at least one token")
    return [max(1, longest - 3 * (b % 5)) for b in range(batch)]


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--batch", type=int, default=8)
    p.add_argument("--prompt", type=int, default=100)
    p.add_argument("--steps", type=int, default=16)
    p.add_argument("--graph", action="store_true")
    a = p.parse_args()
    dev = torch.device("cuda")
    layer = DecoderLayer(a.batch, a.prompt + a.steps + 8)
    torch.manual_seed(1)
    x = layer.prompts([torch.randn(n, layer.hidden, device=dev).bfloat16() for n in prompt_lengths(a.prompt, a.batch)])
    one = torch.ones(a.batch, dtype=torch.int32, device=dev)
    step = lambda: x.copy_(rms(layer.forward(x, one, None, 1)))   # noqa: E731
    if a.graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        step = graph.replay
    step()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        step()
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / a.steps
    print(f"{a.batch} sequences of {layer.lens.tolist()} tokens: {t * 1e6:.1f} us a step"
          f"{' (graph)' if a.graph else ''}, output rms {x.float().square().mean().sqrt().item():.3f}")


if __name__ == "__main__":
    main()
