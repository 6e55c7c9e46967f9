"""One decoder layer of quantized linears, from prompt to decode.

    python examples/decoder_layer.py [--batch 8] [--prompt 100] [--steps 16] [--graph]
                                     [--adapters 3] [--groups 4] [--act8] [--drafts 3]

Every step runs on this library: the norms with the residual's addition
(rms_norm), the INT4 linears around attention (qgemm_w4a16), the norm and
rotation of query and key heads (qk_norm_rope), the 8-bit paged cache and attention
over it (kv8_append, attn_kv8), and an INT4 mixture of experts (moe_w4a16).
Prompts are fed in chunks of at most 64 rows, then one token per sequence and step;
with --graph the decode step is captured once and replayed.  Weights are random.

--adapters: the sequences' own low-rank adapters beside both projections (lora_add),
some sequences without one.  --groups: experts chosen by biased sigmoid scores
within the best half of that many groups (moe_route, moe_w4a16_picked).  --act8: the
first projection on 8-bit rows (rms_norm_q8, qgemm_w4a8_rows).  --drafts: every step
verifies that many drafted tokens a sequence against the probabilities of an INT4
head (verify_drafts), and the cache is left as if only the accepted ones had been fed.
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

    def __init__(self, batch, max_len, *, hidden=1024, hq=16, hkv=4, d=64, experts=16, top_k=4, inter=512, adapters=0,
                 rank=8, groups=1, act8=False, seed=0, device="cuda"):
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
        self.act8, self.groups = act8, groups
        self.bias = 0.1 * torch.randn(experts, generator=g, device=device) if groups > 1 else None
        self.lora, self.ids, self.lora_scales = {}, None, None
        if adapters:
            for name, n, k in (("qkv", (hq + 2 * hkv) * d, hidden), ("o", hidden, hq * d)):
                self.lora[name] = (torch.stack([weight(rank, k) for _ in range(adapters)]),
                                   torch.stack([weight(n, rank) for _ in range(adapters)]))
            self.lora_scales = 0.5 + torch.rand(adapters, generator=g, device=device)
            self.ids = (torch.arange(batch, device=device) % (adapters + 1) - 1).to(torch.int32)   # -1: without one

    def _adapt(self, name: str, y: torch.Tensor, x: torch.Tensor, ids: torch.Tensor | None) -> torch.Tensor:
        """The rows' adapters beside a projection, over its output."""
        return y if ids is None else qg.lora_add(y, x, *self.lora[name], ids, scales=self.lora_scales, out=y)

    def forward(self, x: torch.Tensor, counts: torch.Tensor, cu: torch.Tensor | None, max_rows: int,
                drafted: bool = False) -> torch.Tensor:
        """x [rows, hidden]: the next counts[b] tokens of every sequence, row offsets cu
        (None: the same number each).  drafted: keep_only may take some of them back."""
        batch = self.lens.shape[0]
        before = self.lens.clone()
        self.lens += counts
        rows = x.shape[0]
        if cu is None:
            positions = (before[:, None] + torch.arange(rows // batch, device=x.device)).flatten().to(torch.int32)
            ids = None if self.ids is None else self.ids.repeat_interleave(rows // batch)
        else:
            seq = torch.repeat_interleave(torch.arange(batch, device=x.device), counts.long(), output_size=rows)
            positions = (torch.arange(rows, device=x.device) - cu[seq] + before[seq]).to(torch.int32)
            ids = None if self.ids is None else self.ids[seq]
        width = (self.hq + 2 * self.hkv) * self.d
        if self.act8:
            codes, scales = qg.rms_norm_q8(x, group_scales=True)
            qkv = qg.qgemm_w4a8_rows(codes, scales, self.qkv, width)
            normed = None if ids is None else qg.rms_norm(x)
        else:
            normed = qg.rms_norm(x)
            qkv = qg.qgemm_w4a16(normed, self.qkv, width)
        qkv = self._adapt("qkv", qkv, normed, ids).unflatten(1, (-1, self.d))
        q, k, v = qkv.split((self.hq, self.hkv, self.hkv), 1)
        q, k = qg.qk_norm_rope(q, k, self.q_norm, self.k_norm, self.cos_sin, positions)
        if drafted:   # the pages that hold tokens already and get new ones: theirs are requantized with the new ones' scale
            page = (before // qg.KV8_PAGE).clamp(max=self.table.shape[1] - 1).long()
            page = self.table.gather(1, page[:, None])[:, 0].long()
            self.before = page, self.codes[page], self.scales[page], k, v
        qg.kv8_append(k, v, self.codes, self.scales, self.table, self.lens, cu=cu, max_new=max_rows)
        a = qg.attn_kv8(q, self.codes, self.scales, self.table, self.lens, cu=cu, max_q=max_rows, max_len=self.max_len).flatten(1)
        o = self._adapt("o", qg.qgemm_w4a16(a, self.o, self.hidden), a, ids)
        normed, x = qg.rms_norm(o, residual=x)
        if self.groups > 1:
            chosen, weights = qg.moe_route(normed.float() @ self.router.float().t(), self.top_k, sigmoid=True, bias=self.bias,
                                           groups=self.groups, top_groups=self.groups // 2, group_best=2)
            return x + qg.moe_w4a16_picked(normed, chosen, weights, self.gate_up, self.down, self.inter)
        return x + qg.moe_w4a16(normed, self.router, self.gate_up, self.down, self.inter, self.top_k)

    def keep_only(self, kept: torch.Tensor) -> None:
        """Leaves the cache as if of the last step's rows (`drafted`, the same number each) sequence b had fed the first
        kept[b] >= 1 alone; lens counts these already.  A shorter length by itself would leave them, and the tokens
        before them, with the scales that the others raised, or made NaN."""
        page, codes, scales, k, v = self.before
        self.codes[page], self.scales[page] = codes, scales
        rows = k.shape[0] // kept.shape[0]
        gone = torch.arange(rows, device=k.device) >= kept[:, None]
        order = gone.flatten().to(torch.uint8).argsort(stable=True)      # the kept rows, then those that no sequence has
        cu = torch.cat([torch.zeros_like(kept[:1]), kept.cumsum(0, dtype=torch.int32)])
        qg.kv8_append(k[order], v[order], self.codes, self.scales, self.table, self.lens, cu=cu, max_new=rows)

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


class Speculator:
    """Drafted tokens verified by a layer with an embedding and an INT4 head."""

    def __init__(self, layer: DecoderLayer, vocabulary: int = 4096, seed: int = 1):
        device = layer.router.device
        g = torch.Generator(device=device).manual_seed(seed)
        self.layer, self.vocabulary, self.g = layer, vocabulary, g
        self.embedding = torch.randn(vocabulary, layer.hidden, generator=g, device=device).bfloat16()
        head = (torch.randn(vocabulary, layer.hidden, generator=g, device=device) * layer.hidden ** -0.5).bfloat16()
        self.head = qg.quantize_int4_g32(head)

    def probabilities(self, y: torch.Tensor) -> torch.Tensor:
        return torch.softmax(qg.qgemm_w4a16(qg.rms_norm(y), self.head, self.vocabulary, out_dtype=torch.float32), 1)

    def step(self, last: torch.Tensor, drafts: int) -> tuple:
        """One step for every sequence: its last token and `drafts` drafted ones (drawn evenly
        from the vocabulary here; a draft model's otherwise).  (accepted [b], next token [b]);
        the cache is left with the last and the accepted tokens alone."""
        layer, device = self.layer, last.device
        b, rows = last.shape[0], last.shape[0] * (drafts + 1)
        tokens = torch.randint(0, self.vocabulary, (b, drafts), generator=self.g, device=device)
        q = torch.full((b * drafts, self.vocabulary), 1 / self.vocabulary, device=device)
        x = self.embedding[torch.cat([last[:, None].long(), tokens], 1).flatten()]
        y = layer.forward(x, torch.full_like(layer.lens, drafts + 1), None, drafts + 1, drafted=True)
        cu = torch.arange(0, rows + 1, drafts + 1, dtype=torch.int32, device=device)
        u = torch.rand(b * drafts, generator=self.g, device=device)
        accepted, following = qg.verify_drafts(self.probabilities(y), q, tokens.flatten().to(torch.int32), u,
                                               torch.rand(b, generator=self.g, device=device), cu, lens=layer.lens)
        layer.keep_only(accepted + 1)
        return accepted, following


def prompt_lengths(longest: int, batch: int) -> list:
    """Ragged prompts of at least one token."""
    if longest < 1:
        raise ValueError("a prompt has at least one token")
    return [max(1, longest - 3 * (b % 5)) for b in range(batch)]


def most_tokens(prompt: int, steps: int, drafts: int) -> int:
    """Tokens of the longest sequence: its prompt and all that the steps feed, up to two before the timed ones too."""
    return prompt + (steps + 2) * (drafts + 1)


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--batch", type=int, default=8)
    p.add_argument("--prompt", type=int, default=100)
    p.add_argument("--steps", type=int, default=16)
    p.add_argument("--graph", action="store_true")
    p.add_argument("--adapters", type=int, default=0)
    p.add_argument("--groups", type=int, default=1)
    p.add_argument("--act8", action="store_true")
    p.add_argument("--drafts", type=int, default=0)
    a = p.parse_args()
    if a.drafts and (a.graph or a.batch * (a.drafts + 1) > qg.binding.MAX_M):
        p.error(f"--drafts takes no --graph, and at most {qg.binding.MAX_M} rows a step")
    dev = torch.device("cuda")
    layer = DecoderLayer(a.batch, most_tokens(a.prompt, a.steps, a.drafts), adapters=a.adapters, groups=a.groups, act8=a.act8)
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
    if a.drafts:
        speculator = Speculator(layer)
        last = torch.zeros(a.batch, dtype=torch.int32, device=dev)
        step = lambda: last.copy_(speculator.step(last, a.drafts)[1])   # noqa: E731
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
