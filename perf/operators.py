"""Cases of the decoder-layer operators around the quantized linears.

Four operators, each called as a decoder calls it:

* ``norm_rope``: RMS norm of every query and key head with the position
  rotation in the same pass (qg.qk_norm_rope), on the q and k columns of a
  fused projection's output;
* ``kv8``: a chunk of new keys and values appended to a paged cache held in
  8 bits, and the sequences read back (qg.kv8_append, qg.kv8_read);
* ``attn``: attention of a few query rows per sequence over that cache
  (qg.attn_kv8);
* ``moe``: a whole mixture-of-experts layer with packed INT4 experts
  (qg.moe_w4a16).

``run`` computes the plain form where ``own`` is false: elementary torch
operations in 32 bits, rounded once at the end.  Where ``own`` is true it makes
the framework's calls.  The cache and the packed weight are described in
include/qgemm.h; their layouts are repeated below in plain indexing.
"""
import torch

own = False

PAGE = 64      # tokens in a page of the cache
BLOCK = 16     # tokens sharing a scale (per head, keys and values apart)
TILE = 9472    # bytes of a 64-row x 256-k tile of the packed INT4 weight


def listed():
    return [
        # one decode step of one request: latency only
        {"name": "norm_rope_one", "op": "norm_rope", "t": 1, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "pairs": False},
        # a decode batch, wide heads, a quarter of each rotated in adjacent pairs
        {"name": "norm_rope_batch", "op": "norm_rope", "t": 61, "hq": 16, "hkv": 2, "d": 256, "rot": 64, "pairs": True},
        # a long prompt of odd length: bound by memory
        {"name": "norm_rope_prompt", "op": "norm_rope", "t": 16383, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "pairs": False},
        # single new tokens on short sequences, blocks that are partly filled
        {"name": "kv8_tokens", "op": "kv8", "b": 3, "new_lo": 1, "new_hi": 1, "old_lo": 90, "old_hi": 203, "hkv": 8, "d": 128},
        # chunks of two ragged prompts, one of them after a short prefix
        {"name": "kv8_prompts", "op": "kv8", "b": 2, "new_lo": 5001, "new_hi": 16001, "old_lo": 0, "old_hi": 41, "hkv": 8, "d": 128},
        # the first tokens of one request
        {"name": "attn_short", "op": "attn", "b": 1, "q": 1, "ragged": False, "hq": 32, "hkv": 8, "d": 128, "lo": 37, "hi": 37, "window": 0},
        # a decode batch of mixed lengths with an idle slot of length 0
        {"name": "attn_batch", "op": "attn", "b": 48, "q": 1, "ragged": False, "hq": 32, "hkv": 8, "d": 128, "lo": 0, "hi": 4095, "window": 0},
        # one long document, every query head on one key head (this layer set's 32 query heads and 256-row KV projection)
        {"name": "attn_long", "op": "attn", "b": 1, "q": 1, "ragged": False, "hq": 32, "hkv": 1, "d": 128, "lo": 131071, "hi": 131071, "window": 0},
        # ragged verification of drafted tokens, six query heads to a key head, sliding window
        {"name": "attn_verify", "op": "attn", "b": 8, "q": 9, "ragged": True, "hq": 24, "hkv": 4, "d": 64, "lo": 511, "hi": 8191, "window": 4096},
        # one token through many small experts: latency and little traffic
        {"name": "moe_one", "op": "moe", "t": 1, "e": 128, "k": 8, "h": 2048, "inter": 768, "renorm": True},
        # a decode batch: most experts hit by one or two tokens
        {"name": "moe_batch", "op": "moe", "t": 17, "e": 64, "k": 6, "h": 2048, "inter": 1024, "renorm": False},
        # the largest decode batch on a few large experts: every weight read, several tokens each
        {"name": "moe_large", "op": "moe", "t": 64, "e": 8, "k": 2, "h": 4096, "inter": 14336, "renorm": True},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm_rope", "kv8", "attn", "attn", "moe", "moe"])
    if op == "norm_rope":
        d, hkv = rng.choice([64, 80, 96, 128, 192, 256]), rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 3, 4, 6, 8])
        return {"op": op, "t": _log(rng, 1, max(1, 16383 * 40 * 128 // ((hq + hkv) * d))), "hq": hq, "hkv": hkv, "d": d,
                "rot": d if rng.random() < 0.6 else 32, "pairs": rng.random() < 0.4}
    if op == "kv8":
        b, d, hkv = _log(rng, 1, 64), rng.choice([64, 128, 192, 256]), rng.choice([1, 2, 4, 8])
        most = max(2, 20000 * 1024 // (b * hkv * d))
        new = _log(rng, 1, min(16000, most))
        old = rng.randrange(0, min(300, most) + 1)
        return {"op": op, "b": b, "new_lo": max(1, new // 3), "new_hi": new, "old_lo": old // 2, "old_hi": old, "hkv": hkv, "d": d}
    if op == "attn":
        d, hkv = rng.choice([64, 128, 192, 256]), rng.choice([1, 2, 4, 8])
        hq, b = hkv * rng.choice([1, 2, 4, 5, 6, 8, 16]), _log(rng, 1, 64)
        q = 1 if rng.random() < 0.5 else _log(rng, 2, 64)
        hi = _log(rng, max(q, 8), max(q, 8, min(131071, 48 * 2048 * 1024 // (b * hkv * d), 131071 * 32 * 128 // (b * hq * q * d))))
        return {"op": op, "b": b, "q": q, "ragged": q > 1 and rng.random() < 0.7, "hq": hq, "hkv": hkv, "d": d,
                "lo": rng.randrange(0, hi + 1), "hi": hi, "window": 0 if rng.random() < 0.7 else _log(rng, 16, 4096)}
    e, k = rng.choice([(8, 2), (16, 4), (32, 4), (64, 6), (128, 8), (160, 6)])
    h = rng.choice([1024, 1280, 2048, 2560, 4096])
    inter = 256 * (2 * _log(rng, 1, max(1, min(27, 4 * 4096 * 56 // (e * h) - 1))) + 1)
    return {"op": op, "t": _log(rng, 1, 64), "e": e, "k": k, "h": h, "inter": inter, "renorm": rng.random() < 0.5}


def _spread(lo, hi, n):
    """n whole numbers evenly from lo to hi (hi alone for n = 1)."""
    return [hi] if n == 1 else [lo + i * (hi - lo) // (n - 1) for i in range(n)]


def _queries(c):
    """Query rows of each sequence."""
    return _spread(1, c["q"], c["b"]) if c["ragged"] else [c["q"]] * c["b"]


def _lengths(c):
    """Tokens of each sequence in the cache, the new ones among them."""
    if c["op"] == "kv8":
        return [n + o for n, o in zip(_news(c), _olds(c))]
    return _spread(c["lo"], c["hi"], c["b"])


def _news(c):
    return _spread(c["new_lo"], c["new_hi"], c["b"])


def _olds(c):
    return _spread(c["old_hi"], c["old_lo"], c["b"])


def work(case):
    c = case
    if c["op"] == "norm_rope":
        heads = c["t"] * (c["hq"] + c["hkv"])
        return {"bytes": heads * c["d"] * 4 + c["t"] * (c["rot"] * 4 + 4) + 4 * c["d"],
                "flops": heads * (4 * c["d"] + 3 * c["rot"])}
    if c["op"] == "kv8":
        n, total, row = sum(_news(c)), sum(_lengths(c)), 2 * c["hkv"] * c["d"]
        return {"bytes": n * row * 3 + total * row + c["b"] * max(_lengths(c)) * row * 2 + total // BLOCK * 8 * c["hkv"],
                "flops": n * row * 4 + total * row}
    if c["op"] == "attn":
        seen = pairs = rows = 0
        for n, q in zip(_lengths(c), _queries(c)):
            rows += q
            first = n - q + 1 - c["window"] if c["window"] else 0
            seen += n - min(n, max(0, first))
            for i in range(q):
                p = n - q + i + 1
                if p > 0:
                    pairs += min(p, c["window"]) if c["window"] else p
        return {"bytes": seen * c["hkv"] * (2 * c["d"] + 8 / BLOCK) + rows * c["hq"] * c["d"] * 4,
                "flops": pairs * c["hq"] * c["d"] * 4}
    expert = 3 * c["h"] * c["inter"]
    hit = c["e"] * (1 - (1 - c["k"] / c["e"]) ** c["t"])   # experts that some token picks, on average
    return {"bytes": hit * expert * 37 / 64 + c["e"] * c["h"] * 2 + c["t"] * c["h"] * 4,
            "flops": 2 * c["t"] * (c["k"] * expert + c["e"] * c["h"])}


def _cache(c, g, dev, full):
    """A cache in use: pages in no order, codes and scales as a quantizer leaves them."""
    b, lens = c["b"], _lengths(c)
    width = max(1, -(-max(lens) // PAGE))
    need = [width if full else -(-n // PAGE) for n in lens]
    pages = max(1, sum(need))
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(b, width, dtype=torch.int32, device=dev)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    shape = (pages, c["hkv"], 2, PAGE * c["d"])
    codes = torch.empty(shape, dtype=torch.int8, device=dev)
    for p in range(0, pages, 1024):   # a part at a time: the draws are in 32 bits
        part = torch.randn((min(1024, pages - p),) + shape[1:], generator=g, device=dev)
        codes[p:p + 1024] = (part * 40).round().clamp(-127, 127).to(torch.int8)
    scales = 0.02 + 0.02 * torch.rand(pages, c["hkv"], 2, PAGE // BLOCK, generator=g, device=dev)
    return {"codes": codes, "scales": scales, "table": table,
            "lens": torch.tensor(lens, dtype=torch.int32, device=dev), "max_len": max(1, max(lens))}


def _packed(e, n, k, g, dev):
    """Packed INT4 experts: codes of all values, zero points about the middle, scales of weights near 1 / sqrt(k)."""
    t = torch.empty(e, n // 64 * (k // 256), TILE, dtype=torch.uint8, device=dev)
    t[..., :8192] = torch.randint(0, 256, t.shape[:2] + (8192,), generator=g, device=dev, dtype=torch.uint8)
    s = (0.15 + 0.1 * torch.rand(t.shape[:2] + (512,), generator=g, device=dev)) / k ** 0.5
    t[..., 8192:9216] = s.to(torch.float16).view(torch.uint8)
    z = torch.randint(6, 10, t.shape[:2] + (256, 2), generator=g, device=dev, dtype=torch.uint8)
    t[..., 9216:] = z[..., 0] | (z[..., 1] << 4)
    return t.reshape(e, -1)


def _starts(counts, dev):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device=dev)


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "norm_rope":
        t, d, heads = c["t"], c["d"], c["hq"] + 2 * c["hkv"]
        qkv = torch.randn(t, heads * d, generator=g, device=dev).to(torch.bfloat16)   # a fused projection's output
        s["q"] = qkv[:, :c["hq"] * d].unflatten(1, (c["hq"], d))
        s["k"] = qkv[:, c["hq"] * d:(c["hq"] + c["hkv"]) * d].unflatten(1, (c["hkv"], d))
        s["qw"] = (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(torch.bfloat16)
        s["kw"] = (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(torch.bfloat16)
        most = 32768
        angle = torch.arange(most, device=dev, dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, c["rot"], 2, device=dev, dtype=torch.float64) / c["rot"])
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)
        first = torch.randint(0, most - t + 1, (1,), generator=g, device=dev)
        s["pos"] = (torch.randint(0, most, (t,), generator=g, device=dev) if t < 256 else
                    first + torch.arange(t, device=dev)).to(torch.int32)
    elif c["op"] == "kv8":
        s |= _cache(c, g, dev, True)
        row = torch.randn(sum(_news(c)), 2, c["hkv"], c["d"], generator=g, device=dev)
        row[..., 3] *= 4   # a channel that stands out, as keys have
        row = row.to(torch.bfloat16)
        s["k"], s["v"], s["cu"], s["max_new"] = row[:, 0], row[:, 1], _starts(_news(c), dev), max(_news(c))
    elif c["op"] == "attn":
        s |= _cache(c, g, dev, False)
        q = _queries(c)
        s["q"] = (2 * torch.randn(sum(q), c["hq"], c["d"], generator=g, device=dev)).to(torch.bfloat16)
        s["cu"], s["max_q"] = _starts(q, dev) if c["ragged"] else None, max(q)
    else:
        s["x"] = torch.randn(c["t"], c["h"], generator=g, device=dev).to(torch.bfloat16)
        s["router"] = (1.5 / c["h"] ** 0.5 * torch.randn(c["e"], c["h"], generator=g, device=dev)).to(torch.bfloat16)
        s["gate_up"] = _packed(c["e"], 2 * c["inter"], c["h"], g, dev)   # rows: gate, then up
        s["down"] = _packed(c["e"], c["h"], c["inter"], g, dev)
    return s


def run(state):
    s, c = state, state["case"]
    if own:
        import gemm_decode_qgemm_amd as qg
        if c["op"] == "norm_rope":
            return qg.qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["cos_sin"], s["pos"], adjacent_pairs=c["pairs"])
        if c["op"] == "kv8":
            qg.kv8_append(s["k"], s["v"], s["codes"], s["scales"], s["table"], s["lens"], cu=s["cu"], max_new=s["max_new"])
            return qg.kv8_read(s["codes"], s["scales"], s["table"], s["lens"], s["max_len"])
        if c["op"] == "attn":
            return qg.attn_kv8(s["q"], s["codes"], s["scales"], s["table"], s["lens"], cu=s["cu"], max_q=s["max_q"],
                               max_len=s["max_len"], window=c["window"])
        return qg.moe_w4a16(s["x"], s["router"], s["gate_up"], s["down"], c["inter"], c["k"], renormalize=c["renorm"])
    return {"norm_rope": _plain_norm_rope, "kv8": _plain_kv8, "attn": _plain_attn, "moe": _plain_moe}[c["op"]](s, c)


# ---- the plain forms ---------------------------------------------------------

def _rotate(x, cos, sin, rot, pairs):
    r, rest = x[..., :rot], x[..., rot:]
    a, b = (r[..., 0::2], r[..., 1::2]) if pairs else (r[..., :rot // 2], r[..., rot // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([u, v], -1).flatten(-2) if pairs else torch.cat([u, v], -1)
    return torch.cat([r, rest], -1)


def _plain_norm_rope(s, c):
    cs = s["cos_sin"][s["pos"].long()][:, None]
    cos, sin = cs[..., :c["rot"] // 2], cs[..., c["rot"] // 2:]

    def one(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
        return _rotate(x, cos, sin, c["rot"], c["pairs"]).to(torch.bfloat16)

    return one(s["q"], s["qw"]), one(s["k"], s["kw"])


def _unpack_cache(s, c):
    """Codes [b, hkv, tokens, d] of keys and values, and scales [b, hkv, 2, blocks]."""
    b, width = s["table"].shape
    t, h, d = s["table"].long(), c["hkv"], c["d"]
    k = s["codes"][:, :, 0][t].view(b, width, h, PAGE, d).transpose(1, 2).reshape(b, h, width * PAGE, d)
    v = s["codes"][:, :, 1][t].view(b, width, h, d, 4, 4, 4)   # a channel's tokens: [quad][block][token of the quad]
    v = v.permute(0, 2, 1, 5, 4, 6, 3).reshape(b, h, width * PAGE, d)
    sc = s["scales"][t].permute(0, 2, 3, 1, 4).reshape(b, h, 2, width * PAGE // BLOCK)
    return k, v, sc


def _values(codes, scale):
    return codes.float() * scale.repeat_interleave(BLOCK, -1)[..., None]


def _plain_kv8(s, c):
    codes_k, codes_v, old_scale = _unpack_cache(s, c)
    b, h, n, d = codes_k.shape
    lens, cu = s["lens"].long(), s["cu"].long()
    old = lens - (cu[1:] - cu[:-1])
    j = torch.arange(n, device=lens.device)
    fresh = (j >= old[:, None]) & (j < lens[:, None])                       # [b, n]
    row = (cu[:-1, None] + j - old[:, None]).clamp(0, s["k"].shape[0] - 1)
    start = torch.arange(n // BLOCK, device=lens.device) * BLOCK
    kept = start < old[:, None]                                             # blocks that hold earlier tokens
    touched = (start < lens[:, None]) & (start + BLOCK > old[:, None])
    out = []
    for which, new, codes in ((0, s["k"], codes_k), (1, s["v"], codes_v)):
        x = torch.where(fresh[:, None, :, None], new.float()[row].transpose(1, 2), 0.0)   # [b, h, n, d]
        top = x.abs().reshape(b, h, -1, BLOCK * d).amax(-1) * (1 / 127)
        before = torch.where(kept[:, None], old_scale[:, :, which], 0.0)
        scale = torch.where(touched[:, None], torch.maximum(before, top), old_scale[:, :, which])
        shrink = torch.where(touched[:, None] & (scale > before), before / scale, 1.0)
        held = (codes.float() * shrink.repeat_interleave(BLOCK, -1)[..., None]).round()
        wide = scale.repeat_interleave(BLOCK, -1)[..., None]
        q = torch.where(wide > 0, (x / wide).round().clamp(-127, 127), 0.0)
        here = fresh[:, None, :, None]
        past = touched.repeat_interleave(BLOCK, -1)[:, None, :, None] & (j >= lens[:, None])[:, None, :, None]
        codes = torch.where(past, 0.0, torch.where(here, q, held)).to(torch.int8)
        pages = codes.reshape(b, h, n // PAGE, PAGE, d).transpose(1, 2)
        if which:
            pages = pages.unflatten(3, (4, 4, 4)).permute(0, 1, 2, 6, 4, 3, 5)   # [d][quad][block][token]
        t = s["table"].long().flatten()
        s["codes"][t, :, which] = pages.reshape(-1, h, PAGE * d)
        s["scales"][t, :, which] = scale.reshape(b, h, -1, 4).transpose(1, 2).reshape(-1, h, 4)
        value = torch.where((j < lens[:, None])[:, None, :, None], _values(codes, scale), 0.0)
        out.append(value[:, :, :s["max_len"]].transpose(1, 2).to(torch.bfloat16).contiguous())
    return tuple(out)


def _plain_attn(s, c):
    ck, cv, sc = _unpack_cache(s, c)
    k, v = _values(ck, sc[:, :, 0]), _values(cv, sc[:, :, 1])               # [b, hkv, n, d]
    b, h, n, d = k.shape
    lens, mq = s["lens"].long(), s["max_q"]
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(b + 1, device=k.device) * mq
    nq = cu[1:] - cu[:-1]
    i = torch.arange(mq, device=k.device)
    row = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)                # [b, mq]
    q = s["q"].float()[row].view(b, mq, h, -1, d).permute(0, 2, 3, 1, 4)    # [b, hkv, group, mq, d]
    pos = (lens - nq)[:, None] + i
    j = torch.arange(n, device=k.device)
    seen = j <= pos[..., None]                                              # [b, mq, n]
    if c["window"]:
        seen &= j > pos[..., None] - c["window"]
    group = q.shape[2]
    score = torch.matmul(q.reshape(b, h, group * mq, d), k.transpose(2, 3)) * d ** -0.5
    score = score.view(b, h, group, mq, n).masked_fill(~seen[:, None, None], -torch.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -torch.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    o = torch.matmul(p.view(b, h, group * mq, n), v).view(b, h, group, mq, d).permute(0, 3, 1, 2, 4)
    o = o.reshape(b, mq, h * group, d).to(torch.bfloat16)
    return o[i < nq[:, None]] if s["cu"] is not None else o.reshape(b * mq, h * group, d)


def _unpack_weight(packed, n, k):
    """Packed INT4 [*, bytes] -> 32-bit values [*, n, k]."""
    t = packed.view(-1, n // 64, k // 256, TILE)
    m = t.shape[0]
    c = t[..., :8192].unflatten(-1, (8, 64, 4, 4))                          # [group][row][dword][byte]
    c = torch.stack([c & 15, c >> 4], -1).flatten(-2)                       # nibbles of a dword, low first
    order = torch.tensor([0, 4, 1, 5, 2, 6, 3, 7], device=t.device)         # nibble that holds k = 8 d + e
    c = c.index_select(-1, order).flatten(-2)                               # [m, rb, kt, group, row, 32]
    s = t[..., 8192:9216].contiguous().view(torch.float16).unflatten(-1, (64, 8))
    z = t[..., 9216:]
    z = torch.stack([z & 15, z >> 4], -1).flatten(-2).unflatten(-1, (64, 8))   # [row][group]
    w = (c.float() - z.transpose(-1, -2)[..., None].float()) * s.transpose(-1, -2)[..., None].float()
    return w.permute(0, 1, 4, 2, 3, 5).reshape(m, n, k)


def _plain_moe(s, c):
    t, e, top, h, inter = c["t"], c["e"], c["k"], c["h"], c["inter"]
    x = s["x"].float()
    logits = x @ s["router"].float().t()
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    ids, chosen = order.indices[:, :top], order.values[:, :top]
    if c["renorm"]:
        p = torch.exp(chosen - chosen[:, :1])
        p = p / p.sum(1, keepdim=True)
    else:
        p = torch.exp(chosen - chosen[:, :1]) / torch.exp(logits - chosen[:, :1]).sum(1, keepdim=True)
    if t * top < e:   # the picked experts alone, one product per pick
        flat = ids.flatten()
        gu = torch.matmul(_unpack_weight(s["gate_up"][flat], 2 * inter, h), x.repeat_interleave(top, 0)[..., None])[..., 0]
        a = gu[:, :inter] * torch.sigmoid(gu[:, :inter]) * gu[:, inter:]
        y = torch.matmul(_unpack_weight(s["down"][flat], h, inter), a[..., None])[..., 0]
        y = (y.view(t, top, h) * p[..., None]).sum(1)
    else:             # every expert on every token
        gu = torch.matmul(x, _unpack_weight(s["gate_up"], 2 * inter, h).transpose(1, 2))   # [e, t, 2 inter]
        a = gu[..., :inter] * torch.sigmoid(gu[..., :inter]) * gu[..., inter:]
        y = torch.matmul(a, _unpack_weight(s["down"], h, inter).transpose(1, 2))           # [e, t, h]
        w = torch.zeros(t, e, device=x.device).scatter_(1, ids, p)
        y = (y * w.t()[..., None]).sum(0)
    return y.to(torch.bfloat16)


# ---- the definitions in 64 bits ------------------------------------------------

def _exact_tokens(s, c, i, n):
    """Keys and values [hkv, n, d] of the first n tokens of sequence i, as codes and scales [hkv, n]."""
    j = torch.arange(n, device=s["codes"].device)
    page, at = s["table"][i].long()[j // PAGE], j % PAGE
    block = at // BLOCK
    d = torch.arange(c["d"], device=j.device)
    k = s["codes"][page[:, None], :, 0, (at * c["d"])[:, None] + d]
    v = s["codes"][page[:, None], :, 1, d * PAGE + (at % BLOCK // 4 * 16 + block * 4 + at % 4)[:, None]]   # [n, d, hkv]
    return [(x.permute(2, 0, 1).double(), s["scales"][page, :, w, block].t().double()) for w, x in ((0, k), (1, v))]


def _exact_kv8(s, c):
    news, olds = _news(c), _olds(c)
    out = [torch.zeros(c["b"], s["max_len"], c["hkv"], c["d"], dtype=torch.float64, device=s["k"].device) for _ in range(2)]
    for i in range(c["b"]):
        old, new = olds[i], news[i]
        held = _exact_tokens(s, c, i, old) if old else None
        lo = int(s["cu"][i])
        for which, x in ((0, s["k"]), (1, s["v"])):
            y = x[lo:lo + new].double().transpose(0, 1)                     # [hkv, new, d]
            whole = old // BLOCK * BLOCK
            if old:
                codes, sc = held[which]
                out[which][i, :whole] = (codes * sc[..., None])[:, :whole].transpose(0, 1)
            part = old - whole                                              # tokens already in the first touched block
            pad = -(part + new) % BLOCK
            y = torch.cat([torch.zeros(c["hkv"], part, c["d"], device=y.device, dtype=y.dtype), y,
                           torch.zeros(c["hkv"], pad, c["d"], device=y.device, dtype=y.dtype)], 1)
            y = y.unflatten(1, (-1, BLOCK))                                 # [hkv, blocks, 16, d]
            scale = y.abs().amax((2, 3)) / 127
            if part:
                before = sc[:, whole]
                scale[:, 0] = torch.maximum(scale[:, 0], before)
            q = torch.round(y / scale[..., None, None]).clamp(-127, 127)
            if part:
                q[:, 0, :part] = torch.round(codes[:, whole:] * (before / scale[:, 0])[:, None, None])
            out[which][i, whole:old + new] = (q * scale[..., None, None]).flatten(1, 2)[:, :part + new].transpose(0, 1)
    return tuple(out)


def _exact_attn(s, c):
    group, parts, at = c["hq"] // c["hkv"], [], 0
    for i, (n, nq) in enumerate(zip(_lengths(c), _queries(c))):
        q = s["q"][at:at + nq].double().unflatten(1, (c["hkv"], group))     # [nq, hkv, group, d]
        at += nq
        o = torch.zeros_like(q)
        if n:
            (ck, sk), (cv, sv) = _exact_tokens(s, c, i, n)
            k, v = ck * sk[..., None], cv * sv[..., None]
            for r in range(nq):
                end = n - nq + r + 1
                first = max(0, end - c["window"]) if c["window"] else 0
                if end > 0:
                    w = torch.softmax(torch.matmul(q[r], k[:, first:end].transpose(1, 2)) / c["d"] ** 0.5, -1)
                    o[r] = torch.matmul(w, v[:, first:end])
        parts.append(o.flatten(1, 2))
    return torch.cat(parts)


def _exact_weight(packed, n, k):
    """One packed matrix in 64 bits: nibble p of a dword holds k = 8 d + e with p = 4 (e % 2) + e / 2."""
    t = packed.view(n // 64, k // 256, TILE)
    w = torch.empty(n // 64, 64, k // 256, 8, 4, 8, dtype=torch.float64, device=packed.device)   # [rb, row, kt, group, dword, e]
    scale = t[..., 8192:9216].contiguous().view(torch.float16).view(n // 64, k // 256, 64, 8).double()
    zero = t[..., 9216:].contiguous().view(torch.int32).view(n // 64, k // 256, 64)
    words = t[..., :8192].contiguous().view(torch.int32).view(n // 64, k // 256, 8, 64, 4)
    for g in range(8):
        z = (zero >> (4 * g) & 15).transpose(1, 2).double()                 # [rb, row, kt]
        sc = scale[..., g].transpose(1, 2)
        for e in range(8):
            q = (words[:, :, g] >> (4 * (4 * (e % 2) + e // 2)) & 15).transpose(1, 2).double()   # [rb, row, kt, dword]
            w[:, :, :, g, :, e] = (q - z[..., None]) * sc[..., None]
    return w.view(n, k)


def _exact_moe(s, c):
    x = s["x"].double()
    logits = torch.matmul(x, s["router"].double().t())
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    if c["renorm"]:
        w = torch.softmax(torch.gather(logits, 1, ids), 1)
    else:
        w = torch.gather(torch.softmax(logits, 1), 1, ids)
    y = torch.zeros_like(x)
    for e in ids.unique().tolist():
        tok, slot = (ids == e).nonzero(as_tuple=True)
        gu = torch.matmul(x[tok], _exact_weight(s["gate_up"][e], 2 * c["inter"], c["h"]).t())
        a = torch.nn.functional.silu(gu[:, :c["inter"]]) * gu[:, c["inter"]:]
        y[tok] += w[tok, slot][:, None] * torch.matmul(a, _exact_weight(s["down"][e], c["h"], c["inter"]).t())
    return y


def _exact_norm_rope(s, c):
    cs = s["cos_sin"].double()[s["pos"].long()]
    half = c["rot"] // 2
    turn = torch.complex(cs[:, :half], cs[:, half:])[:, None]               # [t, 1, rot / 2]
    out = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        y = x.double()
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.double()
        r = y[..., :c["rot"]].clone()
        if c["pairs"]:
            z = torch.complex(r[..., 0::2].contiguous(), r[..., 1::2].contiguous()) * turn
            r = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(r[..., :half].contiguous(), r[..., half:].contiguous()) * turn
            r = torch.cat([z.real, z.imag], -1)
        out.append(torch.cat([r, y[..., c["rot"]:]], -1))
    return tuple(out)


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_rope": _exact_norm_rope, "kv8": _exact_kv8, "attn": _exact_attn, "moe": _exact_moe}[case["op"]](s, case)
