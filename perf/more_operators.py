"""Cases of the serving-step operators around the quantized linears.

Four operators, each called as a serving step calls it:

* ``norm``: a sub-layer's output added to the residual stream and the RMS norm
  of the sum, in bf16 (qg.rms_norm) or as the 8-bit rows with scales that the
  W4A8 linears take (qg.rms_norm_q8);
* ``lora``: the low-rank adapters of many requests added to a shared
  projection's output (qg.lora_add);
* ``route``: the choice of experts from a router's logits: softmax or sigmoid
  scores, a balancing bias, groups, top-k and their weights (qg.moe_route);
* ``verify``: drafted tokens accepted or rejected against the target's
  probabilities, and the next token drawn, from given random numbers
  (qg.verify_drafts).

``run`` computes the plain form where ``own`` is false: elementary torch
operations in 32 bits (64 where values next to a border decide), rounded once
at the end.  Where ``own`` is true it makes the framework's calls.
"""
import torch

own = False

GROUP = 32     # channels that share a scale of the 8-bit rows, where rows do not


def listed():
    return [
        # one token of one request between two sub-layers: latency only
        {"name": "norm_one", "op": "norm", "t": 1, "h": 6656, "x32": False, "res": "bf16", "out": "bf16"},
        # a decode batch, quantized for the W4A8 linear that follows, one scale a row
        {"name": "norm_batch_q8", "op": "norm", "t": 61, "h": 6656, "x32": False, "res": "bf16", "out": "row"},
        # a long prompt of odd length on a residual stream kept in 32 bits, one scale per 32 channels: bound by memory
        {"name": "norm_prompt_q8", "op": "norm", "t": 16383, "h": 4096, "x32": False, "res": "f32", "out": "group"},
        # one request's adapter beside its key/value projection: latency only
        {"name": "lora_one", "op": "lora", "m": 1, "k": 6656, "n": 256, "r": 16, "adapters": 4, "plain": 0, "y32": False},
        # a decode batch of several requests per adapter, some without one, beside the fused projection
        {"name": "lora_batch", "op": "lora", "m": 41, "k": 6656, "n": 8448, "r": 16, "adapters": 24, "plain": 5, "y32": False},
        # the largest batch, an adapter of higher rank for every request, beside the widest projection
        {"name": "lora_large", "op": "lora", "m": 64, "k": 6656, "n": 39936, "r": 64, "adapters": 64, "plain": 0, "y32": False},
        # one token, biased sigmoid scores in groups
        {"name": "route_one", "op": "route", "t": 1, "e": 256, "k": 8, "groups": 8, "top_groups": 4, "best": 2,
         "sigmoid": True, "bias": True, "renorm": True, "half": False},
        # a decode batch, softmax scores of 16-bit logits, experts masked out among them
        {"name": "route_batch", "op": "route", "t": 61, "e": 128, "k": 8, "groups": 1, "top_groups": 1, "best": 1,
         "sigmoid": False, "bias": False, "renorm": False, "half": True},
        # a long prompt of odd length
        {"name": "route_prompt", "op": "route", "t": 16385, "e": 256, "k": 8, "groups": 8, "top_groups": 4, "best": 2,
         "sigmoid": True, "bias": True, "renorm": True, "half": False},
        # one request with three drafted tokens
        {"name": "verify_one", "op": "verify", "b": 1, "lo": 3, "hi": 3, "v": 32000, "half": False, "sure": False, "cut": False},
        # a ragged batch, drafts looked up (without probabilities) in 16 bits, sequences without any among them
        {"name": "verify_batch", "op": "verify", "b": 61, "lo": 0, "hi": 7, "v": 32768, "half": True, "sure": True, "cut": False},
        # the largest batch on a large vocabulary of odd size, unlikely tokens cut off
        {"name": "verify_large", "op": "verify", "b": 64, "lo": 5, "hi": 5, "v": 131071, "half": False, "sure": False, "cut": True},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "lora", "route", "verify"])
    if op == "norm":
        h = GROUP * _log(rng, 2, 19968 // GROUP)
        return {"op": op, "t": _log(rng, 1, max(1, min(65536, 16383 * 4096 // h))), "h": h, "x32": rng.random() < 0.2,
                "res": rng.choice(["none", "bf16", "bf16", "f32"]), "out": rng.choice(["bf16", "row", "group"])}
    if op == "lora":
        m, r = _log(rng, 1, 64), rng.choice([8, 16, 16, 24, 32, 64, 128])
        adapters = _log(rng, 1, 64)
        k = 256 * _log(rng, 4, 78)
        n = _log(rng, 64, min(39936, max(64, 64 * 64 * 46592 // (min(m, adapters) * r) - k)))
        return {"op": op, "m": m, "k": k, "n": n, "r": r, "adapters": adapters, "plain": rng.randrange(0, m // 4 + 1),
                "y32": rng.random() < 0.3}
    if op == "route":
        e = rng.choice([8, 16, 60, 64, 128, 160, 256, 384, 512])
        groups = 1 if e == 60 or rng.random() < 0.4 else rng.choice([2, 4, 8])
        top = rng.randrange(1, groups + 1)
        return {"op": op, "t": _log(rng, 1, max(1, 16385 * 256 // e)), "e": e, "k": _log(rng, 1, min(16, e // groups * top)),
                "groups": groups, "top_groups": top, "best": rng.choice([1, 2]) if e // groups > 1 else 1,
                "sigmoid": rng.random() < 0.6, "bias": rng.random() < 0.6, "renorm": rng.random() < 0.6,
                "half": rng.random() < 0.4}
    b, v = _log(rng, 1, 64), _log(rng, 1000, 131071)
    hi = rng.randrange(0, 9)
    hi = min(hi, 64 * 6 * 131071 // (b * v) - 1)
    return {"op": op, "b": b, "lo": rng.randrange(0, hi + 1), "hi": hi, "v": v, "half": rng.random() < 0.3,
            "sure": rng.random() < 0.3, "cut": rng.random() < 0.5}


def _drafts(c):
    """Drafted tokens of each sequence, evenly from lo to hi (hi alone for one sequence)."""
    return [c["hi"]] if c["b"] == 1 else [c["lo"] + i * (c["hi"] - c["lo"]) // (c["b"] - 1) for i in range(c["b"])]


def _in_use(c):
    """Adapters that the rows of a batch name."""
    return min(c["adapters"], c["m"] - c["plain"])


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["t"] * c["h"]
        stream = {"none": 0, "bf16": 4, "f32": 8}[c["res"]]
        out = {"bf16": 2 * n, "row": n + 4 * c["t"], "group": n + n // GROUP * 4}[c["out"]]
        return {"bytes": n * ((4 if c["x32"] else 2) + stream) + 2 * c["h"] + out, "flops": n * (5 if c["out"] == "bf16" else 8)}
    if c["op"] == "lora":
        held = _in_use(c) * c["r"] * (c["k"] + c["n"]) * 2
        rows = c["m"] - c["plain"]
        return {"bytes": held + c["m"] * (c["k"] * 2 + c["n"] * (8 if c["y32"] else 4)),
                "flops": 2 * rows * c["r"] * (c["k"] + c["n"])}
    if c["op"] == "route":
        n = c["t"] * c["e"]
        return {"bytes": n * (2 if c["half"] else 4) + 8 * c["t"] * c["k"], "flops": 8 * n}
    rows = 1 if c["sure"] else 2
    return {"bytes": c["b"] * c["v"] * rows * (2 if c["half"] else 4) + 16 * sum(_drafts(c)), "flops": 3 * c["b"] * c["v"]}


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"case": c}

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    if c["op"] == "norm":
        x = randn(c["t"], c["h"])
        x[:, 7 % c["h"]] *= 20   # a channel that stands out, as hidden states have
        s["x"] = x if c["x32"] else x.to(torch.bfloat16)
        s["weight"] = (1 + 0.2 * randn(c["h"])).to(torch.bfloat16)
        s["residual"] = None if c["res"] == "none" else 4 * randn(c["t"], c["h"])
        if c["res"] == "bf16":
            s["residual"] = s["residual"].to(torch.bfloat16)
    elif c["op"] == "lora":
        s["x"] = randn(c["m"], c["k"]).to(torch.bfloat16)
        y = randn(c["m"], c["n"])                                          # the shared projection's output
        s["y"] = y if c["y32"] else y.to(torch.bfloat16)
        s["a"] = (randn(c["adapters"], c["r"], c["k"]) * c["k"] ** -0.5).to(torch.bfloat16)
        s["b"] = (randn(c["adapters"], c["n"], c["r"]) * c["r"] ** -0.5).to(torch.bfloat16)
        s["scales"] = 0.2 + 0.3 * torch.rand(c["adapters"], generator=g, device=dev)
        order = torch.randperm(c["adapters"], generator=g, device=dev)     # the adapters in use are any of those held
        ids = order[torch.arange(c["m"], device=dev) % _in_use(c)]
        ids[c["m"] - c["plain"]:] = -1                                     # requests without an adapter
        s["ids"] = ids[torch.randperm(c["m"], generator=g, device=dev)].to(torch.int32)
    elif c["op"] == "route":
        l = 2 * randn(c["t"], c["e"])
        if not c["sigmoid"]:   # an expert that is down
            l[:, int(torch.randint(0, c["e"], (1,), generator=g, device=dev))] = -torch.inf
        s["logits"] = l.to(torch.bfloat16) if c["half"] else l
        s["bias"] = 0.1 * randn(c["e"]) if c["bias"] else None
    else:
        counts = _drafts(c)
        rows = sum(counts) + c["b"]
        cu = [0]
        for n in counts:
            cu.append(cu[-1] + n + 1)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        row = torch.tensor([cu[i] + j for i, n in enumerate(counts) for j in range(n)], dtype=torch.int64, device=dev)
        logits = 3 * randn(rows, c["v"])

        def probabilities(z):
            p = torch.softmax(z, 1)
            if c["cut"]:
                p = torch.where(p >= 2e-2 / c["v"], p, 0.0)
                p /= p.sum(1, keepdim=True)
            return p.to(torch.bfloat16) if c["half"] else p

        s["target"] = probabilities(logits)
        z = logits[row] + randn(len(row), c["v"])                          # a draft model that mostly agrees
        q = probabilities(z)
        noise = -torch.log(torch.rand(q.shape, generator=g, device=dev).clamp_min(1e-30))
        s["tokens"] = (q.float() / noise).argmax(1).to(torch.int32) if len(row) else torch.zeros(0, dtype=torch.int32, device=dev)
        s["draft"] = None if c["sure"] else q
        s["u"] = torch.rand(len(row), generator=g, device=dev)
        s["u_next"] = torch.rand(c["b"], generator=g, device=dev)
    return s


def run(state):
    s, c = state, state["case"]
    if own:
        import gemm_decode_qgemm_amd as qg
        if c["op"] == "norm":
            if c["out"] == "bf16":
                return qg.rms_norm(s["x"], s["weight"], residual=s["residual"])
            codes, scales, *r = qg.rms_norm_q8(s["x"], s["weight"], residual=s["residual"], group_scales=c["out"] == "group")
            values = torch.empty(s["x"].shape, dtype=torch.bfloat16, device=s["x"].device)
            wide = (c["t"], -1, GROUP) if c["out"] == "group" else (c["t"], 1, c["h"])
            torch.mul(codes.view(wide), scales.view(c["t"], -1, 1), out=values.view(wide))
            return (values, *r)
        if c["op"] == "lora":
            return qg.lora_add(s["y"], s["x"], s["a"], s["b"], s["ids"], scales=s["scales"])
        if c["op"] == "route":
            return qg.moe_route(s["logits"], c["k"], sigmoid=c["sigmoid"], bias=s["bias"], groups=c["groups"],
                                top_groups=c["top_groups"], group_best=c["best"], renormalize=c["renorm"], scale=2.5)
        return qg.verify_drafts(s["target"], s["draft"], s["tokens"], s["u"], s["u_next"], s["cu"])
    return {"norm": _plain_norm, "lora": _plain_lora, "route": _plain_route, "verify": _plain_verify}[c["op"]](s, c)


# ---- the plain forms ---------------------------------------------------------

def _plain_norm(s, c):
    x = s["x"].float()
    if s["residual"] is not None:
        x = x + s["residual"].float()
    y = x * torch.rsqrt((x * x).mean(1, keepdim=True) + 1e-6) * s["weight"].float()
    if c["out"] != "bf16":
        wide = y.view(c["t"], -1, GROUP) if c["out"] == "group" else y[:, None]
        scale = wide.abs().amax(2, keepdim=True) / 127
        y = ((wide / scale).round().clamp(-127, 127) * scale).view(c["t"], c["h"])
    y = y.to(torch.bfloat16)
    return y if s["residual"] is None and c["out"] == "bf16" else (y,) if s["residual"] is None else (y, x.to(s["residual"].dtype))


def _plain_lora(s, c):
    ids = s["ids"].long()
    at = ids.clamp_min(0)
    v = torch.matmul(s["a"][at].float(), s["x"].float()[..., None])        # [m, r, 1]
    add = torch.matmul(s["b"][at].float(), v)[..., 0] * s["scales"][at][:, None]
    return (s["y"].float() + torch.where(ids[:, None] >= 0, add, 0.0)).to(s["y"].dtype)


def _plain_route(s, c):
    l = s["logits"].double()
    if c["sigmoid"]:
        score = 1 / (1 + torch.exp(-l))
    else:
        score = torch.exp(l - l.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    choice = score + s["bias"].double() if s["bias"] is not None else score
    if c["groups"] > 1:
        g = choice.view(c["t"], c["groups"], -1)
        rank = torch.sort(g, dim=2, descending=True).values[..., :c["best"]].sum(2)
        kept = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        open_ = torch.zeros(rank.shape, dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        choice = torch.where(open_[..., None], g, -torch.inf).view(c["t"], c["e"])
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    w = torch.gather(score, 1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return ids.to(torch.int32), (2.5 * w).float()


def _plain_verify(s, c):
    b, cu, dev = c["b"], s["cu"].long(), s["cu"].device
    n, most = cu[1:] - cu[:-1] - 1, max(1, c["hi"])
    i = torch.arange(most, device=dev)
    seq = torch.arange(b, device=dev)
    drafted = cu[:-1, None] - seq[:, None] + i                             # rows of the draft's tensors [b, most]
    drafted = drafted.clamp(max=max(0, s["u"].shape[0] - 1))
    first = torch.zeros(b, dtype=torch.int64, device=dev)
    if s["u"].shape[0]:
        x = s["tokens"].long()[drafted]
        p = s["target"][(cu[:-1, None] + i).clamp(max=s["target"].shape[0] - 1), x].double()
        q = s["draft"][drafted, x].double() if s["draft"] is not None else torch.ones_like(p)
        ok = (s["u"][drafted].double() * q < p) & (i < n[:, None])
        first = ok.long().cumprod(1).sum(1)
    row = s["target"][cu[:-1] + first].double()
    left = row
    if s["u"].shape[0]:
        at = (cu[:-1] - seq + first).clamp(max=s["u"].shape[0] - 1)
        if s["draft"] is not None:
            other = s["draft"][at].double()
        else:
            other = torch.zeros_like(row).scatter_(1, s["tokens"].long()[at][:, None], torch.inf)
        left = torch.where((first < n)[:, None], (row - other).clamp_min(0), row)
    total = left.cumsum(1)
    token = (total <= s["u_next"].double()[:, None] * total[:, -1:]).sum(1)
    return first.to(torch.int32), token.to(torch.int32)


# ---- the definitions in 64 bits ------------------------------------------------

def _exact_norm(s, c):
    r = s["x"].double()
    if s["residual"] is not None:
        r = r + s["residual"].double()
    y = r / (r.pow(2).sum(1, keepdim=True) / c["h"] + 1e-6).sqrt() * s["weight"].double()
    if c["out"] != "bf16":
        y = y.unflatten(1, (-1, GROUP if c["out"] == "group" else c["h"]))
        step = torch.linalg.vector_norm(y, torch.inf, dim=2, keepdim=True) / 127
        y = (torch.round(y / step) * step).flatten(1)
    return (y if c["out"] == "bf16" else (y,)) if s["residual"] is None else (y, r)


def _exact_lora(s, c):
    out, x = s["y"].double(), s["x"].double()
    for a in s["ids"].unique().tolist():
        if a >= 0:
            rows = (s["ids"] == a).nonzero()[:, 0]
            low = torch.matmul(x[rows], s["a"][a].double().t())
            out[rows] += s["scales"][a].double() * torch.matmul(low, s["b"][a].double().t())
    return out


def _exact_route(s, c):
    l, e, per = s["logits"].double(), c["e"], c["e"] // c["groups"]
    score = torch.sigmoid(l) if c["sigmoid"] else torch.softmax(l, 1)
    left = score.clone() if s["bias"] is None else score + s["bias"].double()
    if c["groups"] > 1:
        value = torch.stack([left[:, i * per:(i + 1) * per].topk(c["best"], 1).values.sum(1) for i in range(c["groups"])], 1)
        for _ in range(c["groups"] - c["top_groups"]):                     # the worst group goes, the last of equal ones
            worst = c["groups"] - 1 - value.flip(1).argmin(1)
            value.scatter_(1, worst[:, None], torch.inf)
            left[(torch.arange(e, device=l.device) // per)[None] == worst[:, None]] = -torch.inf
    ids, w = [], []
    for _ in range(c["k"]):
        best = (left == left.amax(1, keepdim=True)).to(torch.uint8).argmax(1, keepdim=True)
        ids.append(best)
        w.append(score.gather(1, best))
        left.scatter_(1, best, -torch.inf)
    w = torch.cat(w, 1)
    return torch.cat(ids, 1).to(torch.int32), 2.5 * (w / w.sum(1, keepdim=True) if c["renorm"] else w)


def _exact_verify(s, c):
    taken, following, at = [], [], 0
    tokens, u = s["tokens"].tolist(), s["u"].tolist()
    for i, n in enumerate(_drafts(c)):
        first, j = int(s["cu"][i]), 0
        while j < n:
            p = float(s["target"][first + j, tokens[at + j]])
            q = 1.0 if s["draft"] is None else float(s["draft"][at + j, tokens[at + j]])
            if not u[at + j] * q < p:
                break
            j += 1
        left = s["target"][first + j].double()
        if j < n and s["draft"] is None:
            left[tokens[at + j]] = 0
        elif j < n:
            left = torch.relu(left - s["draft"][at + j].double())
        sums = left.cumsum(0)
        taken.append(j)
        following.append(int(torch.searchsorted(sums, s["u_next"][i].double() * sums[-1], right=True)))
        at += n
    dev = s["cu"].device
    return torch.tensor(taken, dtype=torch.int32, device=dev), torch.tensor(following, dtype=torch.int32, device=dev)


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "lora": _exact_lora, "route": _exact_route, "verify": _exact_verify}[case["op"]](s, case)
