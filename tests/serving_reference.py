"""Plain 64-bit forms of the serving-step operators.  Test infrastructure: shares
no code with the kernels."""
from __future__ import annotations

import numpy as np
import torch


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def half_step(ref: np.ndarray, bits: int) -> np.ndarray:
    """Half a unit in the last place at ref of a type with `bits` significant bits."""
    _, e = np.frexp(np.maximum(np.abs(ref), np.finfo(np.float32).tiny))
    return np.ldexp(1.0, e - bits - 1)


def rms_norm(x, res, w, eps):
    """(y, r) of rows in 64 bits."""
    r = x if res is None else x + res
    y = r / np.sqrt(np.mean(r * r, 1, keepdims=True) + eps)
    return (y if w is None else y * w), r


def lora(y, x, a, b, ids, scales):
    out = y.copy()
    for m, i in enumerate(ids):
        if i >= 0:
            out[m] += (1.0 if scales is None else scales[i]) * (b[i] @ (a[i] @ x[m]))
    return out


def route(l, k, sigmoid, bias, groups, top_groups, best, renorm, scale):
    """(ids, weights) one token at a time, by sorting (value, -index) pairs."""
    t, e = l.shape
    ids, weights = np.zeros((t, k), np.int64), np.zeros((t, k))
    per = e // groups
    for i in range(t):
        with np.errstate(all="ignore"):
            if sigmoid:
                s = 1.0 / (1.0 + np.exp(-l[i]))
            elif np.all(l[i] == -np.inf):
                s = np.zeros(e)
            else:
                s = np.exp(l[i] - np.max(l[i]))
                s = s / s.sum()
        # sigmoid and softmax keep the order of the logits, which decide where neither a bias nor a sum takes part;
        # a NaN (of an infinite logit in a softmax, too) is above all numbers
        c = l[i] if bias is None and (groups == 1 or best == 1) else s if bias is None else s + bias
        pairs = [(bool(np.isnan(c[j])), 0.0 if np.isnan(c[j]) else c[j], -j) for j in range(e)]
        value = []
        for g in range(groups):
            top = sorted(pairs[g * per:(g + 1) * per], reverse=True)[:best]
            value.append((any(p[0] for p in top), sum(p[1] for p in top) if not any(p[0] for p in top) else 0.0, -g))
        kept = {-v[2] for v in sorted(value, reverse=True)[:top_groups]}
        order = sorted((p for p in pairs if -p[2] // per in kept), reverse=True)[:k]
        ids[i] = [-p[2] for p in order]
        w = s[ids[i]]
        if renorm:
            w = w / w.sum() if w.sum() != 0 else np.zeros(k)
        weights[i] = scale * w
    return ids, weights


def verify(target, draft, tokens, u, u_next, cu):
    """(accepted, next) with rows as lists; draft None: certain drafts."""
    accepted, following = [], []
    for b in range(len(cu) - 1):
        n = cu[b + 1] - cu[b] - 1
        j = 0
        while j < n:
            d = cu[b] - b + j
            x = tokens[d]
            inside = 0 <= x < target.shape[1]
            q = (1.0 if draft is None else draft[d, x]) if inside else 0.0
            p = target[cu[b] + j, x] if inside else 0.0
            if not u[d] * q < p:
                break
            j += 1
        row = np.nan_to_num(np.maximum(target[cu[b] + j], 0.0), nan=0.0, posinf=np.inf)
        left = row
        if j < n:
            d = cu[b] - b + j
            if draft is None:
                left = row.copy()
                if 0 <= tokens[d] < row.size:
                    left[tokens[d]] = 0.0
            else:
                with np.errstate(invalid="ignore"):
                    left = np.nan_to_num(np.maximum(target[cu[b] + j] - draft[d], 0.0), nan=0.0, posinf=np.inf)
            if left.sum() == 0:
                left = row
        sums = np.cumsum(left)
        accepted.append(j)
        if not 0 < sums[-1] < np.inf:
            following.append(-1)
        else:
            above = np.nonzero(sums > u_next[b] * sums[-1])[0]
            following.append(int(above[0]) if above.size else int(np.nonzero(left)[0][-1]))
    return accepted, following
