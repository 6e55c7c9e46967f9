"""Plain 64-bit forms of the decoder-layer operators, and their layouts spelled
out one token at a time (include/qgemm.h).  Test infrastructure: shares no code
with the kernels."""
from __future__ import annotations

import math

import numpy as np
import torch

PAGE, BLOCK = 64, 16


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def half_ulp_bf16(ref: np.ndarray) -> np.ndarray:
    """Half a unit in the last place of bf16 (8 significant bits) at ref."""
    _, e = np.frexp(np.maximum(np.abs(ref), np.finfo(np.float32).tiny))
    return np.ldexp(1.0, e - 9)


# ---- head norm and rotation ---------------------------------------------------

def norm_rope(x, w, cos_sin, positions, eps, pairs):
    """x [tokens, heads, d] f64 -> f64."""
    out = np.empty_like(x)
    rot = cos_sin.shape[1]
    half = rot // 2
    for t in range(x.shape[0]):
        for h in range(x.shape[1]):
            v = x[t, h] / math.sqrt(float(np.mean(x[t, h] ** 2)) + eps)
            if w is not None:
                v = v * w
            y = v.copy()
            for i in range(half):
                c, s = cos_sin[positions[t], i], cos_sin[positions[t], half + i]
                a, b = (2 * i, 2 * i + 1) if pairs else (i, half + i)
                y[a], y[b] = v[a] * c - v[b] * s, v[b] * c + v[a] * s
            out[t, h] = y
    return out


# ---- the 8-bit cache -----------------------------------------------------------

def value_offset(c: int, t: int) -> int:
    """Byte of channel c of token t among a page's values."""
    return 64 * c + 16 * ((t % 16) // 4) + 4 * (t // 16) + t % 4


class Cache:
    """The cache in host memory, appended to one block at a time in binary32."""

    def __init__(self, pages, hkv, d, table):
        self.codes = np.zeros((pages, hkv, 2, PAGE * d), np.int8)
        self.scales = np.zeros((pages, hkv, 2, PAGE // BLOCK), np.float32)
        self.table, self.hkv, self.d = table, hkv, d
        self.voff = np.array([[value_offset(c, t) for c in range(d)] for t in range(PAGE)])

    def offsets(self, which, t):
        """Bytes of the channels of token t of a page."""
        return self.voff[t] if which else t * self.d + np.arange(self.d)

    def append(self, b, old, rows_k, rows_v):
        """Rows [n, hkv, d] float32 become tokens old .. old + n of sequence b."""
        n = rows_k.shape[0]
        for which, rows in ((0, rows_k), (1, rows_v)):
            for h in range(self.hkv):
                for blk in range(old // BLOCK, (old + n + BLOCK - 1) // BLOCK):
                    lo, hi = max(old, blk * BLOCK), min(old + n, (blk + 1) * BLOCK)
                    page, at = self.table[b][blk * BLOCK // PAGE], blk % 4
                    new = rows[lo - old:hi - old, h]
                    held = self.scales[page, h, which, at] if lo > blk * BLOCK else np.float32(0)
                    code = self.codes[page, h, which]
                    if not np.isfinite(new).all() or np.isnan(held):
                        s = np.float32(np.nan)
                    else:
                        s = max(held, np.float32(np.abs(new).max() * np.float32(1.0 / 127.0)))
                        if s > held and lo > blk * BLOCK:
                            f = np.float32(held / s)
                            for t in range(blk * BLOCK, lo):
                                o = self.offsets(which, t % PAGE)
                                code[o] = np.rint(code[o].astype(np.float32) * f).astype(np.int8)
                    for t in range(lo, hi):
                        o = self.offsets(which, t % PAGE)
                        if s > 0:
                            code[o] = np.clip(np.rint((rows[t - old, h] / s).astype(np.float32)), -127, 127).astype(np.int8)
                        else:
                            code[o] = 0
                    self.scales[page, h, which, at] = s

    def token(self, b, t, h, which):
        page = self.table[b][t // PAGE]
        return self.codes[page, h, which][self.offsets(which, t % PAGE)], self.scales[page, h, which, t % PAGE // BLOCK]

    def values(self, b, n, which):
        """[n, hkv, d] in 64 bits."""
        out = np.zeros((n, self.hkv, self.d))
        for t in range(n):
            for h in range(self.hkv):
                q, s = self.token(b, t, h, which)
                out[t, h] = q.astype(np.float64) * np.float64(s)
        return out


def attention(q, k, v, length, scale, window):
    """q [nq, hq, d], k and v [length, hkv, d] in 64 bits -> (out, sum of p |v|)."""
    nq, hq, d = q.shape
    out, mass = np.zeros((nq, hq, d)), np.zeros((nq, hq, d))
    group = hq // k.shape[1]
    for t in range(nq):
        end = length - nq + t + 1
        first = max(0, end - window) if window > 0 else 0
        if end <= first:
            continue
        for h in range(hq):
            kk, vv = k[first:end, h // group], v[first:end, h // group]
            s = kk @ q[t, h] * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            out[t, h], mass[t, h] = p @ vv, p @ np.abs(vv)
    return out, mass


# ---- mixture of experts --------------------------------------------------------

def pick(logits: np.ndarray, top: int) -> np.ndarray:
    """Experts of each token, best first; ties go to the lowest index."""
    return np.stack([np.lexsort((np.arange(r.size), -r))[:top] for r in logits])


def moe(x, router, gate_up, down, inter, top, renormalize):
    """x [t, h], router [e, h], gate_up [e][2 inter, h], down [e][h, inter] in 64
    bits -> (y, bound): bound is the sum of the absolute terms behind each y."""
    logits = x @ router.T
    ids = pick(logits, top)
    y, bound = np.zeros_like(x), np.zeros_like(x)
    for t in range(x.shape[0]):
        l = logits[t] - logits[t].max()
        p = np.exp(l)
        p /= p[ids[t]].sum() if renormalize else p.sum()
        for e in ids[t]:
            gu = gate_up[e] @ x[t]
            g, u = gu[:inter], gu[inter:]
            a = g / (1 + np.exp(-g)) * u
            y[t] += p[e] * (down[e] @ a)
            bound[t] += p[e] * (np.abs(down[e]) @ np.abs(a))
    return y, bound
