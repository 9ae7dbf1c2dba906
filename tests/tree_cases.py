"""Drafted trees for the tests: masks over prefill_cases' ragged batches, and the plain 64-bit reference with its bound."""
from __future__ import annotations

import math
import random

import torch


def tree(r: random.Random, n, chain=0.5):
    """Parents of a random tree of n nodes, each after its parent: a chain's next with probability ``chain``."""
    return [-1] + [i - 1 if r.random() < chain else r.randrange(i) for i in range(1, n)]


def ancestors(parents):
    """Mask words of a tree: bit j of word i where j is i or an ancestor of i."""
    words = []
    for i, p in enumerate(parents):
        words.append(1 << i | (words[p] if p >= 0 else 0))
    return words


def signed(words):
    return [w - (1 << 64) if w >> 63 else w for w in words]


def masks(news, seed, gap=0, pad_rows=0, chain=0.5):
    """(int64 [T] masks of random trees of news[s] nodes, rows of no sequence all ones; the parents)."""
    r = random.Random(seed)
    trees = [tree(r, n, chain) if n else [] for n in news]
    words = [(1 << 64) - 1] * gap + [w for t in trees for w in ancestors(t)] + [(1 << 64) - 1] * pad_rows
    return torch.tensor(signed(words), dtype=torch.int64), trees


def seen_of(b, mask, s):
    """[n, L] of sequence s: what each node sees."""
    r0, r1, L = int(b.starts[s]), int(b.starts[s + 1]), int(b.lens[s])
    n = r1 - r0
    seen = torch.zeros(n, L, dtype=torch.bool)
    base = L - n
    for i in range(n):
        if base > 0:
            seen[i, :base] = True
        word = int(mask[r0 + i])
        for j in range(i + 1):
            if word >> j & 1 and base + j >= 0:
                seen[i, base + j] = True
    return seen


def reference(b, mask, work_dtype=None):
    """(out, bound) in float64, [T, Hq, d], NaN where no sequence owns the row.

    The roundings are those of the prefill reference (prefill_cases.reference), whose bound is used as derived there:
    with A = sum_t p_t |V_t|, h = eps(T) / 2 of the type the weights round to, ho of the output's,
        h A + 2^-25 sum_t |V_t| / l                            weights (the second term where T is fp16)
        ho |out| + 2^-25                                       output
        (2 (d + 4) 2^-23 scale max_t sum_i |q_i K_ti| + (L / 16 + 64) 2^-23 + 2^-20) A     fp32 accumulation
    """
    T, Hq, d = b.q.shape
    G = Hq // b.kc.shape[2]
    h = torch.finfo(b.q.dtype if work_dtype is None else work_dtype).eps / 2
    ho = torch.finfo(b.q.dtype).eps / 2
    out = torch.full((T, Hq, d), math.nan, dtype=torch.float64)
    bound = torch.full_like(out, math.nan)
    for s in range(len(b.lens)):
        r0, r1, L = int(b.starts[s]), int(b.starts[s + 1]), int(b.lens[s])
        if r1 == r0:
            continue
        K, V = b.dense(s, b.kc, b.k_scale), b.dense(s, b.vc, b.v_scale)
        seen = seen_of(b, mask, s)
        none = ~seen.any(1)
        for hq in range(Hq):
            q = b.q[r0:r1, hq].double()
            k, v = K[:, hq // G], V[:, hq // G]
            z = torch.where(seen, (q @ k.T) * b.scale, -math.inf)
            mag = torch.where(seen, (q.abs() @ k.abs().T) * abs(b.scale), 0.0)
            mag = mag.amax(1, keepdim=True) if L else torch.zeros(r1 - r0, 1, dtype=torch.float64)
            top = z.amax(1, keepdim=True) if L else torch.zeros(r1 - r0, 1, dtype=torch.float64)
            w = torch.where(seen, torch.exp(z - top), 0.0)
            l = w.sum(1, keepdim=True).clamp(min=1e-300)
            o, A = (w @ v) / l, (w @ v.abs()) / l
            o[none] = 0.0
            out[r0:r1, hq] = o
            flat = (seen.double() @ v.abs()) / l
            acc = 2 * (d + 4) * 2.0 ** -23 * mag + (L / 16 + 64) * 2.0 ** -23 + 2.0 ** -20
            err = h * A + 2.0 ** -25 * flat * (h < 2.0 ** -9) + acc * A
            err[none] = 0.0
            bound[r0:r1, hq] = err + ho * (o.abs() + err) + 2.0 ** -25
    return out, bound
