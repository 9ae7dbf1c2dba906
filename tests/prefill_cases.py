"""Ragged prefill batches for the tests: seeded inputs and a plain 64-bit reference with its error bound.

Slots and table entries that hold no token are poison (NaN, ids outside the pool).
"""
from __future__ import annotations

import math
from dataclasses import dataclass

import numpy as np
import torch

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@dataclass
class Batch:
    q: torch.Tensor             # [T, Hq, d]
    kc: torch.Tensor            # [NB, bs, Hkv, d] (uint8 codes when the scales are set)
    vc: torch.Tensor
    tables: torch.Tensor        # int32 [B, W]
    lens: torch.Tensor          # int32 [B]
    starts: torch.Tensor        # int32 [B + 1]
    scale: float
    max_len: int
    k_scale: torch.Tensor | None = None
    v_scale: torch.Tensor | None = None

    def to(self, device):
        f = lambda t: t.to(device) if isinstance(t, torch.Tensor) else t
        return Batch(*(f(getattr(self, n)) for n in self.__dataclass_fields__))

    def dense(self, s, pool, scale):
        """Sequence s's rows of a pool by position, float64 [L, Hkv, d]."""
        bs, L = pool.shape[1], int(self.lens[s])
        ids = self.tables[s, :-(-L // bs)].long()
        x = pool[ids].flatten(0, 1)[:L]
        if scale is None:
            return x.double()
        return x.view(torch.float8_e4m3fn).double() * scale.double()[None, :, None]


def build(news, totals, heads, kv_heads, dim, block, dtype="bf16", seed=0, scale=None, pad_rows=0, gap=0, e4m3=False):
    """news[s] new tokens at the end of totals[s] positions (a total below its new tokens leaves tokens
    that see nothing); ``gap`` unowned rows before the first sequence, ``pad_rows`` after the last."""
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    need = [-(-t // block) for t in totals]
    NB = sum(need) + 3
    order = torch.randperm(NB, generator=g).int()
    W = max(need + [1]) + 2
    tables = torch.full((len(totals), W), NB + 7, dtype=torch.int32)
    tables[:, -1] = np.iinfo(np.int32).max
    kf = torch.full((NB, block, kv_heads, dim), math.nan)
    vf = torch.full((NB, block, kv_heads, dim), math.nan)
    at = 0
    for s, (t, n) in enumerate(zip(totals, need)):
        ids = order[at:at + n]
        at += n
        tables[s, :n] = ids
        for p in (kf, vf):
            x = torch.full((n * block, kv_heads, dim), math.nan)
            x[:t] = torch.randn(t, kv_heads, dim, generator=g)
            p[ids.long()] = x.view(n, block, kv_heads, dim)
    starts = [gap]
    for n in news:
        starts.append(starts[-1] + n)
    q = torch.randn(starts[-1] + pad_rows, heads, dim, generator=g).to(dt)
    ks = vs = None
    if e4m3:
        ks = torch.rand(kv_heads, generator=g) * 0.02 + 0.01
        vs = torch.rand(kv_heads, generator=g) * 0.02 + 0.01
        kc = (kf / ks[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        vc = (vf / vs[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        kc, vc = kf.to(dt), vf.to(dt)
    return Batch(q, kc, vc, tables, torch.tensor(totals, dtype=torch.int32), torch.tensor(starts, dtype=torch.int32),
                 1.0 / math.sqrt(dim) if scale is None else scale, max(totals + [0]), ks, vs)


def reference(b: Batch, work_dtype=None):
    """(out, bound) in float64, [T, Hq, d], NaN where no sequence owns the row.

    bound, per element, counts every rounding of the kernel with A = sum_t p_t |V_t|:
      * each weight rounded to the work type T (half a step, h = eps(T) / 2, relative; below T's normal
        range, which only fp16 reaches, half its smallest step 2^-25 of a sum of weights that is at
        least 1):                                                    h A + 2^-25 sum_t |V_t| / l
      * the output rounded to T:                                     h |out| + 2^-25
      * fp32 accumulation (each addition off by a step, 2^-23, of the running sum of magnitudes): the
        scores' d terms move a weight by 2 (d + 4) 2^-23 scale max_t sum_i |q_i K_ti| relative, the
        weighted sum's additions (one per 16 positions and a rescale now and then) by (L / 16 + 64) 2^-23,
        exp2 and the division by 2^-20 between them.
    """
    T, Hq, d = b.q.shape
    Hkv = b.kc.shape[2]
    G = Hq // Hkv
    h = torch.finfo(b.q.dtype if work_dtype is None else work_dtype).eps / 2
    ho = torch.finfo(b.q.dtype).eps / 2
    out = torch.full((T, Hq, d), math.nan, dtype=torch.float64)
    bound = torch.full_like(out, math.nan)
    for s in range(len(b.lens)):
        r0, r1, L = int(b.starts[s]), int(b.starts[s + 1]), int(b.lens[s])
        n = r1 - r0
        if n == 0:
            continue
        K, V = b.dense(s, b.kc, b.k_scale), b.dense(s, b.vc, b.v_scale)
        lim = L - n + 1 + torch.arange(n)
        for hq in range(Hq):
            q = b.q[r0:r1, hq].double()
            k, v = K[:, hq // G], V[:, hq // G]
            seen = torch.arange(L)[None, :] < lim[:, None]
            z = torch.where(seen, (q @ k.T) * b.scale, -math.inf)
            mag = torch.where(seen, (q.abs() @ k.abs().T) * abs(b.scale), 0.0).amax(1, keepdim=True) if L else \
                torch.zeros(n, 1, dtype=torch.float64)
            top = z.amax(1, keepdim=True) if L else torch.zeros(n, 1, dtype=torch.float64)
            w = torch.where(seen, torch.exp(z - top), 0.0)
            l = w.sum(1, keepdim=True).clamp(min=1e-300)
            o = (w @ v) / l
            A = (w @ v.abs()) / l
            o[lim <= 0] = 0.0
            out[r0:r1, hq] = o
            flat = (seen.double() @ v.abs()) / l
            acc = 2 * (d + 4) * 2.0 ** -23 * mag + (L / 16 + 64) * 2.0 ** -23 + 2.0 ** -20
            err = h * A + 2.0 ** -25 * flat * (h < 2.0 ** -9) + acc * A
            bound[r0:r1, hq] = err + ho * (o.abs() + err) + 2.0 ** -25
    return out, bound


def check(got, ref, bound, what=""):
    """Owned rows within the bound, the others untouched by the caller's NaN fill."""
    got = got.double().cpu()
    owned = ~torch.isnan(bound)
    assert torch.isnan(got[~owned]).all(), f"{what}: a row of no sequence was written"
    assert not torch.isnan(got[owned]).any(), f"{what}: NaN in an output"
    over = (got - ref).abs()[owned] / bound[owned]
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 1.0, f"{what}: error {worst:.3f} of the bound"
    return worst
