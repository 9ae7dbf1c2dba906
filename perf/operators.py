"""Workloads of the prefill, cache read-back and draft acceptance operators.

Each case is one call a serving loop makes: the attention of a step's new
tokens over the paged cache (``paged_attention_prefill``: prompts, chunks of a
prompt over what is already cached, and running sequences that add one token,
in one ragged batch), the read-back of a cache into dense 16-bit rows
(``paged_kv_gather``), and the acceptance of drafted tokens against the
target's probabilities (``speculative_accept``).

With ``own`` false, ``run`` computes the operators from elementary torch
operations in 32 bits (whole-number sums in 64), rounded once at the end; with
``own`` true it calls the library.  ``exact`` computes them once more from their
definitions in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"f16": 2, "bf16": 2, "f32": 4, "e4m3": 1}
# A final draw sums its weights as whole numbers of this unit (2^-44).
_UNIT = float(1 << 44)


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _prefill(name, dtype, kv, heads, kv_heads, dim, block, **lens):
    return {"name": name, "op": "prefill", "dtype": dtype, "kv": kv, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "block": block, **lens}


def listed():
    return [
        # The smallest step: four short sequences of a small model, some of them one token. Latency.
        _prefill("prefill_small_step", "f16", "f16", 4, 4, 64, 16, news="1,17,5,2", totals="1,17,33,50"),
        # Chunked prefill: eight prompts, 512 new tokens each, over 512 to 4096 tokens cached before.
        _prefill("prefill_chunks_over_prefix", "bf16", "bf16", 32, 8, 128, 16, seqs=8, new_lo=512, new_hi=512,
                 old_lo=512, old_hi=4096, singles=0, lens_seed=1),
        # A mixed step: sixty sequences that decode one token beside four prompt chunks.
        _prefill("prefill_mixed_with_decode", "bf16", "bf16", 32, 8, 128, 16, seqs=64, new_lo=300, new_hi=700,
                 old_lo=511, old_hi=4095, singles=60, lens_seed=2),
        # A long prompt from an empty cache, 64 query heads over 8 KV heads.
        _prefill("prefill_long_prompt", "f16", "f16", 64, 8, 128, 16, news="8192", totals="8192"),
        # The last few tokens of one very long prompt: little to compute, a long cache to read.
        _prefill("prefill_few_rows_long_context", "bf16", "bf16", 64, 8, 128, 32, news="33", totals="65549"),
        # Ragged prompts of a small model: three query heads per KV head, 64-element heads, small blocks.
        _prefill("prefill_ragged_prompts_d64", "f16", "f16", 12, 4, 64, 8, seqs=24, new_lo=5, new_hi=2000, old_lo=0,
                 old_hi=0, singles=0, lens_seed=3),
        # Chunked prefill over an 8-bit cache.
        _prefill("prefill_chunks_over_e4m3", "bf16", "e4m3", 32, 8, 128, 16, seqs=8, new_lo=256, new_hi=512,
                 old_lo=512, old_hi=4096, singles=0, lens_seed=4),
        # Reading a whole 16-bit batch back, to hand it to another process or to a dense kernel.
        {"name": "gather_16bit_batch", "op": "gather", "dtype": "bf16", "kv": "bf16", "kv_heads": 8, "dim": 128,
         "block": 16, "seqs": 64, "lo": 512, "hi": 4096, "lens_seed": 5},
        # Reading an 8-bit cache back as 16-bit rows; mixed lengths, small blocks.
        {"name": "gather_e4m3_mixed", "op": "gather", "dtype": "f16", "kv": "e4m3", "kv_heads": 8, "dim": 128,
         "block": 8, "seqs": 100, "lo": 1, "hi": 1500, "lens_seed": 6},
        # One sequence's drafts against a small vocabulary. Latency.
        {"name": "accept_one_sequence", "op": "accept", "dtype": "f32", "seqs": 1, "drafts": 3, "vocab": 32000,
         "sure": False},
        # A serving batch, a large vocabulary.
        {"name": "accept_batch", "op": "accept", "dtype": "f32", "seqs": 64, "drafts": 4, "vocab": 128000,
         "sure": False},
        # Drafts looked up rather than sampled (no draft probabilities), 16-bit probabilities, an odd vocabulary
        # (every other row starts off a 16-byte boundary).
        {"name": "accept_lookup_drafts_odd_vocab", "op": "accept", "dtype": "bf16", "seqs": 48, "drafts": 7,
         "vocab": 50257, "sure": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("prefill", "prefill", "prefill", "gather", "accept"))
    if kind == "accept":
        dtype = rng.choice(("f32", "f16", "bf16"))
        return {"op": "accept", "dtype": dtype, "seqs": _log_int(rng, 1, 64), "drafts": rng.randint(1, 8),
                "vocab": _log_int(rng, 500, 64000), "sure": rng.random() < 0.3}
    kv_heads = rng.choice((1, 2, 4, 8))
    block = rng.choice((8, 16, 32))
    dtype = rng.choice(("f16", "bf16"))
    if kind == "gather":
        kv = rng.choice((dtype, "e4m3"))
        lo = _log_int(rng, 1, 500)
        return {"op": "gather", "dtype": dtype, "kv": kv, "kv_heads": kv_heads, "dim": rng.choice((64, 128)),
                "block": block, "seqs": rng.randint(1, 64), "lo": lo, "hi": lo + _log_int(rng, 1, 3000),
                "lens_seed": rng.randrange(1 << 20)}
    kv = rng.choice((dtype, dtype, "e4m3"))
    seqs = _log_int(rng, 1, 48)
    new_lo = _log_int(rng, 1, 200)
    case = _prefill("", dtype, kv, kv_heads * rng.choice((1, 2, 3, 4, 5, 8)), kv_heads,
                    128 if kv == "e4m3" else rng.choice((64, 128)), block, seqs=seqs, new_lo=new_lo,
                    new_hi=new_lo + _log_int(rng, 1, 700), old_lo=0, old_hi=_log_int(rng, 1, 4096),
                    singles=rng.choice((0, 0, seqs // 2, seqs)), lens_seed=rng.randrange(1 << 20))
    while work(case)["flops"] > 5 * 10 ** 11:                 # no dearer than the long prompt
        case["seqs"] = case["seqs"] // 2
        case["singles"] = case["singles"] // 2
    return case


def _lens(case):
    """(new tokens, all tokens) of each sequence of a prefill case."""
    if "news" in case:
        return [int(x) for x in case["news"].split(",")], [int(x) for x in case["totals"].split(",")]
    r = random.Random(case["lens_seed"])
    news, totals = [], []
    for s in range(case["seqs"]):
        n = 1 if s < case["singles"] else r.randint(case["new_lo"], case["new_hi"])
        news.append(n)
        totals.append(n + r.randint(case["old_lo"], case["old_hi"]))
    order = list(range(len(news)))
    r.shuffle(order)
    return [news[i] for i in order], [totals[i] for i in order]


def _gather_lens(case):
    r = random.Random(case["lens_seed"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]


def work(case):
    if case["op"] == "prefill":
        news, totals = _lens(case)
        pairs = sum(n * (t - n) + n * (n + 1) // 2 for n, t in zip(news, totals))
        cached = 2 * sum(totals) * case["kv_heads"] * case["dim"] * _BYTES[case["kv"]]
        rows = 2 * sum(news) * case["heads"] * case["dim"] * _BYTES[case["dtype"]]
        tables = 4 * sum(-(-t // case["block"]) for t in totals) + 8 * len(news)
        return {"bytes": cached + rows + tables, "flops": 4 * pairs * case["heads"] * case["dim"]}
    if case["op"] == "gather":
        lens = _gather_lens(case)
        row = 2 * case["kv_heads"] * case["dim"]
        return {"bytes": sum(lens) * row * (_BYTES[case["kv"]] + _BYTES[case["dtype"]]), "flops": 0}
    # The final draw reads a target row; where a draft was refused the draft's row too (of these
    # inputs about 7 drafts in 100 are refused).
    rows = 1.0 if case["sure"] else 1.0 + (1.0 - 0.93 ** case["drafts"])
    return {"bytes": int(case["seqs"] * case["vocab"] * _BYTES[case["dtype"]] * rows)
            + case["seqs"] * case["drafts"] * (8 + 4 + 8), "flops": int(3 * case["seqs"] * case["vocab"])}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _pools(case, totals, gen):
    """K and V pools, block tables (blocks in shuffled order) and, for 8-bit pools, their scales."""
    block, hkv, dim = case["block"], case["kv_heads"], case["dim"]
    need = [-(-t // block) for t in totals]
    blocks = sum(need) + sum(need) // 5 + 1
    order = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    tables = torch.zeros(len(totals), max(1, max(need)), dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = order[at:at + n]
        at += n

    def pool():
        x = torch.randn(blocks, block, hkv, dim, generator=gen, device="cuda", dtype=torch.float32)
        if case["kv"] != "e4m3":
            return x.to(_DT[case["kv"]]), None
        scale = x.abs().amax(dim=(0, 1, 3)) / 448.0
        return (x / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8), scale

    k, k_scale = pool()
    v, v_scale = pool()
    return {"k": k, "v": v, "tables": tables, "k_scale": k_scale, "v_scale": v_scale}


def _starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = {"case": case}
    if case["op"] == "accept":
        B, K, V = case["seqs"], case["drafts"], case["vocab"]
        logits = torch.randn(B, K + 1, V, generator=gen, device="cuda") * 2.0
        p = torch.softmax(logits, -1)
        q = torch.softmax(logits[:, :K] + 0.15 * torch.randn(B, K, V, generator=gen, device="cuda"), -1)
        race = torch.empty_like(q).exponential_(generator=gen)
        st["drafts"] = (q / race).argmax(-1)                      # sampled from the draft's distribution
        st["target"] = p.to(_DT[case["dtype"]])
        st["draft"] = None if case["sure"] else q.to(_DT[case["dtype"]])
        if case["sure"]:
            st["drafts"] = p[:, :K].argmax(-1)                    # a lookup that is often right
        st["uniform"] = torch.rand(B, K + 1, generator=gen, device="cuda")
        st["tokens"] = torch.empty(B, K + 1, dtype=torch.int64, device="cuda")
        st["accepted"] = torch.empty(B, dtype=torch.int32, device="cuda")
        return st
    dt = _DT[case["dtype"]]
    if case["op"] == "gather":
        lens = _gather_lens(case)
        at = _starts(lens)
        st.update(_pools(case, lens, gen), lens=lens, at=at)
        st["k_out"] = torch.empty(at[-1], case["kv_heads"], case["dim"], dtype=dt, device="cuda")
        st["v_out"] = torch.empty_like(st["k_out"])
        st["row_starts"] = torch.tensor(at, dtype=torch.int32, device="cuda")
        st["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        return st
    news, totals = _lens(case)
    at = _starts(news)
    st.update(_pools(case, totals, gen), news=news, totals=totals, at=at)
    st["q"] = torch.randn(at[-1], case["heads"], case["dim"], generator=gen, device="cuda").to(dt)
    st["out"] = torch.empty_like(st["q"])
    st["query_starts"] = torch.tensor(at, dtype=torch.int32, device="cuda")
    st["seq_lens"] = torch.tensor(totals, dtype=torch.int32, device="cuda")
    st["scale"] = 1.0 / math.sqrt(case["dim"])
    if own:
        import paged_kv_cache_156_gb300 as pkv
        st["workspace"] = pkv.alloc_prefill_workspace(len(news), at[-1], case["heads"], case["kv_heads"], case["dim"])
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"prefill": _own_prefill, "gather": _own_gather, "accept": _own_accept}[op](state)
    return {"prefill": _plain_prefill, "gather": _plain_gather, "accept": _plain_accept}[op](state)


def _own_prefill(st):
    import paged_kv_cache_156_gb300 as pkv
    pkv.paged_attention_prefill(st["out"], st["q"], st["k"], st["v"], st["tables"], st["seq_lens"],
                                st["query_starts"], st["scale"], max_seq_len=max(st["totals"]),
                                workspace=st["workspace"], k_scale=st["k_scale"], v_scale=st["v_scale"])
    return st["out"]


def _own_gather(st):
    import paged_kv_cache_156_gb300 as pkv
    pkv.paged_kv_gather(st["k_out"], st["v_out"], st["k"], st["v"], st["tables"], st["seq_lens"], st["row_starts"],
                        k_scale=st["k_scale"], v_scale=st["v_scale"])
    return st["k_out"], st["v_out"]


def _own_accept(st):
    import paged_kv_cache_156_gb300 as pkv
    pkv.speculative_accept(st["tokens"], st["accepted"], st["drafts"], st["target"], st["uniform"],
                           draft_probs=st["draft"])
    return st["tokens"], st["accepted"]


def _dense(st, pool, scale, s, n):
    """The first n positions of sequence s, float32 [n, KV heads, dim]."""
    block = pool.shape[1]
    rows = pool[st["tables"][s, :-(-n // block)].long()].flatten(0, 1)[:n]
    if scale is None:
        return rows.float()
    return rows.view(torch.float8_e4m3fn).float() * scale[:, None]


def _plain_prefill(st):
    case = st["case"]
    group = case["heads"] // case["kv_heads"]
    out = torch.empty_like(st["q"])
    for s, (n, total) in enumerate(zip(st["news"], st["totals"])):
        if n == 0:
            continue
        k = _dense(st, st["k"], st["k_scale"], s, total).permute(1, 2, 0)                  # [Hkv, d, total]
        v = _dense(st, st["v"], st["v_scale"], s, total).transpose(0, 1)                   # [Hkv, total, d]
        step = max(1, (1 << 28) // (case["heads"] * total))                                # rows whose scores fit 1 GB
        for lo in range(0, n, step):
            hi = min(n, lo + step)
            seen = total - n + hi                                                          # no row here sees further
            q = st["q"][st["at"][s] + lo:st["at"][s] + hi].float()
            q = q.view(hi - lo, case["kv_heads"], group, -1).permute(1, 2, 0, 3).flatten(1, 2)   # [Hkv, G m, d]
            z = torch.matmul(q, k[:, :, :seen]).view(case["kv_heads"], group, hi - lo, seen) * st["scale"]
            last = total - n + torch.arange(lo, hi, device=z.device)
            z = z.masked_fill(torch.arange(seen, device=z.device)[None, :] > last[:, None], -math.inf)
            w = torch.exp(z - z.amax(-1, keepdim=True))
            o = torch.matmul(w.flatten(1, 2), v[:, :seen]).view(case["kv_heads"], group, hi - lo, -1)
            o = o / w.sum(-1, keepdim=True)
            out[st["at"][s] + lo:st["at"][s] + hi] = o.permute(2, 0, 1, 3).flatten(1, 2).to(out.dtype)
    return out


def _plain_gather(st):
    k_out, v_out = torch.empty_like(st["k_out"]), torch.empty_like(st["v_out"])
    for s, n in enumerate(st["lens"]):
        at = st["at"][s]
        k_out[at:at + n] = _dense(st, st["k"], st["k_scale"], s, n).to(k_out.dtype)
        v_out[at:at + n] = _dense(st, st["v"], st["v_scale"], s, n).to(v_out.dtype)
    return k_out, v_out


def _plain_accept(st):
    x, p, q, u = st["drafts"], st["target"], st["draft"], st["uniform"]
    B, K = x.shape
    rows = torch.arange(B, device=x.device)
    px = p[:, :K].gather(2, x[..., None])[..., 0].double()
    qx = torch.ones_like(px) if q is None else q.gather(2, x[..., None])[..., 0].double()
    kept = (u[:, :K].double() * qx < px).long().cumprod(1)          # 32-bit factors: the product is exact
    a = kept.sum(1)
    row = p[rows, a].float()
    at = a.clamp(max=K - 1)
    if q is None:
        other = torch.zeros_like(row).scatter_(1, x[rows, at][:, None], math.inf)
    else:
        other = q[rows, at].float()
    left = torch.where((a < K)[:, None], row - other, row)

    def units(w):                                                   # whole units of 2^-44, summed exactly
        w = torch.where(w > 0, w, torch.zeros_like(w)).clamp(max=1.0)
        return (w * _UNIT).to(torch.int64)                          # (the product with 2^44 is exact)

    n = units(left)
    n = torch.where(n.sum(1, keepdim=True) > 0, n, units(row))
    upto = n.cumsum(1)
    total = upto[:, -1]
    mark = torch.minimum((u[:, K].double() * total.double()).long(), total - 1)
    drawn = (upto <= mark[:, None]).sum(1)
    drawn = torch.where(total > 0, drawn, torch.full_like(drawn, -1))
    place = torch.arange(K + 1, device=x.device)[None, :]
    tokens = torch.cat([x, x[:, :1]], 1)
    tokens = torch.where(place < a[:, None], tokens, torch.where(place == a[:, None], drawn[:, None], -1))
    return tokens, a.to(torch.int32)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _positions(st, pool, scale, s, where):
    """Rows at the given positions of sequence s, read one slot each, float64."""
    block = st["case"]["block"]
    slots = st["tables"][s].long()[where // block] * block + where % block
    rows = pool.view(-1, *pool.shape[2:])[slots]
    if scale is None:
        return rows.double()
    return rows.view(torch.float8_e4m3fn).to(torch.float64) * scale.double()[None, :, None]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "gather":
        k = torch.empty(st["k_out"].shape, dtype=torch.float64, device="cuda")
        v = torch.empty_like(k)
        for s, n in enumerate(st["lens"]):
            where = torch.arange(n, device="cuda")
            k[st["at"][s] + where] = _positions(st, st["k"], st["k_scale"], s, where)
            v[st["at"][s] + where] = _positions(st, st["v"], st["v_scale"], s, where)
        return k, v
    if case["op"] == "accept":
        return _exact_accept(st)
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for s, (n, total) in enumerate(zip(st["news"], st["totals"])):
        where = torch.arange(total, device="cuda")
        k = _positions(st, st["k"], st["k_scale"], s, where)
        v = _positions(st, st["v"], st["v_scale"], s, where)
        for h in range(case["heads"]):
            kh, vh = k[:, h // group], v[:, h // group]
            for lo in range(0, n, 1024):
                mine = torch.arange(lo, min(n, lo + 1024), device="cuda")
                limit = total - n + mine + 1                        # token i sees positions below this
                top = int(total - n + min(n, lo + 1024))
                z = torch.einsum("id,td->it", st["q"][st["at"][s] + mine, h].double(), kh[:top]) / math.sqrt(case["dim"])
                z = torch.where(where[None, :top] < limit[:, None], z, torch.full_like(z, -math.inf))
                out[st["at"][s] + mine, h] = torch.einsum("it,td->id", torch.softmax(z, 1), vh[:top])
    return out


def _exact_accept(st):
    x, u = st["drafts"].cpu().numpy(), st["uniform"].cpu().numpy()
    p = st["target"].float().cpu().numpy()
    q = None if st["draft"] is None else st["draft"].float().cpu().numpy()
    B, K = x.shape
    tokens = np.full((B, K + 1), -1, dtype=np.int64)
    accepted = np.zeros(B, dtype=np.int32)
    for b in range(B):
        a = 0
        while a < K and float(u[b, a]) * (1.0 if q is None else float(q[b, a, x[b, a]])) < float(p[b, a, x[b, a]]):
            tokens[b, a] = x[b, a]
            a += 1
        row = p[b, a]
        if a < K and q is None:
            left = row.copy()
            left[x[b, a]] = 0.0
        else:
            left = row - q[b, a] if a < K else row
        for weights in (left, row):
            n = np.floor(np.clip(weights, 0.0, 1.0).astype(np.float64) * 2.0 ** 44).astype(np.uint64)
            upto = np.cumsum(n, dtype=np.uint64)
            total = int(upto[-1])
            if total:
                mark = min(int(float(u[b, K]) * float(total)), total - 1)
                tokens[b, a] = int(np.searchsorted(upto, np.uint64(mark), side="right"))
                break
        accepted[b] = a
    return torch.from_numpy(tokens).cuda(), torch.from_numpy(accepted).cuda()
