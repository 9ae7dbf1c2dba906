"""Workloads of the operators of a tree step: drafted tokens that branch.

A serving loop that drafts a tree of continuations for every sequence makes
four calls a step, and each case is one of them: the tree's keys and values
rotated to their positions and written into the paged cache
(``paged_kv_append_rotary``, which prompts and single tokens take too), the
attention of the tree's tokens over the cache, each over its own ancestors
(``paged_attention_tree``), the walk down the tree that follows the target's
distribution (``speculative_accept_tree``), and the cache made to hold the
accepted path alone (``paged_kv_keep_path``).

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
# A draw sums its weights as whole numbers of this unit (2^-44).
_UNIT = float(1 << 44)
# Logits of a row's likely tokens over the others' (normal, deviation 2): the first then has about 0.4 of the
# probability, the others 0.15, 0.06, ...
_BOOST = (14.0, 13.0, 12.0, 11.0, 10.0, 9.0)


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _rotary(name, dtype, kv, heads, kv_heads, dim, rotary, block, tokens, interleaved, packed, pad, lens_seed):
    return {"name": name, "op": "rotary", "dtype": dtype, "kv": kv, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "rotary": rotary, "block": block, "tokens": tokens, "interleaved": interleaved, "packed": packed, "pad": pad,
            "lens_seed": lens_seed}


def _tree(name, dtype, kv, heads, kv_heads, dim, block, seqs, nodes_lo, nodes_hi, old_lo, old_hi, lens_seed):
    return {"name": name, "op": "tree", "dtype": dtype, "kv": kv, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "block": block, "seqs": seqs, "nodes_lo": nodes_lo, "nodes_hi": nodes_hi, "old_lo": old_lo, "old_hi": old_hi,
            "lens_seed": lens_seed}


def _accept(name, dtype, seqs, nodes_lo, nodes_hi, depth, vocab, lens_seed):
    return {"name": name, "op": "accept", "dtype": dtype, "seqs": seqs, "nodes_lo": nodes_lo, "nodes_hi": nodes_hi,
            "depth": depth, "vocab": vocab, "lens_seed": lens_seed}


def _keep(name, kv, layers, seqs, nodes, kept, old_hi, kv_heads, dim, block, lens_seed):
    return {"name": name, "op": "keep", "kv": kv, "layers": layers, "seqs": seqs, "nodes": nodes, "kept": kept,
            "old_hi": old_hi, "kv_heads": kv_heads, "dim": dim, "block": block, "lens_seed": lens_seed}


def listed():
    return [
        # The new tokens of four sequences of a small model. Latency.
        _rotary("rotary_small_step", "f16", "f16", 4, 4, 64, 64, 16, 4, False, False, 0, 1),
        # A prompt of a large model, out of the projection's packed rows (q, k and v side by side).
        _rotary("rotary_prompt_packed", "bf16", "bf16", 64, 8, 128, 128, 16, 8192, False, True, 0, 2),
        # A tree step's tokens into an 8-bit cache, half of each head rotated, neighbouring elements paired, a few of
        # the rows padding.
        _rotary("rotary_e4m3_partial", "f16", "e4m3", 32, 8, 128, 64, 32, 1037, True, False, 5, 3),
        # Trees of up to eight tokens over four short sequences of a small model. Latency.
        _tree("tree_small_step", "f16", "f16", 4, 4, 64, 16, 4, 1, 8, 1, 50, 5),
        # Sixteen tokens a tree over a serving batch.
        _tree("tree_batch_16", "bf16", "bf16", 32, 8, 128, 16, 64, 16, 16, 512, 4096, 6),
        # Ragged trees up to the largest over mixed lengths, 64 query heads over 8 KV heads.
        _tree("tree_mixed_ragged", "f16", "f16", 64, 8, 128, 16, 128, 1, 64, 32, 2000, 7),
        # One very long sequence.
        _tree("tree_long_context", "bf16", "bf16", 64, 8, 128, 32, 1, 63, 63, 65500, 65500, 8),
        # Trees of 26 tokens over an 8-bit cache.
        _tree("tree_batch_e4m3", "bf16", "e4m3", 32, 8, 128, 16, 64, 26, 26, 512, 4096, 9),
        # One sequence's tree against a small vocabulary. Latency.
        _accept("accept_tree_one", "f16", 1, 8, 8, 4, 32000, 10),
        # A serving batch's trees, a large vocabulary.
        _accept("accept_tree_batch", "f32", 64, 16, 16, 6, 128000, 11),
        # The accepted paths of a serving batch, all 32 layers' caches.
        _keep("keep_path_batch", "bf16", 32, 64, 24, 5, 40, 8, 128, 16, 12),
        # One sequence's, two layers of an 8-bit cache. Latency.
        _keep("keep_path_e4m3_one", "e4m3", 2, 1, 9, 3, 100, 4, 64, 8, 13),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("rotary", "tree", "tree", "tree", "accept", "keep"))
    seed = rng.randrange(1 << 20)
    dtype = rng.choice(("f16", "bf16"))
    kv = rng.choice((dtype, dtype, "e4m3"))
    block = rng.choice((8, 16, 32))
    kv_heads = rng.choice((1, 2, 4, 8))
    if kind == "rotary":
        dim = rng.choice((64, 128))
        return _rotary("", dtype, kv, kv_heads * rng.choice((1, 2, 3, 4, 7, 8)), kv_heads, dim,
                       rng.choice((dim, dim, dim // 2, 48)), block, _log_int(rng, 1, 4096), rng.random() < 0.4,
                       rng.random() < 0.5, rng.randint(0, 3), seed)
    if kind == "accept":
        lo = _log_int(rng, 1, 24)
        return _accept("", rng.choice(("f32", "f16", "bf16")), _log_int(rng, 1, 64), lo, lo + rng.randint(0, 8),
                       rng.randint(1, 8), _log_int(rng, 500, 60000), seed)
    if kind == "keep":
        nodes = rng.randint(3, 64)
        return _keep("", kv, _log_int(rng, 1, 40), _log_int(rng, 1, 48), nodes, rng.randint(1, (nodes - 1) // 2), _log_int(rng, 1, 80),
                     kv_heads, rng.choice((64, 128)), block, seed)
    seqs, lo, old = _log_int(rng, 1, 96), _log_int(rng, 1, 64), _log_int(rng, 1, 2000)
    case = _tree("", dtype, kv, kv_heads * rng.choice((1, 2, 3, 4, 5, 8)), kv_heads, 128 if kv == "e4m3" else rng.choice((64, 128)),
                 block, seqs, lo, min(64, lo + rng.randint(0, 30)), old, old + _log_int(rng, 1, 4000), seed)
    while work(case)["flops"] > 10 ** 11 or work(case)["bytes"] > 6 * 10 ** 8:       # no dearer than the listed ones
        case["seqs"] = max(1, case["seqs"] // 2)
        case["old_hi"] = max(case["old_lo"], case["old_hi"] // 2)
    return case


def _tree_of(r, n, depth):
    """Parents of a tree of n tokens, the root first: up to four children each, in the order of depth."""
    parents, level, kids = [-1], [0], [0]
    while len(parents) < n:
        open_ = [i for i in range(len(parents)) if kids[i] < 4 and level[i] < depth]
        if not open_:                                             # a full tree: more children of the root
            open_ = [0]
        # likelier below the first tokens drafted
        p = open_[min(len(open_) - 1, int(r.expovariate(0.35)))]
        kids[p] += 1
        parents.append(p)
        level.append(level[p] + 1)
        kids.append(0)
    order = sorted(range(n), key=lambda i: level[i])              # (a stable sort: parents stay before children)
    at = {old: new for new, old in enumerate(order)}
    return [at[parents[i]] if i else -1 for i in order], [level[i] for i in order]


def _trees(case, depth=64):
    """(parents, depths) of every sequence's tree."""
    r = random.Random(case["lens_seed"])
    return [_tree_of(r, r.randint(case["nodes_lo"], case["nodes_hi"]), depth) for _ in range(case["seqs"])]


def _lens(case):
    """(tokens in the tree, all positions) of each sequence of a tree case."""
    news = [len(p) for p, _ in _trees(case)]
    r = random.Random(case["lens_seed"] + 1)
    return news, [n + r.randint(case["old_lo"], case["old_hi"]) for n in news]


def work(case):
    if case["op"] == "rotary":
        T, h, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        e = _BYTES[case["dtype"]]
        rows = T * d * (2 * h * e + 2 * hk * (e + _BYTES[case["kv"]]))
        return {"bytes": rows + T * (4 * case["rotary"] + 12), "flops": 3 * T * (h + hk) * case["rotary"]}
    if case["op"] == "tree":
        news, totals = _lens(case)
        pairs = 0
        for (parents, depths), n, t in zip(_trees(case), news, totals):
            pairs += n * (t - n) + sum(d + 1 for d in depths)
        cached = 2 * sum(totals) * case["kv_heads"] * case["dim"] * _BYTES[case["kv"]]
        rows = 2 * sum(news) * case["heads"] * case["dim"] * _BYTES[case["dtype"]]
        tables = 4 * sum(-(-t // case["block"]) for t in totals) + 8 * len(news) + 8 * sum(news)
        return {"bytes": cached + rows + tables, "flops": 4 * pairs * case["heads"] * case["dim"]}
    if case["op"] == "accept":
        # Of these inputs a sequence looks at some 2.1 rows: its root's and those of the tokens it accepts.
        nodes = sum(len(p) for p, _ in _trees(case, case["depth"]))
        return {"bytes": int(2.1 * case["seqs"] * case["vocab"] * _BYTES[case["dtype"]]) + 16 * nodes,
                "flops": int(2.1 * 2 * case["seqs"] * case["vocab"])}
    row = case["kv_heads"] * case["dim"] * (1 if case["kv"] == "e4m3" else 2)
    return {"bytes": 4 * row * case["layers"] * case["seqs"] * case["kept"] + 4 * case["seqs"] * (case["kept"] + 4), "flops": 0}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _tables(totals, block, gen):
    """Block tables (blocks in shuffled order) and the number of blocks in the pool."""
    need = [-(-t // block) for t in totals]
    blocks = sum(need) + sum(need) // 5 + 1
    order = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    tables = torch.zeros(len(totals), max(1, max(need)), dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = order[at:at + n]
        at += n
    return tables, blocks


def _pool(case, blocks, gen):
    """A pool, and for 8-bit pools its scales."""
    x = torch.randn(blocks, case["block"], case["kv_heads"], case["dim"], generator=gen, device="cuda", dtype=torch.float32)
    if case["kv"] != "e4m3":
        return x.to(_DT[case["kv"]]), None
    scale = x.abs().amax(dim=(0, 1, 3)) / 448.0
    return (x / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"rotary": _prepare_rotary, "tree": _prepare_tree, "accept": _prepare_accept, "keep": _prepare_keep}[case["op"]](case, gen)


def _prepare_rotary(case, gen):
    T, h, hk, d, rot = case["tokens"], case["heads"], case["kv_heads"], case["dim"], case["rotary"]
    dt = _DT[case["dtype"]]
    st = {"case": case}
    if case["packed"]:                                            # the projection's output: a row holds q, k and v
        qkv = torch.randn(T, (h + 2 * hk) * d, generator=gen, device="cuda").to(dt)
        st["q"], st["k"], st["v"] = (x.unflatten(1, (-1, d)) for x in qkv.split((h * d, hk * d, hk * d), 1))
    else:
        st["q"] = torch.randn(T, h, d, generator=gen, device="cuda").to(dt)
        st["k"] = torch.randn(T, hk, d, generator=gen, device="cuda").to(dt)
        st["v"] = torch.randn(T, hk, d, generator=gen, device="cuda").to(dt)
    st["q_out"] = torch.empty(T, h, d, dtype=dt, device="cuda")
    blocks = T // case["block"] + T // (5 * case["block"]) + 2
    st["kc"], st["k_scale"] = _pool(case, blocks, gen)
    st["vc"], st["v_scale"] = _pool(case, blocks, gen)
    slots = torch.randperm(blocks * case["block"], generator=gen, device="cuda")[:T]
    if case["pad"]:
        slots[torch.randperm(T, generator=gen, device="cuda")[:min(case["pad"], T - 1)]] = -1
    st["slots"] = slots
    # positions: runs of a few sequences somewhere below 16384
    far = 16384
    first = random.Random(case["lens_seed"]).randrange(far)
    st["positions"] = ((first + torch.arange(T, device="cuda")) % far).to(torch.int32)
    angles = torch.arange(far, dtype=torch.float64, device="cuda")[:, None] * \
        10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    st["cos_sin"] = torch.cat([angles.cos(), angles.sin()], 1).float()
    return st


def _prepare_tree(case, gen):
    news, totals = _lens(case)
    at = _starts(news)
    st = {"case": case, "news": news, "totals": totals, "at": at}
    st["tables"], blocks = _tables(totals, case["block"], gen)
    st["k"], st["k_scale"] = _pool(case, blocks, gen)
    st["v"], st["v_scale"] = _pool(case, blocks, gen)
    st["q"] = torch.randn(at[-1], case["heads"], case["dim"], generator=gen, device="cuda").to(_DT[case["dtype"]])
    st["out"] = torch.empty_like(st["q"])
    st["query_starts"], st["seq_lens"] = _int32(at), _int32(totals)
    masks = []
    for parents, _ in _trees(case):
        m = []
        for i, p in enumerate(parents):
            m.append((m[p] if p >= 0 else 0) | 1 << i)
        masks += [x - (1 << 64) if x >> 63 else x for x in m]
    st["mask"] = torch.tensor(masks, dtype=torch.int64, device="cuda")
    st["scale"] = 1.0 / math.sqrt(case["dim"])
    if own:
        import paged_kv_cache_156_gb300 as pkv
        st["workspace"] = pkv.alloc_prefill_workspace(len(news), at[-1], case["heads"], case["kv_heads"], case["dim"])
    return st


def _prepare_accept(case, gen):
    V, B = case["vocab"], case["seqs"]
    trees = _trees(case, case["depth"])
    at = _starts([len(p) for p, _ in trees])
    T = at[-1]
    logits = torch.randn(T, V, generator=gen, device="cuda") * 2.0
    likely = torch.randint(0, V, (T, 1), generator=gen, device="cuda")
    likely = (likely + torch.arange(6, device="cuda") * (V // 7)) % V               # six different tokens
    logits.scatter_(1, likely, torch.tensor(_BOOST, device="cuda").expand(T, 6))
    st = {"case": case, "at": at, "probs": torch.softmax(logits, -1).to(_DT[case["dtype"]])}
    # a token's children are drafts of its likeliest successors
    rank = []
    for parents, _ in trees:
        seen = [0] * len(parents)
        for p in parents:
            rank.append(0 if p < 0 else min(seen[p], 5))
            if p >= 0:
                seen[p] += 1
    parents = [p for q, _ in trees for p in q]
    row = [a + max(p, 0) for a, (q, _) in zip(at, trees) for p in q]
    st["drafts"] = likely[torch.tensor(row, device="cuda"), torch.tensor(rank, device="cuda")]
    st["parents"], st["query_starts"] = _int32(parents), _int32(at)
    st["uniform"] = torch.rand(T, generator=gen, device="cuda")
    W = case["depth"] + 1
    st["tokens"] = torch.empty(B, W, dtype=torch.int64, device="cuda")
    st["path"] = torch.empty(B, W, dtype=torch.int32, device="cuda")
    st["accepted"] = torch.empty(B, dtype=torch.int32, device="cuda")
    return st


def _prepare_keep(case, gen):
    r = random.Random(case["lens_seed"])
    B, n, kept = case["seqs"], case["nodes"], case["kept"]
    totals = [n + r.randint(0, case["old_hi"]) for _ in range(B)]
    st = {"case": case, "totals": totals}
    st["tables"], blocks = _tables(totals, case["block"], gen)
    st["kc"] = [_pool(case, blocks, gen)[0] for _ in range(case["layers"])]
    st["vc"] = [_pool(case, blocks, gen)[0] for _ in range(case["layers"])]
    # the tokens accepted lie past the places they move to, so that a second call finds the same rows
    path = [[0] + sorted(r.sample(range(kept + 1, n), min(kept, n - kept - 1))) for _ in range(B)]
    st["counts"] = [len(p) - 1 for p in path]
    st["paths"] = path
    st["path"] = _int32([p + [-1] * (kept + 2 - len(p)) for p in path])
    st["accepted"] = _int32(st["counts"])
    st["query_starts"], st["seq_lens"] = _int32([n * i for i in range(B + 1)]), _int32(totals)
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"rotary": _own_rotary, "tree": _own_tree, "accept": _own_accept, "keep": _own_keep}[op](state)
    return {"rotary": _plain_rotary, "tree": _plain_tree, "accept": _plain_accept, "keep": _plain_keep}[op](state)


def _codes(pools):
    """8-bit pools as the numbers their codes are (the scales aside)."""
    return [p.view(torch.float8_e4m3fn) if p.dtype == torch.uint8 else p for p in pools]


def _own_rotary(st):
    import paged_kv_cache_156_gb300 as pkv
    pkv.paged_kv_append_rotary(st["q_out"], st["q"], st["k"], st["v"], st["kc"], st["vc"], st["slots"], st["positions"],
                               st["cos_sin"], interleaved=st["case"]["interleaved"], k_scale=st["k_scale"],
                               v_scale=st["v_scale"])
    return [st["q_out"]] + _codes([st["kc"], st["vc"]])


def _own_tree(st):
    import paged_kv_cache_156_gb300 as pkv
    pkv.paged_attention_tree(st["out"], st["q"], st["k"], st["v"], st["tables"], st["seq_lens"], st["query_starts"],
                             st["mask"], st["scale"], max_seq_len=max(st["totals"]), workspace=st["workspace"],
                             k_scale=st["k_scale"], v_scale=st["v_scale"])
    return st["out"]


def _own_accept(st):
    import paged_kv_cache_156_gb300 as pkv
    pkv.speculative_accept_tree(st["tokens"], st["path"], st["accepted"], st["drafts"], st["parents"],
                                st["query_starts"], st["probs"], st["uniform"])
    return st["tokens"], st["path"], st["accepted"]


def _own_keep(st):
    import paged_kv_cache_156_gb300 as pkv
    pkv.paged_kv_keep_path(st["kc"], st["vc"], st["tables"], st["seq_lens"], st["query_starts"], st["path"],
                           st["accepted"])
    return _codes(st["kc"] + st["vc"])


def _plain_rotary(st):
    case, rot = st["case"], st["case"]["rotary"]
    table = st["cos_sin"][st["positions"].long()]
    c, s = table[:, None, :rot // 2], table[:, None, rot // 2:]

    def turned(x):
        x = x.float()
        if case["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(2)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y = torch.cat([a * c - b * s, b * c + a * s], -1)
        return torch.cat([y, x[..., rot:]], -1)

    live = st["slots"] >= 0
    at = st["slots"][live]
    for pool, rows, scale in ((st["kc"], turned(st["k"])[live], st["k_scale"]), (st["vc"], st["v"][live].float(), st["v_scale"])):
        if scale is not None:
            pool.view(-1, *pool.shape[2:])[at] = (rows / scale[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            pool.view(-1, *pool.shape[2:])[at] = rows.to(pool.dtype)
    return [turned(st["q"]).to(st["q"].dtype)] + _codes([st["kc"], st["vc"]])


def _dense(st, pool, scale, s, n):
    """The first n positions of sequence s, float32 [n, KV heads, dim]."""
    block = pool.shape[1]
    rows = pool[st["tables"][s, :-(-n // block)].long()].flatten(0, 1)[:n]
    if scale is None:
        return rows.float()
    return rows.view(torch.float8_e4m3fn).float() * scale[:, None]


def _plain_tree(st):
    case = st["case"]
    group, hk = case["heads"] // case["kv_heads"], case["kv_heads"]
    out = torch.empty_like(st["q"])
    for s, (n, total) in enumerate(zip(st["news"], st["totals"])):
        k = _dense(st, st["k"], st["k_scale"], s, total).permute(1, 2, 0)                  # [Hkv, d, total]
        v = _dense(st, st["v"], st["v_scale"], s, total).transpose(0, 1)                   # [Hkv, total, d]
        q = st["q"][st["at"][s]:st["at"][s + 1]].float().view(n, hk, group, -1).permute(1, 2, 0, 3).flatten(1, 2)
        z = torch.matmul(q, k).view(hk, group, n, total) * st["scale"]
        bits = (st["mask"][st["at"][s]:st["at"][s + 1], None] >> torch.arange(n, device=z.device)) & 1
        z[..., total - n:].masked_fill_(bits == 0, -math.inf)
        w = torch.exp(z - z.amax(-1, keepdim=True))
        o = torch.matmul(w.flatten(1, 2), v).view(hk, group, n, -1) / w.sum(-1, keepdim=True)
        out[st["at"][s]:st["at"][s + 1]] = o.permute(2, 0, 1, 3).flatten(1, 2).to(out.dtype)
    return out


def _plain_accept(st):
    B, W = st["tokens"].shape
    dev = st["probs"].device
    starts, ends = st["query_starts"][:-1].long(), st["query_starts"][1:].long()
    T = st["drafts"].shape[0]
    node = torch.arange(T, device=dev)
    seq = torch.searchsorted(ends, node, right=True)              # whose tree a node is of
    parent = torch.where(st["parents"] >= 0, starts[seq] + st["parents"], -1)
    tokens = torch.full((B, W), -1, dtype=torch.int64, device=dev)
    path = torch.full((B, W), -1, dtype=torch.int32, device=dev)
    accepted = torch.zeros(B, dtype=torch.int32, device=dev)
    at, alive = starts.clone(), torch.ones(B, dtype=torch.bool, device=dev)
    for step in range(W):
        path[:, step] = torch.where(alive, at - starts, -1).to(torch.int32)
        w = st["probs"][at].float()
        n = (torch.where(w > 0, w, torch.zeros_like(w)).clamp(max=1.0) * _UNIT).to(torch.int64)   # whole units, summed exactly
        upto = n.cumsum(1)
        total = upto[:, -1]
        mark = torch.minimum((st["uniform"][at].double() * total.double()).long(), total - 1)
        y = torch.where(total > 0, (upto <= mark[:, None]).sum(1), -1)
        tokens[:, step] = torch.where(alive, y, -1)
        child = (parent[None, :] == at[:, None]) & (st["drafts"][None, :] == y[:, None])
        found = child.any(1) & alive
        if step == W - 1:
            break
        at = torch.where(found, child.to(torch.uint8).argmax(1), at)                       # (the first of them)
        accepted += found.to(torch.int32)
        alive = found
    return tokens, path, accepted


def _plain_keep(st):
    block, n = st["case"]["block"], st["case"]["nodes"]
    width = st["path"].shape[1]
    rank = torch.arange(width, device="cuda")[None, :]
    live = rank <= st["accepted"][:, None]
    base = (st["seq_lens"] - n).long()[:, None]

    def slots(where):                                             # of positions, the live ones
        blocks = torch.gather(st["tables"].long(), 1, where // block)
        return (blocks * block + where % block)[live]

    src = slots(torch.where(live, base + st["path"], 0))
    dst = slots(torch.where(live, base + rank, 0))
    for pool in st["kc"] + st["vc"]:
        rows = pool.view(-1, *pool.shape[2:])
        rows[dst] = rows[src]                                     # (the right side is whole before the left is written)
    return _codes(st["kc"] + st["vc"])


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
    return {"rotary": _exact_rotary, "tree": _exact_tree, "accept": _exact_accept, "keep": _exact_keep}[case["op"]](st)


def _exact_rotary(st):
    case, rot = st["case"], st["case"]["rotary"]
    table = st["cos_sin"].double()[st["positions"].long()]
    turn = torch.complex(table[:, :rot // 2], table[:, rot // 2:])[:, None, :]              # e^(i angle)
    even = torch.arange(0, rot, 2, device="cuda") if case["interleaved"] else torch.arange(rot // 2, device="cuda")
    odd = even + (1 if case["interleaved"] else rot // 2)

    def turned(x):
        y = x.double().clone(memory_format=torch.contiguous_format)
        z = torch.complex(y[..., even], y[..., odd]) * turn
        y[..., even], y[..., odd] = z.real, z.imag
        return y

    outs = [turned(st["q"])]
    for pool, rows, scale in ((st["kc"], turned(st["k"]), st["k_scale"]), (st["vc"], st["v"].double(), st["v_scale"])):
        full = _codes([pool])[0].to(torch.float64).flatten(0, 1)
        if scale is not None:
            rows = (rows / scale.double()[None, :, None]).clamp(-448.0, 448.0)              # (in codes' units)
        for t, slot in enumerate(st["slots"].tolist()):
            if slot >= 0:
                full[slot] = rows[t]
        outs.append(full.view(pool.shape))
    return outs


def _exact_tree(st):
    case = st["case"]
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for s, ((parents, _), n, total) in enumerate(zip(_trees(case), st["news"], st["totals"])):
        where = torch.arange(total, device="cuda")
        k = _positions(st, st["k"], st["k_scale"], s, where)
        v = _positions(st, st["v"], st["v_scale"], s, where)
        sees = torch.zeros(n, total, dtype=torch.bool)
        sees[:, :total - n] = True
        for i in range(n):                                        # itself and its ancestors
            j = i
            while j >= 0:
                sees[i, total - n + j] = True
                j = parents[j]
        sees = sees.cuda()
        for h in range(case["heads"]):
            z = torch.einsum("id,td->it", st["q"][st["at"][s]:st["at"][s + 1], h].double(), k[:, h // group]) / math.sqrt(case["dim"])
            p = torch.softmax(torch.where(sees, z, torch.full_like(z, -math.inf)), 1)
            out[st["at"][s]:st["at"][s + 1], h] = torch.einsum("it,td->id", p, v[:, h // group])
    return out


def _exact_accept(st):
    B, W = st["tokens"].shape
    drafts, parents, u = st["drafts"].tolist(), st["parents"].tolist(), st["uniform"].cpu().numpy()
    tokens = np.full((B, W), -1, dtype=np.int64)
    path = np.full((B, W), -1, dtype=np.int32)
    accepted = np.zeros(B, dtype=np.int32)
    for b in range(B):
        first, end = st["at"][b], st["at"][b + 1]
        i = 0
        for step in range(W):
            path[b, step] = i
            p = st["probs"][first + i].float().cpu().numpy()
            upto = np.cumsum(np.floor(np.clip(p, 0.0, 1.0).astype(np.float64) * 2.0 ** 44).astype(np.uint64), dtype=np.uint64)
            total = int(upto[-1])
            if total == 0:
                break
            mark = min(int(float(u[first + i]) * float(total)), total - 1)
            y = int(np.searchsorted(upto, np.uint64(mark), side="right"))
            tokens[b, step] = y
            kids = [j for j in range(1, end - first) if parents[first + j] == i and drafts[first + j] == y]
            if step == W - 1 or not kids:
                break
            i = kids[0]
            accepted[b] += 1
    return torch.from_numpy(tokens).cuda(), torch.from_numpy(path).cuda(), torch.from_numpy(accepted).cuda()


def _exact_keep(st):
    outs = []
    block, n = st["case"]["block"], st["case"]["nodes"]
    table = st["tables"].tolist()
    moves = []
    for s, total in enumerate(st["totals"]):
        for i, j in enumerate(st["paths"][s]):
            src, dst = total - n + j, total - n + i
            moves.append((table[s][src // block], src % block, table[s][dst // block], dst % block))
    sb, so, db, do = (torch.tensor(x, device="cuda") for x in zip(*moves))
    for pool in st["kc"] + st["vc"]:
        full = _codes([pool])[0].to(torch.float64)
        full[db, do] = full[sb, so]
        outs.append(full)
    return outs
