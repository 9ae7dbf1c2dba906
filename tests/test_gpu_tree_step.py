"""A tree step as a serving loop runs it: the nodes' K/V rotated and appended, the tree's attention, the accepted path,
the cache made to hold it, and the next decode; against the same tokens appended one after another without branches."""
import math
import random

import pytest
import torch

import paged_kv_cache_156_gb300 as pkv
from tree_cases import ancestors, signed, tree

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_error_word():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pkv.device_error(reset=True)
    yield
    assert pkv.device_error(reset=True) == 0


@pytest.mark.parametrize("planned", [False, True])
@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_tree_step(pool, planned):
    Hq, Hkv, d, bs, V, layers = 16, 4, 128, 16, 200, 2
    old, news = [37, 500, 0, 129], [20, 64, 7, 33]
    B, T = len(old), sum(news)
    r, g = random.Random(1), torch.Generator().manual_seed(2)
    dt, dev = torch.bfloat16, "cuda"
    scale = d ** -0.5
    trees = [tree(r, n, 0.5) for n in news]
    depth = []
    for t in trees:
        for i, p in enumerate(t):
            depth.append(0 if i == 0 else depth[len(depth) - i + p] + 1)
    angles = torch.arange(1000, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    cos_sin = torch.cat([angles.cos(), angles.sin()], 1).float().cuda()
    bm = pkv.BlockManager(200, bs, torch.randperm(200, generator=g).numpy())
    for s in range(B):
        bm.allocate(s, old[s] + news[s])                      # the prompt, and places for the nodes
    tables, lens = (torch.from_numpy(x) for x in bm.block_tables(range(B), 40))
    assert lens.tolist() == [a + n for a, n in zip(old, news)]

    def slot(s, pos):
        return int(tables[s, pos // bs]) * bs + pos % bs

    starts = [sum(news[:i]) for i in range(B + 1)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    i64 = lambda x: torch.tensor(x, dtype=torch.int64, device=dev)
    kw = dict(k_scale=torch.full((Hkv,), 0.02, device=dev), v_scale=torch.full((Hkv,), 0.015, device=dev)) if pool == "e4m3" else {}

    def fresh():
        if pool == "e4m3":
            return [torch.zeros(200, bs, Hkv, d, dtype=torch.uint8, device=dev) for _ in range(layers)]
        return [torch.zeros(200, bs, Hkv, d, dtype=dt, device=dev) for _ in range(layers)]

    rows = lambda n, h: torch.randn(n, h, d, generator=g).to(dt).cuda()
    P = sum(old)
    prompt = [(rows(P, Hkv), rows(P, Hkv)) for _ in range(layers)]
    nodes = [(rows(T, Hq), rows(T, Hkv), rows(T, Hkv)) for _ in range(layers)]
    prompt_slots = i64([slot(s, p) for s in range(B) for p in range(old[s])])
    prompt_pos = i32([p for s in range(B) for p in range(old[s])])

    def load_prompt(kc, vc):
        for l in range(layers):
            pkv.paged_kv_append_rotary(None, None, *prompt[l], kc[l], vc[l], prompt_slots, prompt_pos, cos_sin, **kw)

    # ---- the tree step
    kc, vc = fresh(), fresh()
    load_prompt(kc, vc)
    seq_lens, query_starts, dev_tables = lens.cuda(), i32(starts), tables.cuda()
    mask = torch.tensor(signed([w for t in trees for w in ancestors(t)]), device=dev)
    node_slots = i64([slot(s, old[s] + i) for s in range(B) for i in range(news[s])])
    node_pos = i32([old[s] + depth[starts[s] + i] for s in range(B) for i in range(news[s])])
    ws = pkv.alloc_prefill_workspace(B, T, Hq, Hkv, d)
    top = int(lens.max())
    if planned:
        pkv.prefill_plan(ws, seq_lens, query_starts, T, Hq, Hkv, d, top)
    outs, turned = [], []
    for l in range(layers):
        q, k, v = nodes[l]
        q = q.clone()
        pkv.paged_kv_append_rotary(q, q, k, v, kc[l], vc[l], node_slots, node_pos, cos_sin, **kw)     # (queries in place)
        out = torch.empty_like(q)
        pkv.paged_attention_tree(out, q, kc[l], vc[l], dev_tables, seq_lens, query_starts, mask, scale, max_seq_len=top,
                                 workspace=ws, planned=planned, **kw)
        outs.append(out)
        turned.append(q)
    probs = torch.softmax(4 * torch.randn(T, V, generator=g), -1)
    drafts = torch.zeros(T, dtype=torch.int64)
    for s, t in enumerate(trees):
        kids = {}
        for i, p in enumerate(t[1:], 1):
            k = kids[p] = kids.get(p, -1) + 1
            drafts[starts[s] + i] = probs[starts[s] + p].topk(8).indices[min(k, 7)]
    W = 10
    tokens, path = torch.empty(B, W, dtype=torch.int64, device=dev), torch.empty(B, W, dtype=torch.int32, device=dev)
    count = torch.empty(B, dtype=torch.int32, device=dev)
    pkv.speculative_accept_tree(tokens, path, count, drafts.cuda(), i32([p for t in trees for p in t]), query_starts,
                                probs.cuda(), torch.rand(T, generator=g).cuda())
    pkv.paged_kv_keep_path(kc, vc, dev_tables, seq_lens, query_starts, path, count)
    kept_lens = (seq_lens - query_starts.diff() + count + 1).int()
    last = torch.gather(path, 1, count[:, None].long())[:, 0] + query_starts[:-1]      # the path's last nodes' rows
    decoded = []
    for l in range(layers):
        out = torch.empty(B, Hq, d, dtype=dt, device=dev)
        q = turned[l][last.long()].contiguous()
        if pool == "e4m3":
            pkv.paged_attention_decode_fp8(out, q, kc[l], vc[l], dev_tables, kept_lens, scale=scale, max_seq_len=top, **kw)
        else:
            pkv.paged_attention_decode(out, q, kc[l], vc[l], dev_tables, kept_lens, scale, max_seq_len=top)
        decoded.append(out)
    torch.cuda.synchronize()
    a, paths = count.tolist(), path.tolist()
    assert sum(a) > 0 and all(x < W for x in a)
    for s in range(B):
        p = paths[s][:a[s] + 1]
        assert p[0] == 0 and all(trees[s][j] == i for i, j in zip(p, p[1:])) and paths[s][a[s] + 1:] == [-1] * (W - a[s] - 1)
        assert tokens[s, :a[s]].tolist() == [int(drafts[starts[s] + j]) for j in p[1:]] and 0 <= int(tokens[s, a[s]]) < V

    # ---- the accepted tokens alone, one after another
    want_k, want_v = fresh(), fresh()
    load_prompt(want_k, want_v)
    pick = [(s, i, j) for s in range(B) for i, j in enumerate(paths[s][:a[s] + 1])]
    at = i64([starts[s] + j for s, i, j in pick])
    for l in range(layers):
        _, k, v = nodes[l]
        pkv.paged_kv_append_rotary(None, None, k[at], v[at], want_k[l], want_v[l], i64([slot(s, old[s] + i) for s, i, j in pick]),
                                   i32([old[s] + i for s, i, j in pick]), cos_sin, **kw)
    raw = torch.uint8 if pool == "e4m3" else torch.int16
    for l in range(layers):
        for got, want in ((kc[l], want_k[l]), (vc[l], want_v[l])):
            for s in range(B):
                where = torch.tensor([slot(s, p) for p in range(old[s] + a[s] + 1)])
                assert torch.equal(got.flatten(0, 1).cpu()[where].view(raw), want.flatten(0, 1).cpu()[where].view(raw))
        # the path's last node in the tree, and as the sequence's last token: the same attention but for roundings.  Both
        # round their weights (bf16 2^-8, f16 over E4M3 pools) and their output (2^-8): with |V| up to 448 * 0.015 or 5.5 they
        # stay within 2 (2^-8 + 2^-8) of the largest |V|
        err = (outs[l][last.long()].float() - decoded[l].float()).abs().max()
        assert float(err) <= 4 * 2.0 ** -8 * 6.72
    assert math.isfinite(float(decoded[0].float().sum()))
