"""A tree step's attention and the cache it leaves, each row held to a bound from its own sums.

The drafted nodes' keys and queries share a direction that the rotation hardly turns, so that the nodes carry most of every
node's weight, whatever the prompt's length: one node too few or too many, or a position too early, moves some element of a
row by more than its bound.  That is shown on the reference itself, beside the kernel's outputs, sequence by sequence.
"""
import random

import pytest
import torch

import paged_kv_cache_156_gb300 as pkv
from prefill_cases import DT, Batch
from tree_cases import ancestors, reference, signed, tree

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_error_word():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pkv.device_error(reset=True)
    yield
    assert pkv.device_error(reset=True) == 0


@pytest.mark.parametrize("pool", ["f16", "bf16", "e4m3"])
def test_rows_within_their_own_bounds(pool):
    Hq, Hkv, d, bs, W, dev = 8, 2, 128, 16, 12, "cuda"
    old, news = [37, 500, 0, 129], [20, 64, 7, 33]
    B, T, V = len(old), sum(news), 50
    dt = DT["bf16" if pool == "e4m3" else pool]
    r, g = random.Random(11), torch.Generator().manual_seed(12)
    trees = [tree(r, n, 0.5) for n in news]
    starts = [sum(news[:i]) for i in range(B + 1)]
    depth = []
    for t in trees:
        at = len(depth)
        for i, p in enumerate(t):
            depth.append(0 if i == 0 else depth[at + p] + 1)
    angles = torch.arange(1000, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    cos_sin = torch.cat([angles.cos(), angles.sin()], 1).float().cuda()
    bm = pkv.BlockManager(120, bs, torch.randperm(120, generator=g).numpy())
    for s in range(B):
        bm.allocate(s, old[s] + news[s])
    tables, lens = (torch.from_numpy(x) for x in bm.block_tables(range(B), 40))
    slot = lambda s, pos: int(tables[s, pos // bs]) * bs + pos % bs
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    i64 = lambda x: torch.tensor(x, dtype=torch.int64, device=dev)
    kw = dict(k_scale=torch.full((Hkv,), 0.02, device=dev), v_scale=torch.full((Hkv,), 0.015, device=dev)) if pool == "e4m3" else {}
    fresh = lambda: torch.zeros(120, bs, Hkv, d, dtype=torch.uint8 if pool == "e4m3" else dt, device=dev)

    # elements 48 to 63 of each half turn by less than 0.002 a position: the nodes' scores are about 6 above the prompt's
    common = torch.zeros(d)
    common[48:64] = common[112:128] = 1.46
    rows = lambda n, h, c: (torch.randn(n, h, d, generator=g) + c).to(dt).cuda()
    P = sum(old)
    pk, pv = rows(P, Hkv, 0.0), rows(P, Hkv, 0.0)
    q, k, v = rows(T, Hq, common), rows(T, Hkv, common), rows(T, Hkv, 0.0)
    prompt = (i64([slot(s, p) for s in range(B) for p in range(old[s])]), i32([p for s in range(B) for p in range(old[s])]))

    kc, vc = fresh(), fresh()
    pkv.paged_kv_append_rotary(None, None, pk, pv, kc, vc, *prompt, cos_sin, **kw)
    turned = torch.empty_like(q)
    pkv.paged_kv_append_rotary(turned, q, k, v, kc, vc, i64([slot(s, old[s] + i) for s in range(B) for i in range(news[s])]),
                               i32([old[s] + depth[starts[s] + i] for s in range(B) for i in range(news[s])]), cos_sin, **kw)
    words = [w for t in trees for w in ancestors(t)]
    seq_lens, query_starts, dev_tables, top = lens.cuda(), i32(starts), tables.cuda(), int(lens.max())
    out = torch.empty_like(q)
    pkv.paged_attention_tree(out, turned, kc, vc, dev_tables, seq_lens, query_starts, i64(signed(words)), d ** -0.5,
                             max_seq_len=top, **kw)
    on_host = lambda x, y, qq, ll, ss: Batch(qq.cpu(), x.cpu(), y.cpu(), tables, ll, ss, d ** -0.5, top,
                                             *(t.cpu() for t in kw.values()))
    work = torch.float16 if pool == "e4m3" else None
    step = on_host(kc, vc, turned, lens, torch.tensor(starts, dtype=torch.int32))
    ref, bound = reference(step, torch.tensor(signed(words)), work)
    off = (out.cpu().double() - ref).abs() / bound
    assert float(off.max()) <= 1.0
    # ---- the same reference with a mistake: an ancestor left out (not the node itself alone), another node let in, the
    # nodes a position early
    for s in range(B):
        at, n = starts[s], news[s]
        for name, i in (("the deepest", max(range(n), key=lambda j: depth[at + j])), ("the last", n - 1)):
            wrong = []
            for j in range(i + 1):
                bit = 1 << j
                if j == i and words[at + i] == bit and old[s] == 0:
                    continue                                  # (nothing would be left)
                wrong.append(words[at + i] ^ bit)
            for w in wrong:
                moved = words[:]
                moved[at + i] = w
                one = Batch(step.q, step.kc, step.vc, tables[s:s + 1], lens[s:s + 1],
                            torch.tensor([at, at + n], dtype=torch.int32), step.scale, top, step.k_scale, step.v_scale)
                other, _ = reference(one, torch.tensor(signed(moved)), work)
                miss = (other[at + i] - ref[at + i]).abs() / bound[at + i]
                assert float(miss.max()) > 2.0, (s, name, bin(w), float(miss.max()))
    # ---- the walk, the cache it leaves, and the next decode
    probs = torch.softmax(4 * torch.randn(T, V, generator=g), -1)
    drafts = torch.zeros(T, dtype=torch.int64)
    for s, t in enumerate(trees):
        kids = {}
        for i, p in enumerate(t[1:], 1):
            kids[p] = kids.get(p, -1) + 1
            drafts[starts[s] + i] = probs[starts[s] + p].topk(8).indices[min(kids[p], 7)]
    tokens, path = torch.empty(B, W, dtype=torch.int64, device=dev), torch.empty(B, W, dtype=torch.int32, device=dev)
    count = torch.empty(B, dtype=torch.int32, device=dev)
    pkv.speculative_accept_tree(tokens, path, count, drafts.cuda(), i32([p for t in trees for p in t]), query_starts,
                                probs.cuda(), torch.rand(T, generator=g).cuda())
    pkv.paged_kv_keep_path([kc], [vc], dev_tables, seq_lens, query_starts, path, count)
    kept = (seq_lens - query_starts.diff() + count + 1).int()
    last = (torch.gather(path, 1, count[:, None].long())[:, 0] + query_starts[:-1]).long()
    decode = pkv.paged_attention_decode_fp8 if pool == "e4m3" else pkv.paged_attention_decode
    after = torch.empty(B, Hq, d, dtype=dt, device=dev)
    decode(after, turned[last].contiguous(), kc, vc, dev_tables, kept, scale=d ** -0.5, max_seq_len=top, **kw)
    # the accepted tokens appended one after another, without branches
    a, paths = count.tolist(), path.tolist()
    assert sum(a) > 0
    pick = [(s, i, j) for s in range(B) for i, j in enumerate(paths[s][:a[s] + 1])]
    rows_of = i64([starts[s] + j for s, i, j in pick])
    want_k, want_v = fresh(), fresh()
    pkv.paged_kv_append_rotary(None, None, pk, pv, want_k, want_v, *prompt, cos_sin, **kw)
    pkv.paged_kv_append_rotary(None, None, k[rows_of], v[rows_of], want_k, want_v, i64([slot(s, old[s] + i) for s, i, j in pick]),
                               i32([old[s] + i for s, i, j in pick]), cos_sin, **kw)
    want = torch.empty_like(after)
    decode(want, turned[last].contiguous(), want_k, want_v, dev_tables, kept, scale=d ** -0.5, max_seq_len=top, **kw)
    torch.cuda.synchronize()
    assert torch.equal(after.view(torch.int16), want.view(torch.int16))       # the same rows in the same places
    # the path's last node saw in the tree what a sequence without branches holds: that sequence's reference and its bounds
    line = on_host(want_k, want_v, turned[last], kept.cpu(), torch.arange(B + 1, dtype=torch.int32))
    ref, bound = reference(line, torch.full((B,), -1, dtype=torch.int64), work)
    off = ((out[last].cpu().double() - ref).abs() / bound).flatten(1).amax(1)
    assert float(off.max()) <= 1.0, off
