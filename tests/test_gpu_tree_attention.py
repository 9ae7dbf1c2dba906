"""GPU parity of paged_attention_tree against a plain 64-bit reference.

Every output element is held to the bound that tree_cases.reference derives from
the roundings.  The batches cover single nodes to the largest trees, several
tiles of rows a KV head, trees that cross blocks and 128-position steps, caches
shorter than the tree, masks that leave a node nothing, tiles split over a long
cache, both pool types, and values that must not reach an output.
"""
import math
import random

import pytest
import torch

import paged_kv_cache_156_gb300 as pkv
from prefill_cases import build, check
from tree_cases import ancestors, masks, reference, seen_of, signed

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_error_word():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pkv.device_error(reset=True)
    yield
    assert pkv.device_error(reset=True) == 0


def run(b, mask, **kw):
    out = torch.full_like(b.q, math.nan)
    pkv.paged_attention_tree(out, b.q, b.kc, b.vc, b.tables, b.lens, b.starts, mask.to(b.q.device), b.scale,
                             max_seq_len=b.max_len, k_scale=b.k_scale, v_scale=b.v_scale, **kw)
    return out


def same(x, y):
    return torch.equal(x.view(torch.int16), y.view(torch.int16))


# nodes, totals, heads, kv heads, dim, block, dtype
CASES = {
    "one_node": ([1], [1], 1, 1, 64, 16, "f16"),
    "two_blocks": ([5], [17], 4, 4, 128, 16, "bf16"),
    "small_step": ([1, 8, 5, 2], [1, 17, 33, 50], 4, 4, 64, 16, "f16"),
    "largest": ([64, 63, 64], [64, 200, 1000], 4, 2, 128, 16, "bf16"),
    "across_steps": ([40, 64, 33, 2], [128 + 20, 256 + 1, 384 + 32, 129], 2, 1, 128, 16, "f16"),
    "across_steps_d64": ([40, 64, 33, 2], [128 + 63, 256 + 64, 384 + 32, 128], 3, 1, 64, 8, "bf16"),
    "tile_edges_g4": ([31, 32, 33, 63, 64], [31, 32, 200, 63, 511], 8, 2, 128, 8, "f16"),
    "two_items_g8": ([33, 64, 32], [300, 1300, 32], 16, 2, 128, 32, "bf16"),
    "group_7": ([20, 37, 1], [20, 500, 129], 7, 1, 128, 32, "bf16"),
    "group_40": ([5, 13], [5, 300], 40, 1, 64, 32, "f16"),
    "empty_sequences": ([0, 5, 0, 0, 9, 0], [0, 5, 100, 0, 200, 7], 4, 2, 128, 16, "f16"),
    "shorter_than_the_tree": ([10, 64, 4, 64], [3, 0, 200, 63], 4, 2, 128, 16, "bf16"),
    "long_cache": ([33, 2], [9000, 5001], 16, 2, 128, 32, "bf16"),
    "long_cache_d64": ([3, 40], [7777, 6000], 8, 1, 64, 8, "f16"),
    "long_tree_in_two_parts": ([64], [4096 + 20], 2, 1, 128, 16, "bf16"),
    "many": ([(7 * i) % 65 for i in range(40)], [(7 * i) % 65 + 11 * i for i in range(40)], 8, 2, 128, 16, "bf16"),
}


@pytest.mark.parametrize("name", CASES)
def test_matches_the_reference(name):
    news, totals, heads, kv_heads, dim, block, dtype = CASES[name]
    b = build(news, totals, heads, kv_heads, dim, block, dtype, seed=len(name), pad_rows=3, gap=2)
    mask, _ = masks(news, len(name), gap=2, pad_rows=3)
    ref, bound = reference(b, mask)
    out = run(b.to("cuda"), mask)
    torch.cuda.synchronize()
    print(f"{name}: {check(out, ref, bound, name):.3f} of the bound")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("name", [n for n in CASES if n not in ("one_node", "small_step")])
def test_e4m3_matches_the_reference(name, dtype):
    """The products run in f16 whatever the queries' type: the weights round there."""
    news, totals, heads, kv_heads, dim, block, _ = CASES[name]
    b = build(news, totals, heads, kv_heads, 128, block, dtype, seed=len(name), pad_rows=3, gap=2, e4m3=True)
    mask, _ = masks(news, len(name), gap=2, pad_rows=3)
    ref, bound = reference(b, mask, torch.float16)
    out = run(b.to("cuda"), mask)
    torch.cuda.synchronize()
    print(f"{name}: {check(out, ref, bound, name):.3f} of the bound")


@pytest.mark.parametrize("e4m3", [False, True])
def test_any_mask(e4m3):
    """Masks that are no tree's: nothing, itself only, everything, random bits, bits past the node and past the tree."""
    r = random.Random(3)
    news, totals = [64, 50, 64, 7], [64, 51, 700, 5]
    words = [0, 1 << 63, (1 << 64) - 1]
    words = [r.choice(words) if r.random() < 0.5 else r.getrandbits(64) & r.getrandbits(64) for _ in range(sum(news))]
    mask = torch.tensor(signed(words))
    for dim, heads, kv_heads in ((128, 4, 2), (64, 3, 1))[:1 if e4m3 else 2]:
        b = build(news, totals, heads, kv_heads, dim, 16, "bf16", seed=4, e4m3=e4m3)
        ref, bound = reference(b, mask, torch.float16 if e4m3 else None)
        none = torch.cat([~seen_of(b, mask, s).any(1) for s in range(len(news))])
        assert none.sum() > 5                           # some nodes see nothing
        out = run(b.to("cuda"), mask)
        torch.cuda.synchronize()
        check(out, ref, bound, f"dim {dim}")
        assert not out[none.cuda()].any()


@pytest.mark.parametrize("dtype,heads,kv_heads,dim,e4m3", [("bf16", 8, 2, 128, False), ("f16", 3, 1, 64, False),
                                                            ("f16", 8, 2, 128, True)])
def test_all_ones_is_the_prefill_call(dtype, heads, kv_heads, dim, e4m3):
    """A chain's mask, and all ones, give what the prefill call gives, bit for bit."""
    news, totals = [64, 5, 1, 40], [700, 9000, 257, 40]
    b = build(news, totals, heads, kv_heads, dim, 16, dtype, seed=5, e4m3=e4m3).to("cuda")
    want = torch.full_like(b.q, math.nan)
    pkv.paged_attention_prefill(want, b.q, b.kc, b.vc, b.tables, b.lens, b.starts, b.scale, max_seq_len=b.max_len,
                                k_scale=b.k_scale, v_scale=b.v_scale)
    ones = torch.full((sum(news),), -1, dtype=torch.int64)
    chain = torch.tensor(signed([(1 << (i + 1)) - 1 for n in news for i in range(n)]))
    assert same(run(b, ones), want) and same(run(b, chain), want)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("where", ["k", "v", "kv"])
@pytest.mark.parametrize("dtype,heads,kv_heads,dim", [("bf16", 8, 2, 128), ("f16", 3, 1, 64)])
def test_values_a_node_does_not_see_do_not_reach_it(bad, where, dtype, heads, kv_heads, dim):
    """Non-finite K and V of a few nodes: every node that sees none of them gives the clean run's output, bit for bit;
    one that sees them what the sums give."""
    news, totals = [64, 9, 30, 1], [700, 900, 257, 3]
    mask, _ = masks(news, 6, chain=0.3)
    hit = [[3, 40, 63], [4, 8], [0, 17], []]
    clean = run(build(news, totals, heads, kv_heads, dim, 16, dtype, seed=5).to("cuda"), mask)
    b = build(news, totals, heads, kv_heads, dim, 16, dtype, seed=5)
    for s, nodes in enumerate(hit):
        for k, j in enumerate(nodes):
            pos = totals[s] - news[s] + j
            blk = int(b.tables[s, pos // 16])
            if "k" in where:
                b.kc[blk, pos % 16] = bad
            if "v" in where:
                b.vc[blk, pos % 16, :, k::3] = bad
    got = run(b.to("cuda"), mask)
    torch.cuda.synchronize()
    for s, n in enumerate(news):
        for i in range(n):
            r = int(b.starts[s]) + i
            sees = [k for k, j in enumerate(hit[s]) if int(mask[r]) >> j & 1]
            if not sees:
                assert same(got[r], clean[r]), (s, i)
            elif where == "v":
                for c in range(dim):
                    x = got[r, :, c].float().cpu()
                    if c % 3 not in sees:
                        assert torch.isfinite(x).all(), (s, i, c)
                    elif math.isnan(bad):
                        assert torch.isnan(x).all(), (s, i, c)
                    else:
                        assert (x == bad).all(), (s, i, c)


def test_opposite_infinities_and_those_every_node_sees():
    b = build([40], [200], 4, 1, 64, 16, "bf16", seed=6)
    mask = torch.tensor(signed(ancestors([-1] + [0] * 39)))         # a root and 39 children

    def put(pos, v, col):
        b.vc[int(b.tables[0, pos // 16]), pos % 16, 0, col] = v

    put(160, math.inf, 7)               # the root: every node sees it
    put(165, -math.inf, 7)              # node 5
    put(170, math.inf, 9)               # node 10
    put(100, -math.inf, 9)              # before the tree
    put(20, math.nan, 11)
    got = run(b.to("cuda"), mask)
    torch.cuda.synchronize()
    rest = [i for i in range(40) if i != 5]
    assert torch.isnan(got[5, :, 7]).all() and (got[rest, :, 7] == math.inf).all()
    rest = [i for i in range(40) if i != 10]
    assert torch.isnan(got[10, :, 9]).all() and (got[rest, :, 9] == -math.inf).all()
    assert torch.isnan(got[:, :, 11]).all()
    got[:, :, [7, 9, 11]] = 0
    assert torch.isfinite(got).all()


def test_bad_values_over_many_items():
    """Non-finite V in some sequences' trees and not in their neighbours', more items than the tables' turns: none leaks
    into the next."""
    news = [(13 * i) % 40 + 1 for i in range(300)]
    totals = [n + (37 * i) % 300 for i, n in enumerate(news)]
    b = build(news, totals, 8, 8, 64, 16, "bf16", seed=8)
    mask, _ = masks(news, 9)
    clean = run(b.to("cuda"), mask)
    bad = {}
    r = random.Random(10)
    for s in range(0, 300, 3):
        j = r.randrange(news[s])
        pos = totals[s] - news[s] + j
        h, c = r.randrange(8), r.randrange(64)
        b.vc[int(b.tables[s, pos // 16]), pos % 16, h, c] = r.choice([math.nan, math.inf, -math.inf])
        bad[s] = (j, h, c)
    got = run(b.to("cuda"), mask).float().cpu()
    clean = clean.float().cpu()
    for s in range(300):
        for i in range(news[s]):
            row = int(b.starts[s]) + i
            want = clean[row].clone()
            if s in bad and int(mask[row]) >> bad[s][0] & 1:
                _, h, c = bad[s]
                assert not math.isfinite(got[row, h, c])
                got[row, h, c] = want[h, c]
            assert torch.equal(got[row], want), (s, i)


def test_e4m3_codes_a_node_does_not_see():
    """NaN codes in one node's K and V: nodes that do not see it are the clean run's bit for bit."""
    news, totals = [64, 9, 30], [700, 900, 130]
    mask, _ = masks(news, 12, chain=0.3)

    def batch():
        return build(news, totals, 8, 2, 128, 16, "bf16", seed=5, e4m3=True)

    clean = run(batch().to("cuda"), mask)
    for where in ("v", "k"):
        b = batch()
        hit = [3, 4, 17]
        for s, j in enumerate(hit):
            pos = totals[s] - news[s] + j
            blk = int(b.tables[s, pos // 16])
            if where == "v":
                b.vc[blk, pos % 16, 1, 5] = 0x7f
                b.vc[blk, pos % 16, 1, 70] = 0xff
            else:
                b.kc[blk, pos % 16] = 0x7f
        got = run(b.to("cuda"), mask)
        torch.cuda.synchronize()
        for s, n in enumerate(news):
            for i in range(n):
                r = int(b.starts[s]) + i
                if int(mask[r]) >> hit[s] & 1:
                    if where == "k":
                        assert torch.isnan(got[r]).all()
                    else:
                        assert torch.isnan(got[r, 4:, [5, 70]]).all() and torch.isnan(got[r]).sum() == 8
                else:
                    assert same(got[r], clean[r]), (s, i)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("nodes,heads,kv_heads,block", [(16, 16, 2, 8), (32, 4, 1, 32), (5, 9, 3, 16), (25, 10, 2, 8), (64, 4, 2, 32),
                                                         (1, 64, 8, 16), (2, 128, 2, 8), (3, 40, 1, 32)])
def test_e4m3_trees_of_one_size(nodes, heads, kv_heads, block, dtype):
    """Up to 128 rows a KV head and sequence: one tile each, over one to many steps, with nodes on either side of a step's
    and a block's end, caches shorter than the tree, and positions that are not there."""
    totals = [nodes, 0, nodes // 2, 127, 128, 129, 128 + nodes, 256, 257, 256 + nodes // 2, 383, 640, 1000, 2500, 4096, 4097]
    news = [nodes] * len(totals)
    b = build(news, totals, heads, kv_heads, 128, block, dtype, seed=nodes, pad_rows=len(totals), e4m3=True)
    mask, _ = masks(news, nodes, pad_rows=len(totals))
    ref, bound = reference(b, mask, torch.float16)
    out = run(b.to("cuda"), mask)
    torch.cuda.synchronize()
    print(f"{check(out, ref, bound):.3f} of the bound")


@pytest.mark.parametrize("e4m3", [False, True])
def test_more_sequences_than_a_plan_chunk(e4m3):
    """More than 1024 sequences (the plan kernel reloads them in chunks), some without nodes."""
    r = random.Random(1)
    news = [r.randint(0, 5) for _ in range(1500)]
    totals = [n + r.randint(0, 300) for n in news]
    b = build(news, totals, 4, 2, 128, 16, "bf16", seed=60, e4m3=e4m3)
    mask, _ = masks(news, 61)
    ref, bound = reference(b, mask, torch.float16 if e4m3 else None)
    out = run(b.to("cuda"), mask)
    torch.cuda.synchronize()
    check(out, ref, bound)


@pytest.mark.parametrize("planned", [False, True])
@pytest.mark.parametrize("totals", [[100, 33, 200], [9000, 140, 4000], [64, 1, 70]])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_e4m3_one_tree_larger_than_the_rest(dtype, totals, planned):
    """Few rows a sequence on average, but one of two tiles: over E4M3 pools its tiles follow one another; split tiles,
    trees shorter than the rest's, sequences without nodes."""
    news = [64, 1, 33, 0, 2, 1, 1, 1, 3, 1, 1, 1, 1]
    totals = totals + [0 if n == 0 else n + 130 * i for i, n in enumerate(news[3:])]
    b = build(news, totals, 8, 2, 128, 16, dtype, seed=60, pad_rows=2, e4m3=True)
    mask, _ = masks(news, 61, pad_rows=2)
    ref, bound = reference(b, mask, torch.float16)
    c, kw = b.to("cuda"), {}
    if planned:
        ws = pkv.alloc_prefill_workspace(len(news), c.q.shape[0], 8, 2, 128)
        pkv.prefill_plan(ws, c.lens, c.starts, c.q.shape[0], 8, 2, 128, c.max_len)
        kw = dict(workspace=ws, planned=True)
    out = run(c, mask, **kw)
    torch.cuda.synchronize()
    check(out, ref, bound)


def test_e4m3_bad_codes_over_many_items():
    """Many small trees, NaN codes in some of them: no other tree's output changes, nor a node's that does not see them."""
    news = [(5 * i) % 16 + 1 for i in range(260)]
    totals = [n + (37 * i) % 300 for i, n in enumerate(news)]
    b = build(news, totals, 16, 8, 128, 16, "bf16", seed=62, e4m3=True)
    mask, _ = masks(news, 63)
    ref, bound = reference(b, mask, torch.float16)
    clean = run(b.to("cuda"), mask)
    check(clean, ref, bound)
    r, bad = random.Random(64), {}
    for s in range(0, 260, 3):
        j = r.randrange(news[s])
        pos = totals[s] - news[s] + j
        h, c = r.randrange(8), r.randrange(128)
        b.vc[int(b.tables[s, pos // 16]), pos % 16, h, c] = r.choice([0x7f, 0xff])
        bad[s] = (j, h, c)
    got, clean = run(b.to("cuda"), mask).float().cpu(), clean.float().cpu()
    for s in range(260):
        for i in range(news[s]):
            row = int(b.starts[s]) + i
            if s in bad and int(mask[row]) >> bad[s][0] & 1:
                _, h, c = bad[s]
                assert torch.isnan(got[row, 2 * h:2 * h + 2, c]).all()
                got[row, 2 * h:2 * h + 2, c] = clean[row, 2 * h:2 * h + 2, c]
            assert torch.equal(got[row], clean[row]), (s, i)


def test_all_visible_scores_minus_infinity():
    """A node all of whose visible scores are -inf is NaN, in split tiles too; one that sees a finite score beside them is
    not."""
    for totals in ([64 + 3], [6000]):
        b = build([3], totals, 4, 1, 128, 16, "bf16", seed=13)
        b.q[:] = b.q.abs()
        L = totals[0]
        for pos in range(L):
            b.kc[int(b.tables[0, pos // 16]), pos % 16] = -math.inf
        b.kc[int(b.tables[0, (L - 1) // 16]), (L - 1) % 16] = 1.0      # node 2
        got = run(b.to("cuda"), torch.tensor([0b1, 0b11, 0b100]))
        torch.cuda.synchronize()
        assert torch.isnan(got[:2]).all()
        v = b.vc[int(b.tables[0, (L - 1) // 16]), (L - 1) % 16, 0]
        assert torch.equal(got[2].cpu(), v.expand(4, 128))


@pytest.mark.parametrize("scale", [0.0, -0.09, 3.0, 1e-20])
@pytest.mark.parametrize("e4m3", [False, True])
def test_scales(scale, e4m3):
    news, totals = [50, 1, 64], [70, 500, 900]
    b = build(news, totals, 4, 2, 128, 16, "bf16", seed=8, scale=scale, e4m3=e4m3)
    if e4m3:
        b.k_scale *= torch.tensor([-1.0, 3.0])
    mask, _ = masks(news, 14)
    ref, bound = reference(b, mask, torch.float16 if e4m3 else None)
    out = run(b.to("cuda"), mask)
    torch.cuda.synchronize()
    check(out, ref, bound, f"scale {scale}")


@pytest.mark.parametrize("nodes", [20, 64])
def test_e4m3_zero_scales(nodes):
    """A KV head whose K scale is zero weighs every visible position alike; a zero V scale gives zeros."""
    news, totals = [nodes] * 3, [nodes, 700, 300]
    b = build(news, totals, 16, 4, 128, 16, "f16", seed=11, e4m3=True)
    b.k_scale[1] = 0.0
    b.v_scale[2] = 0.0
    mask, _ = masks(news, 12)
    ref, bound = reference(b, mask, torch.float16)
    out = run(b.to("cuda"), mask)
    torch.cuda.synchronize()
    check(out, ref, bound)
    assert not out[:, 8:12].any()


@pytest.mark.parametrize("e4m3", [False, True])
def test_rows_of_larger_tensors(e4m3):
    """q and out are rows of larger tensors; a group that no TMA box fits (24 rows a token)."""
    news, totals = [5, 1, 9], [400, 30, 9]
    b = build(news, totals, 24, 1, 128, 32, "bf16", seed=17, e4m3=e4m3)
    mask, _ = masks(news, 18)
    ref, bound = reference(b, mask, torch.float16 if e4m3 else None)
    c = b.to("cuda")
    wide_q, wide_out = (torch.full((40, 24, 128), math.nan, dtype=c.q.dtype, device="cuda") for _ in range(2))
    wide_q[7:22] = c.q
    pkv.paged_attention_tree(wide_out[7:22], wide_q[7:22], c.kc, c.vc, c.tables, c.lens, c.starts, mask.cuda(), c.scale,
                             max_seq_len=c.max_len, k_scale=c.k_scale, v_scale=c.v_scale)
    torch.cuda.synchronize()
    check(wide_out[7:22], ref, bound)
    assert torch.isnan(wide_out[:7]).all() and torch.isnan(wide_out[22:]).all()


def test_plans_are_shared_with_the_prefill_call():
    """prefill_plan's plan serves a step's layers; another mask over the same plan is another answer."""
    news, totals = [1, 60, 3, 0, 33], [3000, 900, 3, 40, 77]
    layers = [build(news, totals, 8, 2, 128, 16, "bf16", seed=20 + i) for i in range(2)]
    ws = pkv.alloc_prefill_workspace(len(news), sum(news), 8, 2, 128)
    ws.fill_(0xA5)
    on = [b.to("cuda") for b in layers]
    pkv.prefill_plan(ws, on[0].lens, on[0].starts, sum(news), 8, 2, 128, on[0].max_len)
    for seed in (1, 2):
        mask, _ = masks(news, seed)
        for b, c in zip(layers, on):
            out = run(c, mask, workspace=ws, planned=True)
            torch.cuda.synchronize()
            ref, bound = reference(b, mask)
            check(out, ref, bound)
            assert same(out, run(c, mask))


def test_captured_and_replayed_on_new_inputs():
    news, totals = [1, 60, 40], [2100, 700, 40]
    b = build(news, totals, 8, 2, 128, 16, "bf16", seed=40).to("cuda")
    mask = torch.zeros(101, dtype=torch.int64, device="cuda")
    spaces = [pkv.alloc_prefill_workspace(3, 101, 8, 2, 128) for _ in range(2)]
    outs = [torch.full_like(b.q, math.nan) for _ in spaces]

    def step(out, ws):
        pkv.paged_attention_tree(out, b.q, b.kc, b.vc, b.tables, b.lens, b.starts, mask, b.scale, max_seq_len=2100, workspace=ws)

    step(outs[0], spaces[0])
    torch.cuda.synchronize()
    graphs = []
    for out, ws in zip(outs, spaces):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, capture_error_mode="relaxed"):
            step(out, ws)
        graphs.append(g)
    for rep in range(3):
        news = [1 + rep, 60 - 2 * rep, 40 + rep]
        new = build(news, [2100 - 500 * rep, 700 + rep, 40 + rep], 8, 2, 128, 16, "bf16", seed=41 + rep)
        m, _ = masks(news, 50 + rep)
        assert new.kc.shape[0] <= b.kc.shape[0] and new.q.shape == b.q.shape
        b.q.copy_(new.q)
        b.tables.fill_(-1)
        b.tables[:, :new.tables.shape[1]].copy_(new.tables[:, :b.tables.shape[1]])
        b.kc[:new.kc.shape[0]].copy_(new.kc)
        b.vc[:new.vc.shape[0]].copy_(new.vc)
        b.lens.copy_(new.lens)
        b.starts.copy_(new.starts)
        mask.copy_(m)
        for o in outs:
            o.fill_(math.nan)
        torch.cuda.synchronize()
        for g in graphs:                                    # both at once, each over its own workspace
            with torch.cuda.stream(torch.cuda.Stream()):
                g.replay()
        torch.cuda.synchronize()
        ref, bound = reference(new, m)
        check(outs[0], ref, bound, f"replay {rep}")
        assert same(outs[0], outs[1])


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace, give what they give one after the other: both pool types, few rows
    and many."""
    shapes = [([30, 1, 64], [900, 3000, 64], 8, 2, False), ([26] * 6, [26 + 700 * i for i in range(6)], 8, 2, True),
              ([64, 50], [6000, 1200], 16, 2, True)]
    bs = [build(news, totals, hq, hk, 128, 16, "bf16", seed=13 + i, e4m3=e).to("cuda")
          for i, (news, totals, hq, hk, e) in enumerate(shapes)]
    ms = [masks(news, 70)[0].cuda() for news, *_ in shapes]
    want = [run(b, m) for b, m in zip(bs, ms)]
    streams = [torch.cuda.Stream() for _ in bs]
    spaces = [pkv.alloc_prefill_workspace(len(b.lens), b.q.shape[0], b.q.shape[1], 2, 128) for b in bs]
    outs = [[torch.full_like(b.q, math.nan) for _ in range(8)] for b in bs]
    torch.cuda.synchronize()
    for i in range(8):
        for b, m, s, ws, out in zip(bs, ms, streams, spaces, outs):
            with torch.cuda.stream(s):
                pkv.paged_attention_tree(out[i], b.q, b.kc, b.vc, b.tables, b.lens, b.starts, m, b.scale, max_seq_len=b.max_len,
                                         workspace=ws, k_scale=b.k_scale, v_scale=b.v_scale)
    torch.cuda.synchronize()
    for w, out in zip(want, outs):
        assert all(same(o, w) for o in out)


def test_on_another_stream_and_without_a_workspace():
    news = [50, 1]
    b = build(news, [300, 2000], 4, 2, 64, 8, "f16", seed=50)
    mask, _ = masks(news, 51)
    c, m = b.to("cuda"), mask.cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = torch.full_like(c.q, math.nan)
        pkv.paged_attention_tree(out, c.q, c.kc, c.vc, c.tables, c.lens, c.starts, m)
    s.synchronize()
    ref, bound = reference(b, mask)
    check(out, ref, bound)


def test_more_than_64_nodes_raise_the_error_word():
    """Such a sequence is left out, the others' outputs are right."""
    news, totals = [65, 20, 200], [300, 40, 2500]
    b = build(news, totals, 4, 2, 128, 16, "bf16", seed=80)
    mask = torch.full((sum(news),), -1, dtype=torch.int64)
    mask[65:85] = masks([20], 81)[0]
    out = run(b.to("cuda"), mask)
    torch.cuda.synchronize()
    assert pkv.device_error(reset=True) == 1
    b.starts, b.lens, b.tables = torch.tensor([65, 85], dtype=torch.int32), b.lens[1:2], b.tables[1:2]
    ref, bound = reference(b, mask)
    check(out[65:85], ref[65:85], bound[65:85])


def test_bad_ids_lengths_and_starts_raise_the_error_word():
    def word(**change):
        b = build([20, 3], [300, 40], 4, 2, 128, 16, "bf16", seed=80)
        for k, f in change.items():
            f(getattr(b, k))
        run(b.to("cuda"), torch.full((23,), -1, dtype=torch.int64))
        torch.cuda.synchronize()
        return pkv.device_error(reset=True)

    def put(i, v):
        return lambda t: t.view(-1).__setitem__(i, v)

    assert word() == 0
    assert word(tables=put(2, 1 << 30)) == 1 and word(tables=put(3, -5)) == 1 and word(lens=put(0, 301)) == 1
    for i, v in ((0, -1), (1, 24), (2, 19), (2, 1 << 20)):      # starts before the first row, past the last, decreasing
        assert word(starts=put(i, v)) == 1, (i, v)


def test_repeats_bit_for_bit():
    news = [33, 1, 64]
    b = build(news, [5000, 1200, 600], 8, 2, 128, 16, "bf16", seed=100).to("cuda")
    mask, _ = masks(news, 101)
    first = run(b, mask)
    for _ in range(5):
        assert same(run(b, mask), first)


def test_offsets_past_32_bits():
    """Blocks past the pool's first 2^31 elements, query rows past q's and out's first 2^31."""
    news = [30, 1, 64]
    b = build(news, [100, 900, 300], 32, 8, 128, 32, "bf16", seed=15)
    mask, _ = masks(news, 16)
    ref, bound = reference(b, mask)
    NB = 2 ** 31 // (32 * 8 * 128) + b.kc.shape[0]
    T = 2 ** 31 // (32 * 128) + 1 + b.q.shape[0]
    c = b.to("cuda")
    far = []
    for pool in (c.kc, c.vc):
        x = torch.empty(NB, 32, 8, 128, dtype=torch.bfloat16, device="cuda")
        x[NB - pool.shape[0]:] = pool
        far.append(x)
    q = torch.empty(T, 32, 128, dtype=torch.bfloat16, device="cuda")
    q[T - c.q.shape[0]:] = c.q
    out = torch.full_like(q, math.nan)
    m = torch.zeros(T, dtype=torch.int64, device="cuda")
    m[T - c.q.shape[0]:] = mask.cuda()
    ids = torch.where(c.tables < b.kc.shape[0], c.tables + (NB - b.kc.shape[0]), NB + 7).int()
    pkv.paged_attention_tree(out, q, far[0], far[1], ids, c.lens, c.starts + (T - c.q.shape[0]), m, c.scale,
                             max_seq_len=c.max_len)
    torch.cuda.synchronize()
    check(out[T - c.q.shape[0]:], ref, bound)
    assert torch.isnan(out[T - c.q.shape[0] - 300:T - c.q.shape[0]]).all()
