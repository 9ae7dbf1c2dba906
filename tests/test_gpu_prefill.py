"""GPU parity of paged_attention_prefill against a plain 64-bit reference.

Every output element is held to the bound that prefill_cases.reference derives
from the roundings.  The batches cover one token to several tiles of new
tokens, empty sequences, tokens that see nothing, group sizes that do not
divide a tile, both head sizes, every block size, blocks that end inside a
step, tiles split over a long cache, and values that must not reach an output
(NaN slots, non-finite K/V a token does not see).
"""
import math

import pytest
import torch

import paged_kv_cache_156_gb300 as pkv
from prefill_cases import build, check, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_error_word():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pkv.device_error(reset=True)
    yield
    assert pkv.device_error(reset=True) == 0


def run(b, **kw):
    out = torch.full_like(b.q, math.nan)
    pkv.paged_attention_prefill(out, b.q, b.kc, b.vc, b.tables, b.lens, b.starts, b.scale, max_seq_len=b.max_len,
                                k_scale=b.k_scale, v_scale=b.v_scale, **kw)
    return out


# news, totals, heads, kv heads, dim, block, dtype
CASES = {
    "one_token": ([1], [1], 1, 1, 64, 16, "f16"),
    "two_blocks": ([3], [17], 4, 4, 128, 16, "bf16"),
    "small_step": ([1, 17, 5, 2], [1, 17, 33, 50], 4, 4, 64, 16, "f16"),
    "tile_edges_g1": ([127, 128, 129, 255, 256, 257], [127, 128, 129, 300, 256, 900], 2, 2, 128, 16, "bf16"),
    "tile_edges_g4": ([31, 32, 33, 63, 64, 65], [31, 32, 200, 63, 511, 65], 8, 2, 128, 8, "f16"),
    "group_3_d64": ([43, 85, 86, 171], [43, 1000, 86, 200], 6, 2, 64, 8, "bf16"),
    "group_7": ([20, 37, 1], [20, 500, 129], 7, 1, 128, 32, "bf16"),
    "group_40": ([5, 13], [5, 300], 40, 1, 64, 32, "f16"),
    "empty_sequences": ([0, 5, 0, 0, 9, 0], [0, 5, 100, 0, 200, 7], 4, 2, 128, 16, "f16"),
    "nothing_seen": ([10, 300, 4], [3, 0, 200], 4, 2, 128, 16, "bf16"),
    "decode_rows": ([1] * 9, [1, 15, 16, 17, 127, 128, 129, 1000, 640], 16, 4, 128, 16, "bf16"),
    "mixed": ([1, 700, 1, 1, 90, 1], [2000, 1500, 3, 128, 90, 777], 8, 2, 128, 16, "bf16"),
    "long_cache": ([33, 2], [9000, 5001], 16, 2, 128, 32, "bf16"),
    "long_cache_d64": ([3, 40], [7777, 6000], 8, 1, 64, 8, "f16"),
    "many_tiles": ([1400], [1400], 8, 1, 64, 16, "bf16"),
}


@pytest.mark.parametrize("name", CASES)
def test_matches_the_reference(name):
    news, totals, heads, kv_heads, dim, block, dtype = CASES[name]
    b = build(news, totals, heads, kv_heads, dim, block, dtype, seed=len(name), pad_rows=3, gap=2)
    ref, bound = reference(b)
    out = run(b.to("cuda"))
    torch.cuda.synchronize()
    worst = check(out, ref, bound, name)
    print(f"{name}: {worst:.3f} of the bound")


def f64(b, **kw):
    ref, bound = reference(b)
    out = run(b.to("cuda"), **kw)
    torch.cuda.synchronize()
    return out, ref, bound


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("where", ["k", "v", "kv"])
@pytest.mark.parametrize("dtype,heads,kv_heads,dim", [("bf16", 8, 2, 128), ("f16", 3, 1, 64)])
def test_values_a_token_does_not_see_do_not_reach_it(bad, where, dtype, heads, kv_heads, dim):
    """Non-finite K and V of the last three new tokens (and, in V, of single elements): every earlier
    token's output is the clean run's, bit for bit."""
    news, totals = [300, 5, 1], [700, 900, 257]
    b = build(news, totals, heads, kv_heads, dim, 16, dtype, seed=5)
    clean = run(b.to("cuda"))
    dirty = build(news, totals, heads, kv_heads, dim, 16, dtype, seed=5)
    for s, (n, total) in enumerate(zip(news, totals)):
        for back in range(min(3, n)):
            pos = total - 1 - back
            blk = int(dirty.tables[s, pos // 16])
            if "k" in where:
                dirty.kc[blk, pos % 16] = bad
            if "v" in where:
                dirty.vc[blk, pos % 16, :, back::2] = bad
    got = run(dirty.to("cuda"))
    torch.cuda.synchronize()
    for s, n in enumerate(news):
        r0 = int(b.starts[s])
        keep = n - min(3, n)
        assert torch.equal(got[r0:r0 + keep].view(torch.int16), clean[r0:r0 + keep].view(torch.int16)), s
    if where == "v":
        # the tokens that do see them get what the sums give: a column with one sign of infinity that
        # infinity, else NaN; columns without any stay finite
        r = int(b.starts[1]) - 1                        # the last token of the first sequence sees all three
        for c in range(dim):
            hit = [back for back in range(3) if c >= back and (c - back) % 2 == 0]
            x = got[r, :, c].float().cpu()
            if not hit:
                assert torch.isfinite(x).all()
            elif math.isnan(bad):
                assert torch.isnan(x).all()
            else:
                assert (x == bad).all()


def test_opposite_infinities_give_nan():
    b = build([40], [200], 4, 1, 64, 16, "bf16", seed=6)
    for back, v in ((0, math.inf), (1, -math.inf)):
        pos = 199 - back
        b.vc[int(b.tables[0, pos // 16]), pos % 16, 0, 7] = v
    got = run(b.to("cuda"))
    torch.cuda.synchronize()
    assert torch.isnan(got[39, :, 7]).all() and (got[38, :, 7] == -math.inf).all()
    assert torch.isfinite(got[:38]).all() and torch.isfinite(got[:, :, :7]).all()


def test_non_finite_values_of_split_tiles():
    """A cache long enough to be split: NaN in the last token's V reaches that token alone, through the merge."""
    b = build([9], [6000], 8, 1, 128, 32, "bf16", seed=7)
    b.vc[int(b.tables[0, 5999 // 32]), 5999 % 32, 0, 3] = math.nan
    got = run(b.to("cuda"))
    torch.cuda.synchronize()
    assert torch.isnan(got[8, :, 3]).all()
    got[8, :, 3] = 0
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("scale", [0.0, -0.09, 1.0, 3.0, 1e-20])
def test_scales(scale):
    """A zero scale is the mean of V; negative scales; sharp softmaxes (scores far past the rescale threshold)."""
    b = build([70, 1, 200], [70, 500, 900], 4, 2, 128, 16, "bf16", seed=8, scale=scale)
    out, ref, bound = f64(b)
    check(out, ref, bound, f"scale {scale}")


def test_growing_scores_rescale():
    """Keys that grow along the sequence move the reference maximum at nearly every step."""
    for dtype in ("f16", "bf16"):
        b = build([64], [1500], 4, 1, 64, 16, dtype, seed=9)
        L = 1500
        for pos in range(L):
            b.kc[int(b.tables[0, pos // 16]), pos % 16] = b.kc[int(b.tables[0, pos // 16]), pos % 16] * (0.5 + 4.0 * pos / L)
        out, ref, bound = f64(b)
        check(out, ref, bound, dtype)


def test_planned_layers_share_one_plan():
    """One plan per step, several layers (pools, queries) over it, and the plan is good for another run."""
    news, totals = [1, 200, 3, 0, 77], [3000, 900, 3, 40, 77]
    layers = [build(news, totals, 8, 2, 128, 16, "bf16", seed=20 + i).to("cuda") for i in range(3)]
    b0 = layers[0]
    T = b0.q.shape[0]
    ws = pkv.alloc_prefill_workspace(len(news), T, 8, 2, 128)
    ws.fill_(0xA5)                                      # contents on entry are ignored
    pkv.prefill_plan(ws, b0.lens, b0.starts, T, 8, 2, 128, b0.max_len)
    outs = []
    for _ in range(2):
        for b in layers:
            out = torch.full_like(b.q, math.nan)
            pkv.paged_attention_prefill(out, b.q, b.kc, b.vc, b.tables, b.lens, b.starts, b.scale,
                                        max_seq_len=b.max_len, workspace=ws, planned=True)
            outs.append(out)
    torch.cuda.synchronize()
    for i, b in enumerate(layers):
        ref, bound = reference(b.to("cpu"))
        check(outs[i], ref, bound, f"layer {i}")
        assert torch.equal(outs[i].view(torch.int16), outs[i + 3].view(torch.int16)), "a run over the same plan differs"
        single = run(b)
        assert torch.equal(outs[i].view(torch.int16), single.view(torch.int16))


def test_append_prefill_decode_verify_agree():
    """The operators in a row, as a serving step runs them: slot writes of a chunk, its attention, and the same
    tokens through the verify call; single new tokens through the decode call."""
    news, totals = [8, 8, 8], [8, 500, 1033]
    b = build(news, totals, 16, 4, 128, 16, "bf16", seed=30).to("cuda")
    slots, kn, vn = [], [], []
    for s, (n, t) in enumerate(zip(news, totals)):
        for pos in range(t - n, t):
            blk = int(b.tables[s, pos // 16])
            slots.append(blk * 16 + pos % 16)
            kn.append(b.kc[blk, pos % 16].clone())
            vn.append(b.vc[blk, pos % 16].clone())
            b.kc[blk, pos % 16] = math.nan
            b.vc[blk, pos % 16] = math.nan
    pkv.paged_kv_append(torch.stack(kn), torch.stack(vn), b.kc, b.vc, torch.tensor(slots, device="cuda"))
    out = run(b)
    q4 = b.q.view(3, 8, 16, 128).contiguous()
    ver = torch.full_like(q4, math.nan)
    tables = b.tables.contiguous()
    pkv.paged_attention_verify(ver, q4, b.kc, b.vc, tables, b.lens, b.scale, max_seq_len=b.max_len)
    last = torch.full((3, 16, 128), math.nan, dtype=b.q.dtype, device="cuda")
    pkv.paged_attention_decode(last, q4[:, 7].contiguous(), b.kc, b.vc, tables, b.lens, b.scale, max_seq_len=b.max_len)
    torch.cuda.synchronize()
    ref, bound = reference(b.to("cpu"))
    check(out, ref, bound, "prefill")
    # the other calls round the same way: twice the bound apart at most
    check(ver.view(24, 16, 128), out.double().cpu(), 2 * bound, "verify against prefill")
    check(last, out.view(3, 8, 16, 128)[:, 7].double().cpu(), 2 * bound.view(3, 8, 16, 128)[:, 7], "decode against prefill")


def test_captured_and_replayed_on_new_inputs():
    news, totals = [1, 130, 40], [2100, 700, 40]
    b = build(news, totals, 8, 2, 128, 16, "bf16", seed=40).to("cuda")
    T = b.q.shape[0]
    wsa, wsb = (pkv.alloc_prefill_workspace(3, T, 8, 2, 128) for _ in range(2))
    outa, outb = torch.full_like(b.q, math.nan), torch.full_like(b.q, math.nan)

    def step(out, ws):
        pkv.paged_attention_prefill(out, b.q, b.kc, b.vc, b.tables, b.lens, b.starts, b.scale, max_seq_len=2100, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(outa, wsa)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for out, ws in ((outa, wsa), (outb, wsb)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, capture_error_mode="relaxed"):
            step(out, ws)
        graphs.append(g)
    for rep in range(3):
        # other lengths in the captured buffers (the host bounds stay)
        new = build([1, 130, 40], [2100 - 500 * rep, 700 + rep, 40], 8, 2, 128, 16, "bf16", seed=41 + rep)
        b.q.copy_(new.q)
        b.tables.fill_(-1)
        b.tables[:, :new.tables.shape[1]].copy_(new.tables[:, :b.tables.shape[1]])
        b.kc[:new.kc.shape[0]].copy_(new.kc[:b.kc.shape[0]])
        b.vc[:new.vc.shape[0]].copy_(new.vc[:b.vc.shape[0]])
        b.lens.copy_(new.lens)
        b.starts.copy_(new.starts)
        assert new.kc.shape[0] <= b.kc.shape[0]
        outa.fill_(math.nan)
        outb.fill_(math.nan)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]           # both at once, each over its own workspace
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        ref, bound = reference(new)
        check(outa, ref, bound, f"replay {rep}")
        assert torch.equal(outa.view(torch.int16), outb.view(torch.int16))


def test_on_another_stream_and_without_a_workspace():
    b = build([50, 1], [300, 2000], 4, 2, 64, 8, "f16", seed=50).to("cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = torch.full_like(b.q, math.nan)
        pkv.paged_attention_prefill(out, b.q, b.kc, b.vc, b.tables, b.lens, b.starts)
    s.synchronize()
    ref, bound = reference(b.to("cpu"))
    check(out, ref, bound)


def test_more_sequences_than_a_plan_chunk():
    """More than 1024 sequences (the plan kernel reloads them in chunks), one to three tokens each."""
    import random
    r = random.Random(1)
    news = [r.randint(0, 3) for _ in range(1500)]
    totals = [n + r.randint(0, 40) for n in news]
    b = build(news, totals, 2, 1, 64, 16, "bf16", seed=60)
    out, ref, bound = f64(b)
    check(out, ref, bound)


def test_shared_blocks_and_one_sequence_twice():
    """Two sequences over the same blocks (a forked prompt), and the same queries give the same outputs."""
    b = build([20, 20], [300, 300], 8, 2, 128, 16, "bf16", seed=70)
    b.tables[1] = b.tables[0]
    b.q[20:40] = b.q[:20]
    out, ref, bound = f64(b)
    check(out, ref, bound)
    assert torch.equal(out[:20].view(torch.int16), out[20:40].view(torch.int16))


def test_bad_ids_lengths_and_starts_raise_the_error_word():
    def word(**change):
        b = build([20, 3], [300, 40], 4, 2, 128, 16, "bf16", seed=80)
        for k, f in change.items():
            f(getattr(b, k))
        out = run(b.to("cuda"))
        torch.cuda.synchronize()
        return pkv.device_error(reset=True), out

    def put(i, v):
        return lambda t: t.view(-1).__setitem__(i, v)

    assert word()[0] == 0
    assert word(tables=put(2, 1 << 30))[0] == 1         # a block id past the pool, and a negative one
    assert word(tables=put(3, -5))[0] == 1
    err, out = word(lens=put(0, 301))                   # longer than max_seq_len
    assert err == 1 and torch.isfinite(out).all()
    for i, v in ((0, -1), (1, 24), (2, 19), (2, 1 << 20)):      # starts before the first row, past the last, decreasing
        err, out = word(starts=put(i, v))
        assert err == 1, (i, v)


def test_a_plan_of_other_arguments_never_leaves_the_buffers():
    """The plan of a larger batch run with a smaller one: the entries that do not fit are skipped and reported."""
    big = build([400, 60], [3000, 60], 8, 2, 128, 16, "bf16", seed=90).to("cuda")
    small = build([40, 6], [300, 60], 8, 2, 128, 16, "bf16", seed=91).to("cuda")
    ws = pkv.alloc_prefill_workspace(2, 460, 8, 2, 128)
    pkv.prefill_plan(ws, big.lens, big.starts, 460, 8, 2, 128, big.max_len)
    out = torch.full((60, 8, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    pkv.paged_attention_prefill(out[:46], small.q, small.kc, small.vc, small.tables, small.lens, small.starts,
                                small.scale, max_seq_len=small.max_len, workspace=ws, planned=True)
    torch.cuda.synchronize()
    assert pkv.device_error(reset=True) == 1
    assert torch.isnan(out[46:]).all()


def test_repeats_bit_for_bit():
    b = build([33, 1, 250], [5000, 1200, 600], 8, 2, 128, 16, "bf16", seed=100).to("cuda")
    first = run(b)
    for _ in range(5):
        assert torch.equal(run(b).view(torch.int16), first.view(torch.int16))


E4M3_CASES = ["two_blocks", "tile_edges_g1", "tile_edges_g4", "group_7", "empty_sequences", "nothing_seen", "decode_rows",
              "mixed", "long_cache"]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("name", E4M3_CASES)
def test_e4m3_matches_the_reference(name, dtype):
    """The products run in f16 whatever the queries' type: the weights round there."""
    news, totals, heads, kv_heads, dim, block, _ = CASES[name]
    b = build(news, totals, heads, kv_heads, 128, block, dtype, seed=len(name), pad_rows=3, gap=2, e4m3=True)
    ref, bound = reference(b, torch.float16)
    out = run(b.to("cuda"))
    torch.cuda.synchronize()
    worst = check(out, ref, bound, name)
    print(f"{name}: {worst:.3f} of the bound")


def test_e4m3_codes_a_token_does_not_see():
    """NaN codes in the last new token's K and V: earlier tokens are the clean run's bit for bit; the token itself
    has NaN in the columns whose V holds one."""
    def batch():
        return build([300, 5, 1], [700, 900, 257], 8, 2, 128, 16, "bf16", seed=5, e4m3=True)
    clean = run(batch().to("cuda"))
    b = batch()
    for s, total in enumerate([700, 900, 257]):
        blk = int(b.tables[s, (total - 1) // 16])
        b.vc[blk, (total - 1) % 16, 1, 5] = 0x7f
        b.vc[blk, (total - 1) % 16, 1, 70] = 0xff
    got = run(b.to("cuda"))
    torch.cuda.synchronize()
    for s, n in enumerate([300, 5, 1]):
        r0 = int(b.starts[s])
        assert torch.equal(got[r0:r0 + n - 1].view(torch.int16), clean[r0:r0 + n - 1].view(torch.int16))
        last = got[r0 + n - 1]
        assert torch.isnan(last[4:, [5, 70]]).all()
        assert torch.isnan(last).sum() == 8
    b.kc[int(b.tables[1, 899 // 16]), 899 % 16] = 0x7f
    got = run(b.to("cuda"))
    torch.cuda.synchronize()
    assert torch.isnan(got[304]).all() and torch.equal(got[300:304].view(torch.int16), clean[300:304].view(torch.int16))


def test_e4m3_scales_and_planned():
    b = build([64, 1, 130], [64, 900, 400], 8, 4, 128, 16, "bf16", seed=9, scale=-0.2, e4m3=True)
    b.k_scale *= torch.tensor([1.0, 3.0, 0.2, 1.0])
    b.v_scale *= torch.tensor([1.0, 0.1, 20.0, 1.0])
    ref, bound = reference(b, torch.float16)
    c = b.to("cuda")
    ws = pkv.alloc_prefill_workspace(3, 195, 8, 4, 128)
    pkv.prefill_plan(ws, c.lens, c.starts, 195, 8, 4, 128, c.max_len)
    out = run(c, workspace=ws, planned=True)
    torch.cuda.synchronize()
    check(out, ref, bound)


def test_e4m3_zero_scales():
    """A KV head whose K scale is zero weighs every visible position alike; a zero V scale gives zeros."""
    b = build([40, 1, 260], [40, 700, 300], 8, 4, 128, 16, "f16", seed=11, e4m3=True)
    b.k_scale[1] = 0.0
    b.v_scale[2] = 0.0
    ref, bound = reference(b, torch.float16)
    out = run(b.to("cuda"))
    torch.cuda.synchronize()
    check(out, ref, bound)


def test_planned_batch_that_needs_no_plan():
    """A batch small enough to run without a plan gives the same through prefill_plan and planned."""
    b = build([1, 17, 5, 2], [1, 17, 33, 50], 4, 4, 64, 16, "f16", seed=12)
    ref, bound = reference(b)
    c = b.to("cuda")
    ws = pkv.alloc_prefill_workspace(4, 25, 4, 4, 64)
    ws.fill_(0xA5)
    pkv.prefill_plan(ws, c.lens, c.starts, 25, 4, 4, 64, c.max_len)
    out = run(c, workspace=ws, planned=True)
    torch.cuda.synchronize()
    check(out, ref, bound)
    assert torch.equal(out.view(torch.int16), run(c).view(torch.int16))


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace, give what they give one after the other."""
    bs = [build([300, 1, 40], [900, 3000, 40], 8, 2, 128, 16, "bf16", seed=13).to("cuda"),
          build([33, 1], [6000, 1200], 8, 2, 64, 8, "f16", seed=14).to("cuda")]
    want = [run(b) for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    spaces = [pkv.alloc_prefill_workspace(len(b.lens), b.q.shape[0], 8, 2, b.q.shape[2]) for b in bs]
    outs = [[torch.full_like(b.q, math.nan) for _ in range(8)] for b in bs]
    torch.cuda.synchronize()
    for i in range(8):
        for b, s, ws, out in zip(bs, streams, spaces, outs):
            with torch.cuda.stream(s):
                pkv.paged_attention_prefill(out[i], b.q, b.kc, b.vc, b.tables, b.lens, b.starts, b.scale,
                                            max_seq_len=b.max_len, workspace=ws)
    torch.cuda.synchronize()
    for w, out in zip(want, outs):
        for o in out:
            assert torch.equal(o.view(torch.int16), w.view(torch.int16))


@pytest.mark.parametrize("group", [4, 3])
def test_offsets_past_32_bits(group):
    """Blocks past the pool's first 2^31 elements, query rows past q's and out's first 2^31."""
    b = build([30, 1, 300], [100, 900, 300], 8 * group, 8, 128, 32, "bf16", seed=15)
    ref, bound = reference(b)
    NB = 2 ** 31 // (32 * 8 * 128) + b.kc.shape[0]
    T = 2 ** 31 // (8 * group * 128) + 1 + b.q.shape[0]
    c = b.to("cuda")
    far = []
    for pool in (c.kc, c.vc):
        x = torch.empty(NB, 32, 8, 128, dtype=torch.bfloat16, device="cuda")
        x[NB - pool.shape[0]:] = pool
        far.append(x)
    q = torch.empty(T, 8 * group, 128, dtype=torch.bfloat16, device="cuda")
    q[T - c.q.shape[0]:] = c.q
    out = torch.full_like(q, math.nan)
    ids = torch.where(c.tables < b.kc.shape[0], c.tables + (NB - b.kc.shape[0]), NB + 7).int()
    pkv.paged_attention_prefill(out, q, far[0], far[1], ids, c.lens, c.starts + (T - c.q.shape[0]), c.scale,
                                max_seq_len=c.max_len)
    torch.cuda.synchronize()
    check(out[T - c.q.shape[0]:], ref, bound)
    assert torch.isnan(out[T - c.q.shape[0] - 300:T - c.q.shape[0]]).all()
