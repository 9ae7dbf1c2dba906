"""paged_attention_prefill where the cache or the scores are not finite.

The expected kinds (finite, an infinity, NaN) come from the definition in IEEE arithmetic over the positions that a
token sees: out = sum_t w_t V_t / sum_t w_t, w_t = exp(z_t - max z).  The weights of these inputs stay far above the
smallest 16-bit number unless a test says otherwise.
"""
import math

import pytest
import torch

import paged_kv_cache_156_gb300 as pkv
from prefill_cases import build

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_error_word():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pkv.device_error(reset=True)
    yield
    assert pkv.device_error(reset=True) == 0


def run(b):
    c = b.to("cuda")
    out = torch.full_like(c.q, -7.0)
    pkv.paged_attention_prefill(out, c.q, c.kc, c.vc, c.tables, c.lens, c.starts, c.scale, max_seq_len=c.max_len,
                                k_scale=c.k_scale, v_scale=c.v_scale)
    torch.cuda.synchronize()
    return out.cpu()


def slot(b, s, pos):
    bs = b.kc.shape[1]
    return int(b.tables[s, pos // bs]), pos % bs


def definition(b):
    """[T, Hq, d] in float64: sums over the seen positions only, with IEEE's infinities and NaN."""
    T, Hq, d = b.q.shape
    G = Hq // b.kc.shape[2]
    out = torch.full((T, Hq, d), -7.0, dtype=torch.float64)
    for s in range(len(b.lens)):
        r0, r1, L = int(b.starts[s]), int(b.starts[s + 1]), int(b.lens[s])
        K, V = b.dense(s, b.kc, b.k_scale), b.dense(s, b.vc, b.v_scale)
        for r in range(r0, r1):
            lim = L - (r1 - r0) + (r - r0) + 1
            for h in range(Hq):
                if lim <= 0:
                    out[r, h] = 0.0
                    continue
                z = (K[:lim, h // G] * b.q[r, h].double()).sum(1) * b.scale
                w = torch.exp(z - z.max())
                out[r, h] = (w[:, None] * V[:lim, h // G]).sum(0) / w.sum()
    return out


def same_kind(got, want):
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], want[inf])


# Old positions every token sees (position 550 in the 128-position step that the last tokens see in part), new
# tokens' own; split over a long cache, or not.
@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("dtype,heads,kv_heads,dim", [("bf16", 8, 2, 128), ("f16", 3, 1, 64)])
def test_seen_by_all_and_seen_in_part(dtype, heads, kv_heads, dim, split):
    """What an element that every token sees gave the sum stays when elements that only the last tokens see are added:
    opposite infinities and NaN anywhere give NaN, wherever they lie."""
    total = 6000 if split else 600
    near = total - 50                                   # seen by every token, in the last tokens' step
    b = build([40], [total], heads, kv_heads, dim, 16, dtype, seed=3)
    clean = run(b)
    pairs = [(math.nan, math.inf), (-math.inf, math.inf), (math.inf, -math.inf), (math.inf, math.inf),
             (math.nan, -math.inf), (math.nan, math.nan), (None, math.inf), (None, -math.inf), (-math.inf, None)]
    for i, (old, new) in enumerate(pairs):
        for j, pos in enumerate((100, near)):
            col = 2 * i + j + 1
            if old is not None:
                blk, at = slot(b, 0, pos)
                b.vc[blk, at, 0, col] = old
            if new is not None:
                blk, at = slot(b, 0, total - 1 - i % 3)
                b.vc[blk, at, 0, col] = new
    got, want = run(b), definition(b)
    same_kind(got, want)
    keep = torch.isfinite(want)
    assert torch.equal(got[keep], clean[keep])          # (columns are independent of one another)
    assert torch.isnan(got[39, 0, 1]).all() and torch.isnan(got[39, 0, 3]) and got[39, 0, 7] == math.inf


@pytest.mark.parametrize("split", [False, True])
def test_nan_scores_beside_infinite_values(split):
    """A NaN key that every token sees makes every output NaN, columns with an infinite value among them."""
    total = 6000 if split else 600
    b = build([40], [total], 4, 1, 64, 16, "bf16", seed=4)
    blk, at = slot(b, 0, 77)
    b.kc[blk, at, 0, 5] = math.nan
    blk, at = slot(b, 0, total - 1)
    b.vc[blk, at, 0, 9] = math.inf
    assert torch.isnan(run(b)).all()


@pytest.mark.parametrize("kind", ["bf16", "f16_d64", "e4m3"])
@pytest.mark.parametrize("news", [1, 200])
def test_items_in_a_row_that_all_hold_some(news, kind):
    """Several work items a CTA, one after another, each with an infinite (E4M3: NaN) value that its last tokens see:
    every row has its own sequence's, in its own columns, and no other."""
    e4m3 = kind == "e4m3"
    dim, dtype = (64, "f16") if kind == "f16_d64" else (128, "bf16")
    B = 300 if news == 1 else 60
    totals = [news + (37 * s) % 290 for s in range(B)]
    b = build([news] * B, totals, 8, 8, dim, 16, dtype, seed=9, e4m3=e4m3)
    clean = run(b)
    want = clean.clone()
    bad = math.nan if e4m3 else math.inf
    for s in range(B):
        for back in {0, news // 3, news - 1}:
            blk, at = slot(b, s, totals[s] - 1 - back)
            col = (5 * s + 7 * back) % dim
            b.vc[blk, at, :, col] = 0x7f if e4m3 else bad
            want[news * (s + 1) - 1 - back:news * (s + 1), :, col] = bad
    for _ in range(3):
        got = run(b)
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        keep = ~torch.isnan(want)
        assert torch.equal(got[keep], want[keep])


def all_low(b, s, positions):
    """Keys whose every score is -inf: K = -inf in every column, for the positive queries of these tests."""
    for pos in positions:
        blk, at = slot(b, s, pos)
        b.kc[blk, at] = -math.inf


@pytest.mark.parametrize("dim", [64, 128])
def test_scores_that_are_all_minus_infinity(dim):
    """A token all of whose scores are -inf has no defined softmax: NaN, as the definition gives it.  Tokens with a
    finite score weigh the others 0; tokens that see nothing still get zeros."""
    b = build([6, 5, 300, 9], [6, 40, 700, 4], 4, 2, dim, 16, "bf16", seed=6)
    b.q.copy_(b.q.abs().clamp(min=0.25))
    all_low(b, 0, range(3))                             # its first three tokens see nothing else
    all_low(b, 1, range(40))                            # every token
    all_low(b, 2, range(0, 700, 3))
    got, want = run(b), definition(b)
    same_kind(got, want)
    assert torch.isnan(got[:3]).all() and torch.isnan(got[6:11]).all()
    assert torch.isfinite(got[3:6]).all() and torch.isfinite(got[11:311]).all() and (got[311:316] == 0).all()


@pytest.mark.parametrize("dim", [64, 128])
def test_scores_that_are_all_minus_infinity_over_a_long_cache(dim):
    """The same through the merge of a split tile's parts: every part without a finite score, and all but one."""
    for finite in (None, 17, 4000, 5995):
        b = build([3], [6000], 4, 1, dim, 16, "bf16", seed=7)
        b.q.copy_(b.q.abs().clamp(min=0.25))
        keep = b.kc.clone()
        all_low(b, 0, range(6000))
        if finite is not None:
            blk, at = slot(b, 0, finite)
            b.kc[blk, at] = keep[blk, at]
            v = b.vc[blk, at, 0].double()
        got = run(b)
        if finite is None:
            assert torch.isnan(got).all()
        else:
            # one weight of 1, the others 0: the value itself
            assert (got.double() == v).all()


@pytest.mark.parametrize("total", [600, 6000])
def test_an_infinite_value_of_a_vanishing_weight(total):
    """A weight that 16 bits or fp32 round to zero: the column is an infinity or NaN, never a number."""
    b = build([20], [total], 4, 1, 64, 16, "f16", seed=8)
    b.q.copy_(b.q.abs().clamp(min=0.25))
    for pos, key, col in ((50, -8.0, 3), (51, -200.0, 4), (total - 3, -8.0, 5), (total - 1, -200.0, 6)):
        blk, at = slot(b, 0, pos)
        b.kc[blk, at] = key
        b.vc[blk, at, 0, col] = math.inf
    got = run(b)
    assert not torch.isfinite(got[:, :, 3:5]).any()
    assert not torch.isfinite(got[18:, :, 5]).any() and not torch.isfinite(got[19, :, 6]).any()
    assert torch.isfinite(got[:17, :, 5]).all() and torch.isfinite(got[:19, :, 6]).all()
    assert torch.isfinite(got[:, :, 7:]).all() and torch.isfinite(got[:, :, :3]).all()
