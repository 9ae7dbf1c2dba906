"""paged_kv_gather: rows read back from 16-bit pools bit for bit, from E4M3 pools as round(code * scale),
rows that no position maps to untouched, and the calls around it (slot writes before, chunk attention after)."""
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


def batch(totals, kv_heads=2, dim=64, block=16, dtype="bf16", seed=0, e4m3=False):
    return build([0] * len(totals), totals, kv_heads, kv_heads, dim, block, dtype, seed=seed, e4m3=e4m3)


def gather(b, starts, rows, dtype):
    k = torch.full((rows, b.kc.shape[2], b.kc.shape[3]), math.nan, dtype=dtype, device="cuda")
    v = torch.full_like(k, math.nan)
    c = b.to("cuda")
    pkv.paged_kv_gather(k, v, c.kc, c.vc, c.tables, c.lens, torch.tensor(starts, dtype=torch.int32, device="cuda"),
                        k_scale=c.k_scale, v_scale=c.v_scale)
    torch.cuda.synchronize()
    return k.cpu(), v.cpu()


def expected(b, starts, rows, dtype):
    out = []
    for pool, scale in ((b.kc, b.k_scale), (b.vc, b.v_scale)):
        x = torch.full((rows, pool.shape[2], pool.shape[3]), math.nan, dtype=dtype)
        for s in range(len(b.lens)):
            L = int(b.lens[s])
            ids = b.tables[s, :-(-L // pool.shape[1])].long()
            r = pool[ids].flatten(0, 1)[:L]
            if scale is not None:
                r = (r.view(torch.float8_e4m3fn).float() * scale[:, None]).to(dtype)
            x[starts[s]:starts[s] + L] = r
        out.append(x)
    return out


def same(got, want):
    for g, w in zip(got, want):
        both = torch.isnan(g) & torch.isnan(w)
        assert torch.equal(torch.where(both, torch.zeros_like(g), g), torch.where(both, torch.zeros_like(w), w))


@pytest.mark.parametrize("block", [1, 8, 16, 24, 32])
@pytest.mark.parametrize("kv_heads,dim", [(1, 8), (2, 64), (8, 128), (3, 40)])
@pytest.mark.parametrize("dtype,e4m3", [("f16", False), ("bf16", False), ("f16", True), ("bf16", True)])
def test_rows_read_back(block, kv_heads, dim, dtype, e4m3):
    totals = [1, 0, 17, 33, 0, 0, 100, 7]
    b = batch(totals, kv_heads, dim, block, dtype, seed=block, e4m3=e4m3)
    starts = [3]                                        # rows before the first, between (gaps) and after the last
    for i, t in enumerate(totals):
        starts.append(starts[-1] + t + (5 if i % 3 == 0 else 0))
    rows = starts[-1] + 9
    dt = torch.float16 if dtype == "f16" else torch.bfloat16
    same(gather(b, starts, rows, dt), expected(b, starts, rows, dt))


def test_many_sequences_and_empty_ones():
    import random
    r = random.Random(3)
    totals = [r.choice((0, 0, 1, 2, 30)) for _ in range(1300)]
    b = batch(totals, 1, 64, 16, "bf16", seed=4)
    starts = [0]
    for t in totals:
        starts.append(starts[-1] + t)
    same(gather(b, starts, starts[-1], torch.bfloat16), expected(b, starts, starts[-1], torch.bfloat16))


def test_nan_codes_read_back_as_nan():
    b = batch([20], 2, 64, 16, "bf16", seed=5, e4m3=True)
    b.kc[int(b.tables[0, 0]), 3, 1, 7] = 0xff
    k, v = gather(b, [0, 20], 20, torch.bfloat16)
    assert torch.isnan(k[3, 1, 7]) and torch.isnan(k).sum() == 1 and torch.isfinite(v).all()


def test_bad_entries_raise_the_error_word():
    b = batch([40, 20], 2, 64, 16, "bf16", seed=6)
    good = expected(b, [0, 40, 60], 60, torch.bfloat16)
    b.tables[0, 1] = -1                                 # a block that is not there: its rows stay, the others come
    k, v = gather(b, [0, 40, 60], 60, torch.bfloat16)
    assert pkv.device_error(reset=True) == 1
    assert torch.isnan(k[16:32]).all() and torch.equal(k[:16], good[0][:16]) and torch.equal(k[32:], good[0][32:])
    b = batch([40, 20], 2, 64, 16, "bf16", seed=6)
    for starts in ([0, 30, 60], [0, 40, 39], [-1, 40, 60], [0, 40, 61]):      # too little room, decreasing, out of range
        gather(b, starts, 60, torch.bfloat16)
        assert pkv.device_error(reset=True) == 1, starts


def test_quantized_append_gather_and_prefill_in_a_row():
    """A prompt quantized into an E4M3 pool as it is written, read back block-aligned as a 16-bit pool, and both
    attended: over the codes, and over the rows read back."""
    news, totals = [70, 1, 33], [70, 200, 33]
    b = build(news, totals, 8, 2, 128, 16, "f16", seed=7, e4m3=True)
    c = b.to("cuda")
    x = torch.randn(sum(totals), 2, 128, device="cuda").half()
    y = torch.randn(sum(totals), 2, 128, device="cuda").half()
    slots = torch.cat([(c.tables[s, :-(-t // 16)].long()[:, None] * 16 + torch.arange(16, device="cuda")).flatten()[:t]
                       for s, t in enumerate(totals)])
    pkv.paged_kv_append_fp8(x, y, c.kc, c.vc, slots, c.k_scale, c.v_scale)
    starts, at = [0], 0
    for t in totals:
        starts.append(starts[-1] + -(-t // 16) * 16)    # block-aligned: the rows are a pool of their own
    k16 = torch.zeros(starts[-1], 2, 128, dtype=torch.float16, device="cuda")
    v16 = torch.zeros_like(k16)
    pkv.paged_kv_gather(k16, v16, c.kc, c.vc, c.tables, c.lens, torch.tensor(starts, dtype=torch.int32, device="cuda"),
                        k_scale=c.k_scale, v_scale=c.v_scale)
    tables = torch.zeros(3, 13, dtype=torch.int32, device="cuda")
    for s, t in enumerate(totals):
        n = -(-t // 16)
        tables[s, :n] = torch.arange(starts[s] // 16, starts[s] // 16 + n)
    out8, out16 = torch.full_like(c.q, math.nan), torch.full_like(c.q, math.nan)
    pkv.paged_attention_prefill(out8, c.q, c.kc, c.vc, c.tables, c.lens, c.starts, c.scale, max_seq_len=200,
                                k_scale=c.k_scale, v_scale=c.v_scale)
    pkv.paged_attention_prefill(out16, c.q, k16.view(-1, 16, 2, 128), v16.view(-1, 16, 2, 128), tables, c.lens, c.starts,
                                c.scale, max_seq_len=200)
    torch.cuda.synchronize()
    ref, bound = reference(c.to("cpu"))
    check(out8, ref, bound, "over the codes")
    # over the rows: K and V rounded once more to f16, 2^-11 relative: V moves the output by that times sum p |V|
    # (within the bound's own h A), K a score by 2^-11 scale sum_i |q_i K_i| (at most 0.09 * 60 here), and so a
    # weight by twice that, relative
    slack = 2.0 ** -11 + 2 * 2.0 ** -11 * 0.09 * 60
    amax = float(c.v_scale.max() * 448)
    check(out16, ref, bound + slack * amax, "over the rows read back")


@pytest.mark.parametrize("e4m3", [False, True])
def test_offsets_past_32_bits(e4m3):
    """Blocks past the pool's first 2^31 elements, rows past the outputs' first 2^31."""
    b = batch([70, 0, 200], kv_heads=8, dim=128, block=32, dtype="f16", seed=21, e4m3=e4m3)
    NB = 2 ** 31 // (32 * 8 * 128) + b.kc.shape[0]
    rows = 2 ** 31 // (8 * 128) + 1 + 300
    first = rows - 290
    starts = [0, 75, 75, 280]
    want = expected(b, starts, 290, torch.float16)
    c = b.to("cuda")
    far = []
    for pool in (c.kc, c.vc):
        x = torch.empty(NB, 32, 8, 128, dtype=pool.dtype, device="cuda")
        x[NB - pool.shape[0]:] = pool
        far.append(x)
    k = torch.full((rows, 8, 128), math.nan, dtype=torch.float16, device="cuda")
    v = torch.full_like(k, math.nan)
    ids = torch.where(c.tables < b.kc.shape[0], c.tables + (NB - b.kc.shape[0]), NB + 7).int()
    pkv.paged_kv_gather(k, v, far[0], far[1], ids, c.lens, torch.tensor(starts, dtype=torch.int32, device="cuda") + first,
                        k_scale=c.k_scale, v_scale=c.v_scale)
    torch.cuda.synchronize()
    same((k[first:].cpu(), v[first:].cpu()), want)
    assert torch.isnan(k[first - 300:first]).all()
