"""paged_attention_prefill over the plans that no small batch makes: a tile cut into as many parts as there may be,
batches that the plan kernel lists in several passes beside a long sequence."""
import math
import random

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


def both_ways(b, work_dtype=None):
    """The single call and a planned one, within the reference's bound and bit for bit the same."""
    ref, bound = reference(b, work_dtype)
    c = b.to("cuda")
    T, heads, dim = c.q.shape
    kv_heads = c.kc.shape[2]
    ws = pkv.alloc_prefill_workspace(len(c.lens), T, heads, kv_heads, dim)
    ws.fill_(0xA5)
    outs = []
    for planned in (False, True):
        if planned:
            pkv.prefill_plan(ws, c.lens, c.starts, T, heads, kv_heads, dim, c.max_len)
        out = torch.full_like(c.q, math.nan)
        pkv.paged_attention_prefill(out, c.q, c.kc, c.vc, c.tables, c.lens, c.starts, c.scale, max_seq_len=c.max_len,
                                    workspace=ws, planned=planned, k_scale=c.k_scale, v_scale=c.v_scale)
        outs.append(out)
    torch.cuda.synchronize()
    check(outs[0], ref, bound, "single")
    assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))


# 38912 positions are 304 steps: 152 parts of two steps each on 152 SMs
@pytest.mark.parametrize("news,total", [(1, 38912), (1, 38911), (1, 50001), (33, 40007)])
@pytest.mark.parametrize("kind", ["bf16", "f16_d64", "e4m3"])
def test_one_tile_in_many_parts(news, total, kind):
    e4m3 = kind == "e4m3"
    dim, dtype = (64, "f16") if kind == "f16_d64" else (128, "bf16")
    b = build([news], [total], 8, 1, dim, 32, dtype, seed=31, e4m3=e4m3)
    both_ways(b, torch.float16 if e4m3 else None)


def test_many_sequences_beside_a_long_one():
    """More than 1024 sequences, one of them long enough to be split in a smaller batch."""
    r = random.Random(2)
    news = [r.randint(0, 3) for _ in range(1300)]
    totals = [n + r.randint(0, 40) for n in news]
    news[700], totals[700] = 5, 2500
    both_ways(build(news, totals, 2, 1, 64, 16, "bf16", seed=32))


def test_many_tiles_beside_a_long_sequence():
    """1024 sequences of 2072 tiles in all (264 rows are two tiles, 520 three), one of them long."""
    news = [65 if s % 43 == 0 else 33 for s in range(1024)]
    totals = [n + s % 5 for s, n in enumerate(news)]
    totals[500] = 2500
    both_ways(build(news, totals, 8, 1, 64, 8, "f16", seed=33))
