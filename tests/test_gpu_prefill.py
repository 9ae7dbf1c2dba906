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
    pkv.paged_attention_prefill(out, b.q, b.kc, b.vc, b.tables, b.lens, b.starts, b.scale, max_seq_len=b.max_len, **kw)
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
