"""paged_attention_tree over sequences that share their prefix's blocks, as the block manager's forks do: the blocks are read
once a sequence, whatever hint their loads carry."""
import math

import pytest
import torch

import paged_kv_cache_156_gb300 as pkv
from prefill_cases import build, check
from tree_cases import masks, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_error_word():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pkv.device_error(reset=True)
    yield
    assert pkv.device_error(reset=True) == 0


@pytest.mark.parametrize("dim,heads,kv_heads,e4m3", [(128, 8, 2, False), (128, 16, 2, False), (64, 4, 2, False), (128, 8, 2, True),
                                                     (128, 16, 2, True)])
def test_shared_prefixes(dim, heads, kv_heads, e4m3):
    """Sequences 0 to 4 share 640 positions, 5 and 6 a block's; trees of one item and of two beside one another."""
    news, totals, block = [16, 7, 64, 1, 33, 20, 5], [700, 647, 900, 641, 710, 100, 30], 16
    b = build(news, totals, heads, kv_heads, dim, block, "bf16", seed=dim + heads, e4m3=e4m3)
    for s in range(1, 5):
        b.tables[s, :40] = b.tables[0, :40]
    b.tables[6, 0] = b.tables[5, 0]
    mask, _ = masks(news, 9)
    ref, bound = reference(b, mask, torch.float16 if e4m3 else None)
    c = b.to("cuda")
    for _ in range(2):
        out = torch.full_like(c.q, math.nan)
        pkv.paged_attention_tree(out, c.q, c.kc, c.vc, c.tables, c.lens, c.starts, mask.cuda(), c.scale, max_seq_len=c.max_len,
                                 k_scale=c.k_scale, v_scale=c.v_scale)
        torch.cuda.synchronize()
        check(out, ref, bound)
