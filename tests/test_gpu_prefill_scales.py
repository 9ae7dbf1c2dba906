"""paged_attention_prefill at scales far from the usual: zero and tiny scales over very large scores, E4M3 scales of
either sign, queries at the end of f16's range.  Every output is held to prefill_cases.reference's bound."""
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


def run(b):
    c = b.to("cuda")
    out = torch.full_like(c.q, math.nan)
    pkv.paged_attention_prefill(out, c.q, c.kc, c.vc, c.tables, c.lens, c.starts, c.scale, max_seq_len=c.max_len,
                                k_scale=c.k_scale, v_scale=c.v_scale)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("scale", [0.0, 1e-35, -1e-36])
@pytest.mark.parametrize("total", [500, 5000])
def test_large_scores_and_a_small_scale(scale, total):
    """Scores of 2^115: a zero scale weighs them all alike, a scale of 1e-35 leaves them at about 1."""
    b = build([30, 1], [total, 300], 4, 2, 64, 16, "bf16", seed=21, scale=scale)
    b.q *= 2.0 ** 52
    b.kc *= 2.0 ** 60
    ref, bound = reference(b)
    check(run(b), ref, bound)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [None, -0.1])
def test_e4m3_scales_of_either_sign(dtype, scale):
    """K = code * k_scale[g] for a negative k_scale[g] too, as in the decode call."""
    b = build([40, 1, 260, 9], [40, 700, 300, 6000], 8, 4, 128, 16, dtype, seed=22, scale=scale, e4m3=True)
    b.k_scale *= torch.tensor([1.0, -1.0, 1.0, -2.0])
    b.v_scale *= torch.tensor([1.0, 1.0, -1.0, -1.0])
    ref, bound = reference(b, torch.float16)
    check(run(b), ref, bound)


def test_e4m3_bf16_queries_up_to_the_end_of_f16():
    """A bf16 query is converted to f16: exact between 2^-14 and 65504 in magnitude (65280 is bf16's last there)."""
    b = build([40, 1], [200, 700], 8, 4, 128, 16, "bf16", seed=23, e4m3=True)
    b.q[:, :, ::2] = 2.0 ** -14
    b.q[:, :, 1::16] = 65280.0
    b.q[:, :, 9::16] = -65280.0
    b.k_scale *= 2.0 ** -18
    ref, bound = reference(b, torch.float16)
    check(run(b), ref, bound)
