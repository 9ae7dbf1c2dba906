"""speculative_accept_tree over rows that start off a boundary of four elements and are long enough that several batches of a
warp are on their way at once, one row after another with every offset: whole numbers, so the results must be equal."""
import numpy as np
import pytest
import torch

import paged_kv_cache_156_gb300 as pkv
from test_gpu_accept_tree import DT, draw, ref

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_error_word():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pkv.device_error(reset=True)
    yield
    assert pkv.device_error(reset=True) == 0


def walk(V, dtype, shift, n, B, seed, W=None):
    """B chains of n nodes whose drafts are what their parents' rows draw, the last of them drafting something else; the rows
    start ``shift`` elements into an allocation."""
    g = torch.Generator().manual_seed(seed)
    T, W = B * n, W or n
    flat = torch.empty(T * V + 3, dtype=DT[dtype])
    p = flat[shift:shift + T * V].view(T, V)
    p.copy_(torch.softmax(torch.randn(T, V, generator=g), -1))
    u = torch.rand(T, generator=g)
    u[::5] = 0.0                                              # the row's first token, and its last
    u[3::5] = 1.0 - 2.0 ** -24
    rows = p.float().numpy()
    drafts = torch.zeros(T, dtype=torch.int64)
    for r in range(T - 1):
        if (r + 1) % n:
            drafts[r + 1] = draw(rows[r], float(u[r]))
    for b in range(B):
        drafts[b * n + n - 1] = (int(drafts[b * n + n - 1]) + 1) % V
    parents, starts = [-1] + list(range(n - 1)), [n * b for b in range(B + 1)]
    on = flat.cuda()[shift:shift + T * V].view(T, V)
    assert on.data_ptr() // on.element_size() % 4 == shift
    out = [torch.full((B, W), 77, dtype=torch.int64).cuda(), torch.full((B, W), 77, dtype=torch.int32).cuda(),
           torch.full((B,), 77, dtype=torch.int32).cuda()]
    args = (drafts.cuda(), torch.tensor(parents * B, dtype=torch.int32).cuda(), torch.tensor(starts, dtype=torch.int32).cuda(),
            on, u.cuda())
    want = ref(starts, drafts.tolist(), parents * B, rows, u.numpy(), W)
    assert want[2].tolist() == [min(n - 2, W - 1)] * B
    for _ in range(3):
        pkv.speculative_accept_tree(*out, *args)
        torch.cuda.synchronize()
        for a, b, name in zip(out, want, ("tokens", "path", "count")):
            assert np.array_equal(a.cpu().numpy(), b), (V, dtype, shift, name, a, b)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("V", [98301, 98302, 98303, 98304, 98305, 128001, 128002, 128003, 131072, 131073, 163841, 200003])
def test_long_rows_of_every_offset(V, dtype):
    """Three to seven batches a warp: a V that is no multiple of four puts the walk's rows at every offset in turn."""
    walk(V, dtype, V % 4, 7, 2, V)


@pytest.mark.parametrize("shift", range(4))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_rows_off_their_boundary(dtype, shift):
    """Every row at the same offset, and the largest vocabulary that is no multiple of four."""
    walk(128000, dtype, shift, 6, 3, 10 + shift)
    walk(pkv.ACCEPT_MAX_VOCAB - 1, dtype, shift, 5, 1, 20 + shift)


@pytest.mark.parametrize("dtype", list(DT))
def test_rows_of_one_cta_off_their_boundary(dtype):
    for V in (8189, 8190, 8191, 8192):
        for shift in range(4):
            walk(V, dtype, shift, 6, 2, V + shift)
