"""speculative_accept against a plain reference in Python's whole numbers.

Tokens and counts must be equal: the acceptance test is exact, and the draw sums
whole units of 2^-44, which no order of summation changes.
"""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_156_gb300 as pkv

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _clean_error_word():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pkv.device_error(reset=True)
    yield
    assert pkv.device_error(reset=True) == 0


def ref(x, p, q, u, counts):
    B, K = x.shape
    V = p.shape[2]
    tokens = np.full((B, K + 1), -1, dtype=np.int64)
    accepted = np.zeros(B, dtype=np.int32)
    for b in range(B):
        n = K if counts is None else min(max(int(counts[b]), 0), K)
        a = 0
        while a < n and 0 <= x[b, a] < V and \
                float(u[b, a]) * (1.0 if q is None else float(q[b, a, x[b, a]])) < float(p[b, a, x[b, a]]):
            tokens[b, a] = x[b, a]
            a += 1
        row = p[b, a].astype(np.float32)
        left = row.copy()
        if a < n:
            if q is not None:
                left = row - q[b, a].astype(np.float32)
            elif 0 <= x[b, a] < V:
                left[x[b, a]] = 0
        for w in (left, row):
            w = np.clip(np.nan_to_num(w, nan=0.0, posinf=1.0, neginf=0.0), 0.0, 1.0).astype(np.float64)
            units = [int(v) for v in np.floor(w * 2.0 ** 44)]
            total = sum(units)
            if total:
                z = max(0.0, float(u[b, K])) * float(total) if u[b, K] == u[b, K] else 0.0
                mark = min(int(min(z, 2.0 ** 63)), total - 1)
                run = 0
                for j, v in enumerate(units):
                    run += v
                    if run > mark:
                        tokens[b, a] = j
                        break
                break
        accepted[b] = a
    return tokens, accepted


def run(x, p, q, u, counts=None):
    B, K = x.shape
    tokens = torch.full((B, K + 1), -7, dtype=torch.int64, device="cuda")
    accepted = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    pkv.speculative_accept(tokens, accepted, x.cuda(), p.cuda(), u.cuda(), draft_probs=None if q is None else q.cuda(),
                           num_drafts=None if counts is None else counts.cuda())
    torch.cuda.synchronize()
    return tokens.cpu().numpy(), accepted.cpu().numpy()


def compare(x, p, q, u, counts=None):
    got = run(x, p, q, u, counts)
    f = lambda t: None if t is None else t.float().numpy()
    want = ref(x.numpy(), f(p), f(q), u.numpy(), None if counts is None else counts.numpy())
    assert np.array_equal(got[1], want[1])
    assert np.array_equal(got[0], want[0])
    return got


def inputs(B, K, V, dtype="f32", seed=0, noise=0.5):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(B, K + 1, V, generator=g) * 2
    p = torch.softmax(logits, -1)
    q = torch.softmax(logits[:, :K] + noise * torch.randn(B, K, V, generator=g), -1)
    x = torch.multinomial(q.reshape(-1, V), 1, generator=g).view(B, K) if K else torch.zeros(B, 0, dtype=torch.int64)
    u = torch.rand(B, K + 1, generator=g)
    return x, p.to(DT[dtype]), q.to(DT[dtype]), u


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 3, 127, 128, 129, 1000, 16384, 16385, 50257])
def test_vocabularies(dtype, V):
    for K in (1, 4):
        compare(*inputs(3, K, V, dtype, seed=V + K))


@pytest.mark.parametrize("V", [131072, 131073, 300001])
def test_rows_of_several_rounds(V):
    x, p, q, u = inputs(2, 1, V, seed=V)
    for last in (0.0, 0.3, 0.7, 0.9999999):
        u[:, -1] = last
        compare(x, p, q, u)


@pytest.mark.parametrize("K", [0, 1, 31, 32, 33, 70])
def test_draft_counts(K):
    x, p, q, u = inputs(4, K, 200, seed=K, noise=0.02)
    compare(x, p, q if K else None, u)
    counts = torch.tensor([0, K, K // 2, max(K - 1, 0)], dtype=torch.int32)
    compare(x, p, q if K else None, u, counts)


def test_every_draft_accepted_and_none():
    x, p, q, u = inputs(5, 6, 333, seed=1)
    u[:, :6] = 0.0
    got = compare(x, p, q, u)
    assert (got[1] == 6).all()
    p2 = p.clone()
    for b in range(5):
        p2[b, 0, x[b, 0]] = 0
    got = compare(x, p2, q, u)
    assert (got[1] == 0).all()


def test_the_comparison_is_exact():
    """u q against p where they differ by the last bit, or not at all (equal is refused)."""
    V = 16
    p = torch.zeros(4, 2, V)
    q = torch.zeros(4, 1, V)
    x = torch.zeros(4, 1, dtype=torch.int64)
    u = torch.tensor([[0.5, 0.0], [0.5, 0.0], [1.0 / 3, 0.0], [0.0, 0.0]])
    q[:, 0, 0] = torch.tensor([0.5, 0.5, 0.7, 0.5])
    prod = float(u[2, 0]) * float(q[2, 0, 0])
    p[:, 0, 0] = torch.tensor([0.25, float(np.nextafter(np.float32(0.25), np.float32(1))), prod, 0.0])
    p[:, :, 3] = 0.5
    got = compare(x, p, q, u)
    assert got[1].tolist()[:2] == [0, 1] and got[1][3] == 0


def test_drafts_without_probabilities():
    for dtype in ("f32", "bf16"):
        x, p, _, u = inputs(6, 5, 1001, dtype, seed=3)
        x = p[:, :5].float().argmax(-1)
        u[0, :5] = 0.999
        got = compare(x, p, None, u)
        for b in range(6):                              # a refused draft is never drawn again at its place
            a = got[1][b]
            if a < 5:
                assert got[0][b, a] != x[b, a]


def test_rows_that_leave_nothing():
    """p = q where the draft is refused all the same (a zero product): the target's own row is drawn from; a row
    of zeros, or of NaN, gives -1."""
    V = 300
    p = torch.full((4, 2, V), 1.0 / V)
    q = p[:, :1].clone()
    x = torch.full((4, 1), 5, dtype=torch.int64)
    u = torch.full((4, 2), 0.5)
    p[0, 0, 5] = q[0, 0, 5] = 0.0                       # 0 < 0 is false: refused; p - q = 0 everywhere
    p[1, 0] = 0.0                                       # nothing at all
    p[2, 0] = math.nan
    p[3, 0] = 0.0
    p[3, 0, 7] = -0.25
    got = compare(x, p, q, u)
    assert got[0][0, 0] == 150 and (got[0][1:, 0] == -1).all() and (got[1] == 0).all()


def test_odd_probabilities_and_numbers():
    x, p, q, u = inputs(8, 2, 700, seed=9)
    p[0, 0, ::3] = math.nan
    p[1, 0, 11] = math.inf
    q[2, 0, 13] = math.inf
    p[3, 1, 5] = -1.0
    p[4] = 1e-42                                        # below a unit: the row counts as nothing
    u[5, 2] = -3.0
    u[6, 2] = 5.0
    u[7, 2] = math.nan
    compare(x, p, q, u)


def test_strided_rows_off_a_16_byte_boundary():
    """A base that is aligned to its elements only."""
    x, p, q, u = inputs(3, 2, 257, "bf16", seed=12)
    flat = torch.empty(p.numel() + 1, dtype=torch.bfloat16, device="cuda")
    pv = flat[1:].view(p.shape)
    pv.copy_(p)
    tokens = torch.empty(3, 3, dtype=torch.int64, device="cuda")
    accepted = torch.empty(3, dtype=torch.int32, device="cuda")
    pkv.speculative_accept(tokens, accepted, x.cuda(), pv, u.cuda(), draft_probs=q.cuda())
    torch.cuda.synchronize()
    want = ref(x.numpy(), p.float().numpy(), q.float().numpy(), u.numpy(), None)
    assert np.array_equal(tokens.cpu().numpy(), want[0]) and np.array_equal(accepted.cpu().numpy(), want[1])


def test_bad_tokens_and_counts_raise_the_error_word():
    x, p, q, u = inputs(3, 3, 90, seed=14)
    u[:, :3] = 0.0
    x[1, 1] = 90
    x[2, 0] = -1
    got = run(x, p, q, u)
    assert pkv.device_error(reset=True) == 1
    want = ref(x.numpy(), p.numpy(), q.numpy(), u.numpy(), None)
    assert np.array_equal(got[0], want[0]) and got[1].tolist() == [3, 1, 0]
    x, p, q, u = inputs(3, 3, 90, seed=14)
    counts = torch.tensor([-1, 4, 2], dtype=torch.int32)
    got = run(x, p, q, u, counts)
    assert pkv.device_error(reset=True) == 1
    want = ref(x.numpy(), p.numpy(), q.numpy(), u.numpy(), counts.numpy())
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_captured_replayed_and_repeated():
    x, p, q, u = (t.cuda() for t in inputs(16, 4, 5000, seed=20))
    tokens = torch.empty(16, 5, dtype=torch.int64, device="cuda")
    accepted = torch.empty(16, dtype=torch.int32, device="cuda")

    def step():
        pkv.speculative_accept(tokens, accepted, x, p, u, draft_probs=q)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        step()
    for seed in (21, 22):
        new = inputs(16, 4, 5000, seed=seed)
        for dst, src in zip((x, p, q, u), new):
            dst.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        want = ref(*(t.numpy() for t in new), None)
        assert np.array_equal(tokens.cpu().numpy(), want[0]) and np.array_equal(accepted.cpu().numpy(), want[1])


def test_the_tokens_follow_the_target():
    """First tokens of 20000 calls' worth of sequences against the target's probabilities: each of 5 tokens within
    5 standard deviations of its binomial count (a correct sampler misses one of them in under 1 of 300000 runs)."""
    B, V = 20000, 5
    g = torch.Generator().manual_seed(30)
    p1 = torch.tensor([0.4, 0.3, 0.2, 0.05, 0.05])
    q1 = torch.tensor([0.1, 0.2, 0.3, 0.2, 0.2])
    p, q = p1.repeat(B, 2, 1), q1.repeat(B, 1, 1)
    x = torch.multinomial(q1.repeat(B, 1), 1, generator=g)
    u = torch.rand(B, 2, generator=g)
    first = run(x, p, q, u)[0][:, 0]
    for j in range(V):
        n = int((first == j).sum())
        mean, sd = B * float(p1[j]), math.sqrt(B * float(p1[j]) * (1 - float(p1[j])))
        assert abs(n - mean) < 5 * sd, (j, n, mean)


def test_offsets_past_32_bits():
    """Probabilities past the first 2^31: the last sequence keeps all its drafts but the last, or all of them."""
    B, K, V = 64, 64, pkv.ACCEPT_MAX_VOCAB
    target = torch.zeros(B, K + 1, V, dtype=torch.float16, device="cuda")
    assert target.numel() > 2 ** 31
    drafts = torch.full((B, K), 5, dtype=torch.int64)
    drafts[-1] = V - 1 - torch.arange(K)
    target[-1, torch.arange(K), drafts[-1].cuda()] = 1.0
    target[-1, K, V - 3] = 1.0
    uniform = torch.full((B, K + 1), 0.5, device="cuda")
    for kept in (K, K - 1):
        if kept < K:
            target[-1, K - 1, V - K] = 0.0
            target[-1, K - 1, V - 1] = 0.25
        tokens = torch.full((B, K + 1), 7, dtype=torch.int64, device="cuda")
        accepted = torch.full((B,), 7, dtype=torch.int32, device="cuda")
        pkv.speculative_accept(tokens, accepted, drafts.cuda(), target, uniform)
        assert int(accepted[-1]) == kept and tokens[-1, :kept].cpu().equal(drafts[-1, :kept])
        assert int(tokens[-1, kept]) == (V - 3 if kept == K else V - 1)
        assert (accepted[:-1] == 0).all() and (tokens[:-1] == -1).all()


@pytest.mark.parametrize("dtype,V", [("f32", pkv.ACCEPT_MAX_VOCAB), ("bf16", pkv.ACCEPT_MAX_VOCAB), ("f32", 40001), ("f16", 40002)])
@pytest.mark.parametrize("poff,qoff", [(0, 1), (1, 0), (2, 3), (3, 3)])
def test_the_two_rows_stand_differently(dtype, V, poff, qoff):
    """Target and draft rows at every distance from a boundary of four elements, up to the largest vocabulary."""
    x, p, q, u = inputs(1, 1, V, dtype, seed=30 + poff, noise=1.0)
    rows = []
    for t, off in ((p, poff), (q, qoff)):
        flat = torch.full((t.numel() + 8,), math.nan, dtype=t.dtype, device="cuda")
        rows.append(flat[off:off + t.numel()].view(t.shape))
        rows[-1].copy_(t)
    u[:, 0] = 1.0                                       # (refused wherever p <= q)
    for last in (0.0, 0.5, 0.9999999):
        u[:, -1] = last
        tokens = torch.empty(1, 2, dtype=torch.int64, device="cuda")
        accepted = torch.empty(1, dtype=torch.int32, device="cuda")
        pkv.speculative_accept(tokens, accepted, x.cuda(), rows[0], u.cuda(), draft_probs=rows[1])
        want = ref(x.numpy(), p.float().numpy(), q.float().numpy(), u.numpy(), None)
        assert np.array_equal(tokens.cpu().numpy(), want[0]) and np.array_equal(accepted.cpu().numpy(), want[1])
