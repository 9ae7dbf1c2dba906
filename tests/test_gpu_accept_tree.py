"""speculative_accept_tree against a plain reference in Python's whole numbers: tokens, paths and counts must be equal
(the draw sums whole units of 2^-44, which no order of summation changes)."""
import math
import random

import numpy as np
import pytest
import torch

import paged_kv_cache_156_gb300 as pkv
from tree_cases import tree

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _clean_error_word():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pkv.device_error(reset=True)
    yield
    assert pkv.device_error(reset=True) == 0


def draw(p, u):
    """The first token whose inclusive sum of units exceeds floor(u total), -1 without weight."""
    p = np.clip(np.nan_to_num(p.astype(np.float32), nan=0.0, posinf=1.0, neginf=0.0), 0.0, 1.0).astype(np.float64)
    units = np.floor(p * 2.0 ** 44).astype(np.uint64)
    upto = np.cumsum(units, dtype=np.uint64)                  # (below 2^63)
    total = int(upto[-1])
    if total == 0:
        return -1
    z = float(u) * float(total) if u == u and u > 0 else 0.0
    return int(np.searchsorted(upto, np.uint64(min(int(min(z, 2.0 ** 63)), total - 1)), side="right"))


def ref(starts, drafts, parents, p, u, W):
    B = len(starts) - 1
    tokens, path = np.full((B, W), -1, dtype=np.int64), np.full((B, W), -1, dtype=np.int32)
    count = np.zeros(B, dtype=np.int32)
    for b in range(B):
        r0, n = starts[b], starts[b + 1] - starts[b]
        i, k = 0, 0
        while n > 0:
            path[b, k] = i
            y = tokens[b, k] = draw(p[r0 + i], u[r0 + i])
            kids = [j for j in range(1, n) if parents[r0 + j] == i and drafts[r0 + j] == y and y >= 0]
            if not kids or k + 1 == W:
                break
            i, k = kids[0], k + 1
        count[b] = k
    return tokens, path, count


class Case:
    def __init__(self, news, V, W, dtype, seed, sharp=8.0, gap=0, pad=0):
        r = random.Random(seed)
        g = torch.Generator().manual_seed(seed)
        self.starts = [gap]
        for n in news:
            self.starts.append(self.starts[-1] + n)
        T = self.starts[-1] + pad
        self.p = torch.softmax(torch.randn(T, V, generator=g) * sharp ** 0.5 * 2, -1).to(DT[dtype])
        self.u = torch.rand(T, generator=g)
        self.parents, self.drafts = torch.full((T,), 99, dtype=torch.int32), torch.randint(0, V, (T,), generator=g)
        for b, n in enumerate(news):
            if not n:
                continue
            par = tree(r, n, 0.4)
            par[0] = r.choice([-1, 0, 77])                    # a root's parent is not looked at
            self.parents[self.starts[b]:self.starts[b] + n] = torch.tensor(par, dtype=torch.int32)
            kids = {}
            for j in range(1, n):                             # children draft likely successors, now and then the same
                row = self.p[self.starts[b] + par[j]]
                k = kids.setdefault(par[j], [])
                likely = row.float().topk(min(4, V)).indices.tolist()
                k.append(r.choice(likely))
                self.drafts[self.starts[b] + j] = k[-1]
        self.W, self.T, self.B = W, T, len(news)

    def run(self):
        tokens = torch.full((self.B, self.W), 12345, dtype=torch.int64, device="cuda")
        path = torch.full((self.B, self.W), 12345, dtype=torch.int32, device="cuda")
        count = torch.full((self.B,), 12345, dtype=torch.int32, device="cuda")
        self.on = [x.cuda() for x in (self.drafts, self.parents, torch.tensor(self.starts, dtype=torch.int32), self.p, self.u)]
        pkv.speculative_accept_tree(tokens, path, count, *self.on)
        torch.cuda.synchronize()
        return tokens.cpu().numpy(), path.cpu().numpy(), count.cpu().numpy()

    def check(self):
        got = self.run()
        want = ref(self.starts, self.drafts.tolist(), self.parents.tolist(), self.p.float().numpy(), self.u.numpy(), self.W)
        for a, b, name in zip(got, want, ("tokens", "path", "count")):
            assert np.array_equal(a, b), (name, a, b)
        return want


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("news,V,W", [([1], 1, 1), ([1], 5, 3), ([3, 1, 7], 2, 4), ([8], 1000, 5), ([16] * 9, 4099, 8),
                                       ([64, 63, 0, 1, 33], 517, 64), ([0, 0], 100, 2), ([20] * 4, 32000, 7),
                                       ([12, 40], 50257, 6), ([64] * 30, 129, 3)])
def test_matches_the_reference(news, V, W, dtype):
    total = 0
    for seed in range(4):
        c = Case(news, V, W, dtype, 100 * seed + V % 97, gap=2, pad=3)
        total += int(c.check()[2].sum())
    if max(news) >= 8 and W > 2:
        assert total > 0                                      # some drafts were accepted


def test_rows_off_every_boundary():
    """Vocabularies of every remainder, 16-bit rows at every element."""
    for V in range(120, 137):
        for dtype in ("bf16", "f32"):
            Case([6, 11, 2], V, 6, dtype, V).check()


@pytest.mark.parametrize("V", [8185, 8191, 8192, 8193, 8196])
def test_around_the_vocabulary_of_one_cta(V):
    for dtype in DT:
        c = Case([9, 1, 30, 16], V, 6, dtype, V, gap=1)
        c.check()
        c.u[::2] = 1.0 - 2.0 ** -24                           # the row's last tokens, and its first
        c.u[1::2] = 0.0
        c.check()


def test_the_largest_vocabulary():
    c = Case([4, 6], pkv.ACCEPT_MAX_VOCAB, 5, "bf16", 3)
    c.check()
    c.u[:] = torch.tensor([0.0, 1.0 - 2.0 ** -24, 0.5, 0.999, 0.0, 1.0 - 2.0 ** -24, 0.25, 0.75, 0.1, 0.9])
    c.check()


def test_a_chain_of_certain_drafts():
    """One-hot rows: the walk follows the drafts to the tree's end, or to the width's."""
    n, V = 64, 300
    for W in (1, 2, 64, 40):
        c = Case([n, n], V, W, "f32", 5)
        c.p = torch.zeros(2 * n, V)
        want = torch.randint(0, V, (2 * n,), generator=torch.Generator().manual_seed(1))
        c.p[torch.arange(2 * n), want] = 1.0
        c.parents[:] = torch.tensor([-1] + list(range(n - 1))).repeat(2)
        c.drafts[1:] = want[:-1]                              # node j drafts its parent's only successor
        c.drafts[n + 9] = (int(want[n + 8]) + 1) % V          # the second chain breaks at its ninth node
        tokens, path, count = c.check()
        assert count[0] == min(W, n) - 1 and count[1] == min(W - 1, 8)


def test_children_of_the_same_token_and_foreign_ones():
    """The first child that drafted the token is taken; a node of another parent, or a draft outside the vocabulary, is not."""
    V = 50
    c = Case([6], V, 4, "f32", 6)
    c.p = torch.zeros(6, V)
    c.p[:, 7] = 1.0
    c.parents[:] = torch.tensor([-1, 0, 0, 0, 2, 1])
    c.drafts[:] = torch.tensor([7, 8, 7, 7, 1 << 40, 7])
    tokens, path, count = c.check()
    assert path[0].tolist() == [0, 2, -1, -1] and tokens[0].tolist() == [7, 7, -1, -1]
    c.drafts[4] = 7 + (1 << 32)                               # (not 7, whatever 32 bits say)
    assert c.check()[2][0] == 1
    c.drafts[4] = -1
    c.p[2] = 0.0                                              # and no weight at all: -1, which no draft is
    tokens, path, count = c.check()
    assert tokens[0].tolist() == [7, -1, -1, -1] and path[0].tolist() == [0, 2, -1, -1]


def test_odd_weights_and_random_numbers():
    c = Case([5, 5, 5], 333, 5, "f32", 7)
    c.p[0, ::2] = -1.0
    c.p[0, 1::4] = math.nan
    c.p[0, 3] = math.inf
    c.p[5] = math.nan
    c.p[10] = 2.0 ** -45                                      # below a unit
    c.check()
    for u in (0.0, -0.5, 1.0, 7.0, math.nan, math.inf, 1.0 - 2.0 ** -24):
        c = Case([5, 9], 333, 5, "f16", 8)
        c.u[:] = u
        c.check()


def test_bad_trees_raise_the_error_word():
    c = Case([6, 5], 64, 5, "f32", 9)
    c.parents[3], c.parents[4], c.parents[8] = 3, 6, -1       # itself, a later node, none: nobody's child
    c.drafts[6:] = 0
    c.run()
    assert pkv.device_error(reset=True) == 1
    c.check()                                                 # (the reference's walk: such a node is on no path)
    assert pkv.device_error(reset=True) == 1
    for starts in ([-1, 6, 11], [0, 12, 11], [0, 6, 5], [0, 6, 1 << 30]):
        c = Case([6, 5], 64, 5, "f32", 9)
        c.starts = starts
        tokens, path, count = c.run()
        assert pkv.device_error(reset=True) == 1
        for b in range(2):
            if not (0 <= starts[b] <= starts[b + 1] <= 11):
                assert (tokens[b] == -1).all() and (path[b] == -1).all() and count[b] == 0
            else:
                assert path[b, 0] == 0
    c = Case([65, 3], 64, 5, "f32", 9)
    tokens, path, count = c.run()
    assert pkv.device_error(reset=True) == 1
    assert (tokens[0] == -1).all() and count[0] == 0 and path[1, 0] == 0


def test_streams_and_graphs():
    cases = [Case([12] * 20, 3001, 6, "bf16", 30 + i) for i in range(3)]
    want = [c.check() for c in cases]
    outs = [[torch.empty(20, 6, dtype=torch.int64, device="cuda"), torch.empty(20, 6, dtype=torch.int32, device="cuda"),
             torch.empty(20, dtype=torch.int32, device="cuda")] for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, o in zip(cases, outs):
            with torch.cuda.stream(torch.cuda.Stream()):
                pkv.speculative_accept_tree(*o, *c.on)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(o, w))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        pkv.speculative_accept_tree(*outs[0], *cases[0].on)
    for i in (1, 2):
        for a, b in zip(cases[0].on, cases[i].on):
            a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(outs[0], want[i]))


def test_offsets_past_32_bits():
    """A sequence whose rows lie past the first 2^31 elements of target_probs."""
    V = 400001
    T = 2 ** 31 // V + 8
    c = Case([7], V, 5, "f16", 40)
    want = c.check()
    p = torch.zeros(T, V, dtype=torch.float16, device="cuda")
    p[T - 7:] = c.p.cuda()
    full = lambda x: torch.cat([torch.zeros(T - 7, dtype=x.dtype), x]).cuda()
    tokens, path, count = (torch.empty(s, dtype=d, device="cuda") for s, d in (((1, 5), torch.int64), ((1, 5), torch.int32), ((1,), torch.int32)))
    pkv.speculative_accept_tree(tokens, path, count, full(c.drafts), full(c.parents),
                                torch.tensor([T - 7, T], dtype=torch.int32).cuda(), p, full(c.u))
    torch.cuda.synchronize()
    for a, b in zip((tokens, path, count), want):
        assert np.array_equal(a.cpu().numpy(), b)
