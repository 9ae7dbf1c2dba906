"""paged_kv_keep_path against plain moves of whole rows: every pool bit for bit, rows of no move as they were."""
import random

import pytest
import torch

import paged_kv_cache_156_gb300 as pkv

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_error_word():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pkv.device_error(reset=True)
    yield
    assert pkv.device_error(reset=True) == 0


class Case:
    """news[s] nodes at the end of totals[s] positions, paths[s] kept."""
    def __init__(self, news, totals, paths, layers, Hkv, d, bs, dtype, seed=0, W=None, gap=0):
        g = torch.Generator().manual_seed(seed)
        need = [-(-t // bs) for t in totals]
        self.NB, self.bs = sum(need) + 3, bs
        order = torch.randperm(self.NB, generator=g).int()
        self.tables = torch.full((len(news), max(need + [1]) + 1), self.NB + 9, dtype=torch.int32)
        at = 0
        for s, n in enumerate(need):
            self.tables[s, :n] = order[at:at + n]
            at += n
        el = torch.uint8 if dtype == "e4m3" else torch.int16
        self.pools = [torch.randint(0, 256 if dtype == "e4m3" else 30000, (self.NB, bs, Hkv, d), generator=g, dtype=el)
                      for _ in range(2 * layers)]
        self.view = {"e4m3": torch.uint8, "f16": torch.float16, "bf16": torch.bfloat16}[dtype]
        W = W or max(len(p) for p in paths) + 1
        self.path = torch.full((len(news), W), 1 << 20, dtype=torch.int32)
        for s, p in enumerate(paths):
            self.path[s, :len(p)] = torch.tensor(p, dtype=torch.int32)
        self.count = torch.tensor([max(len(p) - 1, 0) for p in paths], dtype=torch.int32)
        self.starts = torch.tensor([gap + sum(news[:i]) for i in range(len(news) + 1)], dtype=torch.int32)
        self.lens = torch.tensor(totals, dtype=torch.int32)
        self.news, self.totals, self.paths = news, totals, paths

    def expected(self, skip=()):
        out = [p.clone() for p in self.pools]
        for s, (n, L, path) in enumerate(zip(self.news, self.totals, self.paths)):
            if s in skip:
                continue
            at = [divmod(L - n + j, self.bs) for j in range(n)]
            where = [(int(self.tables[s, b]), o) for b, o in at]
            for p, q in zip(out, self.pools):
                for i, j in enumerate(path):
                    p[where[i]] = q[where[j]]
        return out

    def on(self):
        self.dev = [p.cuda() for p in self.pools]
        pools = [p.view(self.view) for p in self.dev]
        return [pools[0::2], pools[1::2]] + [t.cuda() for t in (self.tables, self.lens, self.starts, self.path, self.count)]

    def check(self, skip=()):
        pkv.paged_kv_keep_path(*self.on())
        torch.cuda.synchronize()
        for i, (got, want) in enumerate(zip(self.dev, self.expected(skip))):
            assert torch.equal(got.cpu(), want), f"pool {i}"


def random_paths(r, news):
    return [[0] + sorted(r.sample(range(1, n), r.randint(0, n - 1))) if n else [] for n in news]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("Hkv,d,bs,layers", [(1, 16, 1, 1), (4, 64, 8, 2), (8, 128, 16, 3), (3, 80, 7, 1), (2, 128, 32, 70)])
def test_random_paths(Hkv, d, bs, layers, dtype):
    r = random.Random(Hkv)
    news = [1, 64, 0, 33, 7, 2, 64, 20]
    totals = [1, 64, 9, 40, 300, 2, 129, 25]
    for seed in range(2):
        Case(news, totals, random_paths(r, news), layers, Hkv, d, bs, dtype, seed, gap=5).check()


def test_paths_at_the_edges():
    """The root alone, every node (nothing moves), the last nodes only, every other one (each place another's source)."""
    n = 64
    paths = [[0], list(range(n)), [0] + list(range(n - 9, n)), list(range(0, n, 2)), [0, 63], [0, 2, 3, 4, 5], [0, 1, 2, 62]]
    for W in (64, None):
        Case([n] * len(paths), [n + 13 * i for i in range(len(paths))], paths, 2, 8, 128, 16, "bf16", W=W).check()


def test_a_row_wider_than_a_block_of_threads():
    Case([9, 5], [20, 90], [[0, 4, 5, 8], [0, 3]], 2, 40, 256, 16, "bf16").check()


def test_bad_paths_are_left_alone_and_raise_the_error_word():
    news, totals = [8] * 3, [30, 8, 100]
    good = [[0, 3, 5], [0, 7], [0, 1, 4]]
    for s, change in ((0, dict(path=[1, 3, 5])), (1, dict(path=[0, 8])), (2, dict(path=[0, 4, 4])), (0, dict(path=[0, 5, 3])),
                      (1, dict(path=[0, -1])), (2, dict(count=-1)), (2, dict(count=3)), (0, dict(count=8)), (1, dict(count=64)),
                      (1, dict(length=7)), (2, dict(length=1 << 30)), (0, dict(length=-5))):
        c = Case(news, totals, good, 2, 2, 64, 16, "f16", W=3 if change.get("count") == 3 else 10)
        if "path" in change:
            c.path[s, :len(change["path"])] = torch.tensor(change["path"], dtype=torch.int32)
        if "count" in change:
            c.count[s] = change["count"]
        if "length" in change:
            c.lens[s] = change["length"]
        c.check(skip=(s,))
        assert pkv.device_error(reset=True) == 1, change
    c = Case([65, 8], [100, 8], [[0, 9], [0, 3]], 1, 2, 64, 16, "f16")
    c.check(skip=(0,))
    assert pkv.device_error(reset=True) == 1
    c = Case([8, 8], [30, 8], [[0, 9 - 2], [0, 3]], 1, 2, 64, 16, "f16")
    c.starts[1] = -3                                          # (differences below 0, and above 64 nodes' worth)
    c.starts[2] = 100
    c.check(skip=(0, 1))
    assert pkv.device_error(reset=True) == 1
    c = Case([0, 4], [30, 8], [[], [0, 3]], 1, 2, 64, 16, "f16")
    c.count[0] = 1                                            # kept drafts of no tree
    c.check(skip=(0,))
    assert pkv.device_error(reset=True) == 1


def test_bad_table_entries_raise_the_error_word():
    """A row whose block is out of range is not moved; the sequence's other rows are."""
    c = Case([20], [40], [[0, 2, 17]], 2, 2, 64, 16, "f16")
    want = c.expected()
    c.tables[0, 2] = c.NB                                     # position 37, the last source
    pkv.paged_kv_keep_path(*c.on())
    torch.cuda.synchronize()
    assert pkv.device_error(reset=True) == 1
    blk, off = int(c.tables[0, 22 // 16]), 22 % 16
    for got, w, before in zip(c.dev, want, c.pools):
        got = got.cpu()
        assert torch.equal(got[blk, off], before[blk, off])
        got[blk, off] = w[blk, off]
        assert torch.equal(got, w)
    c.tables[0, 2] = -1
    pkv.paged_kv_keep_path(*c.on())
    torch.cuda.synchronize()
    assert pkv.device_error(reset=True) == 1


def test_single_pools_streams_and_graphs():
    r = random.Random(5)
    news, totals = [20, 30], [50, 64]
    c = Case(news, totals, random_paths(r, news), 1, 4, 64, 16, "bf16", W=32)
    k, v, *rest = c.on()
    with torch.cuda.stream(torch.cuda.Stream()):
        pkv.paged_kv_keep_path(k[0], v[0], *rest)
    torch.cuda.synchronize()
    for got, want in zip(c.dev, c.expected()):
        assert torch.equal(got.cpu(), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        pkv.paged_kv_keep_path(k, v, *rest)
    for seed in (1, 2):
        new = Case(news, totals, random_paths(r, news), 1, 4, 64, 16, "bf16", seed, W=32)
        for a, b in zip(c.dev, new.pools):
            a.copy_(b)
        for a, b in zip(rest, (new.tables, new.lens, new.starts, new.path, new.count)):
            a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        for got, want in zip(c.dev, new.expected()):
            assert torch.equal(got.cpu(), want)


def test_offsets_past_32_bits():
    """Blocks past a pool's first 2^31 elements."""
    c = Case([30], [100], [[0, 4, 9, 29]], 1, 8, 128, 32, "bf16")
    NB = 2 ** 31 // (32 * 8 * 128) + c.NB
    big = [torch.zeros(NB, 32, 8, 128, dtype=torch.int16, device="cuda") for _ in c.pools]
    for b, p in zip(big, c.pools):
        b[NB - c.NB:] = p.cuda()
    k, v, tables, *rest = c.on()
    pkv.paged_kv_keep_path(big[0].view(torch.bfloat16), big[1].view(torch.bfloat16), (tables + (NB - c.NB)).int(), *rest)
    torch.cuda.synchronize()
    for b, want in zip(big, c.expected()):
        assert torch.equal(b[NB - c.NB:].cpu(), want)
        assert not b[:c.NB].any()
