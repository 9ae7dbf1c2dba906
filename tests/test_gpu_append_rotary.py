"""paged_kv_append_rotary against a plain reference.

Rotated values are held to a bound in 64 bits: two products and a sum, each rounded to fp32 (2^-24 relative), then one
rounding to the output's type: |x c - y s| is off by at most 2^-24 (2 |x c| + 2 |y s|) (a product's rounding and the
sum's; (1 + 2^-24)^2 taken as 1 + 2 2^-24, with 2^-40 for the rest) before half a step of the type, 2^-25 where fp16's
subnormals round.  Codes of E4M3 pools must be the ones that fp32 products, sums and divisions rounded one by one give.
What is not rotated, values, and every slot that no token has are bit for bit.
"""
import math

import pytest
import torch

import paged_kv_cache_156_gb300 as pkv

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _clean_error_word():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pkv.device_error(reset=True)
    yield
    assert pkv.device_error(reset=True) == 0


def table(P, r, base=10000.0):
    a = torch.arange(P, dtype=torch.float64)[:, None] * base ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    return torch.cat([a.cos(), a.sin()], 1).float()


def turned(x, cs, interleaved, dtype):
    """(rotated x, the sum of its products' magnitudes) in ``dtype``, each operation rounded there."""
    r = cs.shape[1]
    c, s = cs[:, None, :r // 2].to(dtype), cs[:, None, r // 2:].to(dtype)
    x = x.to(dtype)
    y, mag = x.clone(), torch.zeros_like(x)
    a, b = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    mag[..., a] = (x[..., a] * c).abs() + (x[..., b] * s).abs()
    mag[..., b] = (x[..., b] * c).abs() + (x[..., a] * s).abs()
    return y, mag


class Call:
    def __init__(self, T, Hq, Hkv, d, r, bs, dtype, e4m3=False, packed=False, P=997, seed=0, blocks=None):
        g = torch.Generator().manual_seed(seed)
        dt = DT[dtype]
        if packed:
            qkv = torch.randn(T, (Hq + 2 * Hkv) * d + 8, generator=g).to(dt).cuda()
            self.packed = qkv
            self.q, self.k, self.v = (x.unflatten(1, (-1, d)) for x in
                                      qkv[:, :-8].split((Hq * d, Hkv * d, Hkv * d), 1))
        else:
            self.q, self.k, self.v = (torch.randn(T, h, d, generator=g).to(dt).cuda() for h in (Hq, Hkv, Hkv))
        NB = blocks or -(-T // bs) + 2
        if e4m3:
            self.kc, self.vc = (torch.randint(0, 256, (NB, bs, Hkv, d), generator=g, dtype=torch.uint8).cuda() for _ in "kv")
            self.ks, self.vs = ((torch.rand(Hkv, generator=g) * 0.02 + 0.002).cuda() for _ in "kv")
        else:
            self.kc, self.vc = (torch.full((NB, bs, Hkv, d), math.nan, dtype=dt, device="cuda") for _ in "kv")
            self.ks = self.vs = None
        self.slots = torch.randperm(NB * bs, generator=g)[:T].cuda()
        self.pos = torch.randint(0, P, (T,), generator=g, dtype=torch.int32).cuda()
        self.cs = table(P, r).cuda()
        self.q_out = torch.full((T, Hq, d), math.nan, dtype=dt, device="cuda")

    def run(self, interleaved=False, q_out=None, q="q"):
        pkv.paged_kv_append_rotary(self.q_out if q_out is None else q_out, self.q if q == "q" else q, self.k, self.v, self.kc,
                                   self.vc, self.slots, self.pos, self.cs, interleaved=interleaved, k_scale=self.ks,
                                   v_scale=self.vs)


def verify(c, interleaved, before_k, before_v, live=None, q=None, q_out=None):
    """The call's outputs against the reference; ``live``: the tokens whose rows are cached."""
    q = c.q if q is None else q
    q_out = c.q_out if q_out is None else q_out
    T = c.k.shape[0]
    live = torch.ones(T, dtype=torch.bool) if live is None else live
    cs = c.cs.cpu()[c.pos.cpu().long().clamp(0, c.cs.shape[0] - 1)]
    r = cs.shape[1]
    half = torch.finfo(q.dtype).eps / 2

    def check(got, x):
        want, mag = turned(x.cpu(), cs, interleaved, torch.float64)
        err = 2.0 ** -23 * mag * (1 + 2.0 ** -16)
        bound = err + half * (want.abs() + err) + 2.0 ** -25
        got = got.cpu().double()
        worst = ((got - want).abs() / bound)[live if got.shape[0] == T and x is not q else slice(None)]
        assert not torch.isnan(worst).any() and (worst.numel() == 0 or float(worst.max()) <= 1.0)

    check(q_out, q)
    assert torch.equal(q_out[..., r:].cpu().view(torch.int16), q[..., r:].contiguous().cpu().view(torch.int16))
    at = c.slots.cpu()[live]
    for pool, before, x, scale, turns in ((c.kc, before_k, c.k, c.ks, True), (c.vc, before_v, c.v, c.vs, False)):
        flat, old = pool.flatten(0, 1).cpu(), before.flatten(0, 1).cpu()
        rest = torch.ones(flat.shape[0], dtype=torch.bool)
        rest[at] = False
        raw = torch.uint8 if scale is not None else torch.int16
        assert torch.equal(flat[rest].view(raw), old[rest].view(raw)), "a slot of no token was written"
        if scale is not None:
            y = (turned(x.cpu(), cs, interleaved, torch.float32)[0] if turns else x.cpu().float())
            want = (y / scale.cpu()[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            assert torch.equal(flat[at], want[live])
        elif turns:
            got = torch.zeros(T, *flat.shape[1:], dtype=flat.dtype)
            got[live] = flat[at]
            check(got, x)
            assert torch.equal(flat[at][..., r:].view(raw), x.cpu()[live][..., r:].contiguous().view(raw))
        else:
            assert torch.equal(flat[at].view(raw), x.cpu()[live].contiguous().view(raw))


# tokens, heads, kv heads, dim, rotary, block, dtype
CASES = [
    (1, 1, 1, 16, 16, 1, "f16"), (1, 4, 4, 64, 64, 16, "bf16"), (4, 4, 4, 64, 64, 16, "f16"), (17, 32, 8, 128, 128, 16, "bf16"),
    (64, 64, 8, 128, 64, 32, "f16"), (33, 12, 4, 64, 48, 8, "bf16"), (130, 7, 1, 80, 32, 16, "f16"),
    (5, 3, 3, 256, 16, 5, "bf16"), (3, 128, 16, 128, 128, 16, "f16"), (300, 5, 1, 112, 112, 7, "bf16"),
    (2, 2, 1, 4096, 4096, 3, "f16"), (999, 32, 8, 128, 128, 16, "bf16"),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_matches_the_reference(case, packed, interleaved):
    c = Call(*case, packed=packed, seed=case[0])
    k0, v0 = c.kc.clone(), c.vc.clone()
    c.run(interleaved)
    verify(c, interleaved, k0, v0)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_e4m3_pools(case, interleaved):
    c = Call(*case, e4m3=True, packed=case[0] % 2 == 1, seed=case[0])
    c.v[0, 0, :4] = torch.tensor([1e4, -1e4, math.nan, 0.0], dtype=c.v.dtype)       # saturates, NaN stays NaN
    k0, v0 = c.kc.clone(), c.vc.clone()
    c.run(interleaved)
    got = c.vc.flatten(0, 1)[c.slots[0], 0, :4].tolist()
    assert got[0] == 0x7e and got[1] == 0xfe and got[2] & 0x7f == 0x7f and got[3] == 0
    c.v[0, 0, 2] = 0                                                                 # (the sign of a NaN's code is not fixed)
    want = c.vc.flatten(0, 1)
    want[c.slots[0], 0, 2] = 0
    verify(c, interleaved, k0, v0)


def test_unpadded_codes_equal_the_append_call():
    """Angles of zero: the call is paged_kv_append_fp8 (and paged_kv_append), bit for bit."""
    for e4m3 in (True, False):
        c = Call(77, 8, 2, 128, 128, 16, "bf16", e4m3=e4m3, seed=3)
        c.pos.zero_()
        kc, vc = c.kc.clone(), c.vc.clone()
        c.run()
        if e4m3:
            pkv.paged_kv_append_fp8(c.k, c.v, kc, vc, c.slots, c.ks, c.vs)
        else:
            pkv.paged_kv_append(c.k, c.v, kc, vc, c.slots)
        raw = torch.uint8 if e4m3 else torch.int16
        assert torch.equal(kc.view(raw), c.kc.view(raw)) and torch.equal(vc.view(raw), c.vc.view(raw))
        assert torch.equal(c.q_out, c.q)


@pytest.mark.parametrize("packed", [False, True])
def test_queries_in_place_and_none(packed):
    c = Call(50, 8, 2, 128, 64, 16, "bf16", packed=packed, seed=4)
    k0, v0, q = c.kc.clone(), c.vc.clone(), c.q.clone()
    c.run(q_out=c.q)
    verify(c, False, k0, v0, q=q, q_out=c.q)
    d = Call(50, 8, 2, 128, 64, 16, "bf16", packed=packed, seed=4)
    pkv.paged_kv_append_rotary(None, None, d.k, d.v, d.kc, d.vc, d.slots, d.pos, d.cs)
    assert torch.equal(d.kc.view(torch.int16), c.kc.view(torch.int16)) and torch.equal(d.vc.view(torch.int16), c.vc.view(torch.int16))
    assert torch.equal(d.q, q)
    if packed:
        assert torch.equal(d.packed[:, -8:], c.packed[:, -8:])


def test_padding_and_no_tokens():
    """Negative slots are not cached, their queries turn all the same; a negative position beside one leaves the token out."""
    c = Call(20, 4, 2, 64, 64, 16, "f16", seed=5)
    c.slots[3], c.slots[9], c.slots[19] = -1, -7, -(1 << 62)
    live = torch.ones(20, dtype=torch.bool)
    live[[3, 9, 19]] = False
    c.pos[9] = -1
    k0, v0 = c.kc.clone(), c.vc.clone()
    c.run()
    assert torch.isnan(c.q_out[9]).all()
    c.q_out[9] = 0                              # (position -1: the rest as if at position 0)
    c.pos[9] = 0
    c.q[9] = 0
    verify(c, False, k0, v0, live)
    e = Call(1, 4, 2, 64, 64, 16, "f16")
    pkv.paged_kv_append_rotary(e.q_out[:0], e.q[:0], e.k[:0], e.v[:0], e.kc, e.vc, e.slots[:0], e.pos[:0], e.cs)
    assert torch.isnan(e.kc).all()


def test_slots_and_positions_out_of_range():
    c = Call(6, 4, 2, 64, 64, 16, "f16", seed=6)
    n = c.kc.shape[0] * 16
    k0, v0 = c.kc.clone(), c.vc.clone()
    c.slots[1], c.slots[4] = n, 1 << 40                       # not cached, turned
    c.pos[2], c.pos[5] = 997, -1                              # left out
    c.run()
    torch.cuda.synchronize()
    assert pkv.device_error(reset=True) == 1
    live = torch.tensor([True, False, False, True, False, False])
    assert torch.isnan(c.q_out[[2, 5]]).all()
    c.q_out[[2, 5]] = 0
    c.q[[2, 5]] = 0
    verify(c, False, k0, v0, live)
    for bad in (997, 2 ** 31 - 1, -2 ** 31):
        c = Call(1, 4, 2, 64, 64, 16, "f16", seed=7)
        c.pos[0] = bad
        c.run()
        torch.cuda.synchronize()
        assert pkv.device_error(reset=True) == 1 and torch.isnan(c.kc).all() and torch.isnan(c.q_out).all()


def test_non_finite_values_stay_in_their_pairs():
    c = Call(3, 4, 2, 64, 32, 16, "bf16", seed=8)
    c.q[1, 2, 5], c.k[1, 1, 20], c.v[2, 0, 7] = math.nan, math.inf, -math.inf
    c.run()
    q, k, v = c.q_out[1, 2], c.kc.flatten(0, 1)[c.slots[1], 1], c.vc.flatten(0, 1)[c.slots[2], 0]
    assert torch.isnan(q).nonzero().flatten().tolist() == [5, 21]
    assert (~torch.isfinite(k)).nonzero().flatten().tolist() == [4, 20] and v[7] == -math.inf
    assert torch.isfinite(c.q_out[0]).all() and torch.isfinite(c.q_out[2]).all()


def test_far_positions():
    """The table's last rows, and rows past the first 2^31 bytes of it."""
    c = Call(4, 2, 1, 128, 128, 16, "f16", seed=9)
    P = 2 ** 31 // (128 * 4) + 1000
    big = torch.zeros(P, 128, device="cuda")
    rows = torch.tensor([0, 996, P - 1, P - 500], dtype=torch.int32)
    big[rows.long().cuda()] = c.cs[[5, 6, 7, 8]]
    c.pos = rows.cuda()
    k0, v0, small = c.kc.clone(), c.vc.clone(), c.cs
    c.cs = big
    c.run()
    c.cs, c.pos = small, torch.tensor([5, 6, 7, 8], dtype=torch.int32).cuda()
    verify(c, False, k0, v0)


def test_offsets_past_32_bits():
    """Slots past the pool's first 2^31 elements, tokens past the rows' first 2^31."""
    bs, Hkv, d = 32, 8, 128
    c = Call(40, 8, Hkv, d, d, bs, "bf16", blocks=2 ** 31 // (bs * Hkv * d) + 4, seed=10)
    n = c.kc.shape[0] * bs
    c.slots = (n - 1 - 3 * torch.arange(40)).cuda()
    width = 2 ** 31 // 39 // 8 * 8 + 8                        # the last token's row lies past 2^31 elements
    rows = torch.empty(40 * width, dtype=torch.bfloat16, device="cuda").view(40, width)
    rows[:, :8 * d] = c.q.flatten(1)
    c.q = rows[:, :8 * d].unflatten(1, (8, d))
    c.run()
    torch.cuda.synchronize()
    tail = slice(n - 128, n)
    small = Call(40, 8, Hkv, d, d, bs, "bf16", seed=10)       # the same rows into a small pool
    small.slots = (127 - 3 * torch.arange(40)).clamp(min=0).cuda()
    small.kc, small.vc = (torch.full((4, bs, Hkv, d), math.nan, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    small.k, small.v, small.pos, small.cs = c.k, c.v, c.pos, c.cs
    small.run(q_out=small.q_out)
    assert torch.equal(small.kc.flatten(0, 1).view(torch.int16), c.kc.flatten(0, 1)[tail].view(torch.int16))
    assert torch.equal(small.vc.flatten(0, 1).view(torch.int16), c.vc.flatten(0, 1)[tail].view(torch.int16))
    assert torch.equal(c.q_out, small.q_out)


def test_other_streams_and_graphs():
    calls = [Call(64, 8, 2, 128, 128, 16, "bf16", seed=20 + i, e4m3=i == 1) for i in range(2)]
    want = [Call(64, 8, 2, 128, 128, 16, "bf16", seed=20 + i, e4m3=i == 1) for i in range(2)]
    for w in want:
        w.run()
    torch.cuda.synchronize()
    for c in calls:
        with torch.cuda.stream(torch.cuda.Stream()):
            c.run()
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        raw = torch.uint8 if w.ks is not None else torch.int16
        assert torch.equal(c.q_out, w.q_out) and torch.equal(c.kc.view(raw), w.kc.view(raw))
    c, g = calls[0], torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        c.run()
    for seed in (31, 32):
        new = Call(64, 8, 2, 128, 128, 16, "bf16", seed=seed)
        for a, b in ((c.q, new.q), (c.k, new.k), (c.v, new.v), (c.slots, new.slots), (c.pos, new.pos)):
            a.copy_(b)
        c.kc.fill_(math.nan)
        c.vc.fill_(math.nan)
        k0, v0 = c.kc.clone(), c.vc.clone()
        g.replay()
        torch.cuda.synchronize()
        verify(c, False, k0, v0)
