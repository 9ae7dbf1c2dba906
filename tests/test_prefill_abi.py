"""Host-side validation of the prefill, gather and accept calls: bad arguments are refused before any CUDA call,
empty work is accepted without touching the device, and the binding checks shapes and types.  No GPU."""
import ctypes

import pytest
import torch

import paged_kv_cache_156_gb300 as pkv
from paged_kv_cache_156_gb300 import _build

null = ctypes.c_void_p(0)
fake = ctypes.c_void_p(256)             # a non-null, aligned address that nothing dereferences
odd = ctypes.c_void_p(258)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkv.load()


def prefill(lib, fp8=False, ptr=fake, B=2, T=10, max_len=40, Hq=8, Hkv=2, d=128, bs=16, nb=10, scale=1.0, dt=0, ws=null,
            ws_bytes=0, planned=0, width=4, starts=fake, lens=fake, ks=fake, vs=fake, tables=fake):
    args = [ptr, ptr, ptr, ptr, tables, width, lens, starts, B, T, max_len, Hq, Hkv, d, bs, nb, scale, dt]
    if fp8:
        return lib.pkv_paged_attention_prefill_fp8(*args, ks, vs, ws, ws_bytes, planned, null)
    return lib.pkv_paged_attention_prefill(*args, ws, ws_bytes, planned, null)


@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_refusals(lib, fp8):
    def call(**kw):
        return prefill(lib, fp8, **kw), lib.pkv_last_error()

    ok_ws = dict(ws=fake, ws_bytes=1 << 40)
    for kw, status, word in (
            (dict(d=96), pkv.PKV_ERR_UNSUPPORTED, b"head_dim"), (dict(bs=12), pkv.PKV_ERR_UNSUPPORTED, b"block_size"),
            (dict(dt=2), pkv.PKV_ERR_UNSUPPORTED, b"dtype"), (dict(dt=3), pkv.PKV_ERR_UNSUPPORTED, b"dtype"),
            (dict(Hq=7), pkv.PKV_ERR_INVALID, b"num_heads"), (dict(Hkv=0), pkv.PKV_ERR_INVALID, b"num_heads"),
            (dict(B=-1), pkv.PKV_ERR_INVALID, b"num_seqs"), (dict(B=65536), pkv.PKV_ERR_INVALID, b"num_seqs"),
            (dict(T=-1), pkv.PKV_ERR_INVALID, b"num_tokens"), (dict(T=1 << 27), pkv.PKV_ERR_INVALID, b"num_tokens"),
            (dict(T=1 << 62), pkv.PKV_ERR_INVALID, b"num_tokens"),
            (dict(max_len=-1), pkv.PKV_ERR_INVALID, b"max_seq_len"), (dict(max_len=65), pkv.PKV_ERR_INVALID, b"max_seq_len"),
            (dict(nb=0), pkv.PKV_ERR_INVALID, b"num_blocks"), (dict(nb=(1 << 31) + 1), pkv.PKV_ERR_INVALID, b"num_blocks"),
            (dict(scale=float("nan")), pkv.PKV_ERR_INVALID, b"scale"), (dict(scale=float("inf")), pkv.PKV_ERR_INVALID, b"scale"),
            (dict(planned=2), pkv.PKV_ERR_INVALID, b"planned"), (dict(planned=-1), pkv.PKV_ERR_INVALID, b"planned"),
            (dict(starts=null), pkv.PKV_ERR_INVALID, b"null"), (dict(lens=odd), pkv.PKV_ERR_INVALID, b"aligned"),
            (dict(), pkv.PKV_ERR_WORKSPACE, b"workspace"), (dict(ws=fake, ws_bytes=100), pkv.PKV_ERR_WORKSPACE, b"workspace"),
            (dict(ws=odd, ws_bytes=1 << 40), pkv.PKV_ERR_WORKSPACE, b"workspace"),
            (dict(ptr=null, **ok_ws), pkv.PKV_ERR_INVALID, b"null"), (dict(tables=null, **ok_ws), pkv.PKV_ERR_INVALID, b"null"),
            (dict(ptr=ctypes.c_void_p(264), **ok_ws), pkv.PKV_ERR_INVALID, b"16-byte")):
        st, msg = call(**kw)
        assert st == status and word in msg, (kw, st, msg)
    # no sequences or no new tokens: nothing to do
    assert call(B=0)[0] == pkv.PKV_OK and call(T=0)[0] == pkv.PKV_OK
    if fp8:
        assert call(d=64)[0] == pkv.PKV_ERR_UNSUPPORTED
        for kw in (dict(ks=null), dict(vs=null), dict(ks=odd), dict(vs=odd)):
            assert call(**kw)[0] == pkv.PKV_ERR_INVALID


def test_prefill_plan_refusals_and_workspace(lib):
    def plan(lens=fake, starts=fake, B=2, T=10, max_len=40, Hq=8, Hkv=2, d=128, ws=null, n=0):
        return lib.pkv_prefill_plan(lens, starts, B, T, max_len, Hq, Hkv, d, ws, n, null)

    assert plan(d=80) == pkv.PKV_ERR_UNSUPPORTED and plan(Hq=9) == pkv.PKV_ERR_INVALID
    assert plan(lens=null) == pkv.PKV_ERR_INVALID and plan(starts=odd) == pkv.PKV_ERR_INVALID
    assert plan() == pkv.PKV_ERR_WORKSPACE and plan(B=0) == pkv.PKV_OK and plan(T=0) == pkv.PKV_OK
    n = pkv.prefill_workspace_bytes
    for B in (1, 64, 1024, 65535):
        for T in (0, 1, 513, 100000):
            for Hq, Hkv in ((1, 1), (32, 8), (64, 8), (40, 1)):
                for d in (64, 128):
                    # without a GPU the layout takes 152 SMs: at least the partials of two parts an SM, and it
                    # never shrinks as tokens are added
                    assert n(B, T, Hq, Hkv, d) <= n(B, T + 1, Hq, Hkv, d) < 1 << 34
    for bad in ((1, -1, 8, 2, 128), (1, 1, 8, 3, 128), (1, 1, 8, 2, 100), (-1, 1, 8, 2, 128), (1, 1 << 30, 8, 2, 128)):
        with pytest.raises(ValueError):
            n(*bad)


def test_gather_refusals(lib):
    def call(fp8=False, out=fake, pool=fake, tables=fake, width=4, lens=fake, starts=fake, B=2, R=10, nb=10, bs=16, Hkv=2,
             d=64, dt=0, ks=fake, vs=fake):
        args = [out, out, pool, pool, tables, width, lens, starts, B, R, nb, bs, Hkv, d, dt]
        if fp8:
            return lib.pkv_paged_kv_gather_fp8(*args, ks, vs, null)
        return lib.pkv_paged_kv_gather(*args, null)

    for fp8 in (False, True):
        assert call(fp8, dt=2) == pkv.PKV_ERR_UNSUPPORTED and call(fp8, dt=3) == pkv.PKV_ERR_UNSUPPORTED
        for kw in (dict(B=-1), dict(R=-1), dict(R=1 << 31), dict(d=4), dict(d=12), dict(Hkv=0), dict(Hkv=4097), dict(d=4104),
                   dict(nb=0), dict(bs=0), dict(width=-1), dict(out=null), dict(pool=null), dict(tables=null),
                   dict(lens=null), dict(starts=null), dict(out=ctypes.c_void_p(264)), dict(pool=ctypes.c_void_p(260)),
                   dict(tables=odd), dict(lens=odd), dict(starts=odd)):
            assert call(fp8, **kw) == pkv.PKV_ERR_INVALID, (fp8, kw)
        assert call(fp8, B=0) == pkv.PKV_OK and call(fp8, R=0) == pkv.PKV_OK
    assert call(pool=ctypes.c_void_p(264)) == pkv.PKV_ERR_INVALID       # (8-byte aligned is enough for E4M3 only)
    assert call(True, ks=null) == pkv.PKV_ERR_INVALID and call(True, vs=odd) == pkv.PKV_ERR_INVALID


def test_accept_refusals(lib):
    def call(tokens=fake, acc=fake, drafts=fake, counts=null, target=fake, draft=null, uniform=fake, B=2, K=3, V=100, dt=3):
        return lib.pkv_speculative_accept(tokens, acc, drafts, counts, target, draft, uniform, B, K, V, dt, null)

    assert call(dt=2) == pkv.PKV_ERR_UNSUPPORTED and call(dt=4) == pkv.PKV_ERR_UNSUPPORTED
    for kw in (dict(B=-1), dict(B=(1 << 24) + 1), dict(K=-1), dict(K=1025), dict(V=0), dict(V=pkv.ACCEPT_MAX_VOCAB + 1),
               dict(tokens=null), dict(acc=null), dict(drafts=null), dict(target=null), dict(uniform=null),
               dict(tokens=ctypes.c_void_p(260)), dict(drafts=ctypes.c_void_p(260)), dict(acc=odd), dict(counts=odd),
               dict(uniform=odd), dict(target=odd), dict(draft=odd), dict(target=ctypes.c_void_p(257), dt=1)):
        assert call(**kw) == pkv.PKV_ERR_INVALID, kw
    assert call(B=0) == pkv.PKV_OK


def test_header_and_binding_agree_on_the_vocabulary_limit():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "pkv.h")).read()
    assert int(re.search(r"#define\s+PKV_ACCEPT_MAX_VOCAB\s+(\d+)", text).group(1)) == pkv.ACCEPT_MAX_VOCAB
    assert re.search(r"PKV_F32\s*=\s*3", text) and pkv._PROB_DT[torch.float32] == 3


class OnDevice(torch.Tensor):
    """A stand-in that reports a CUDA device: the binding's checks run without one."""
    @property
    def is_cuda(self):
        return True

    @property
    def device(self):
        return torch.device("cuda", self._index)


def on(t, i=0):
    x = torch.Tensor._make_subclass(OnDevice, t)
    x._index = i
    return x


def test_binding_refuses_cpu_tensors_and_two_devices():
    h = lambda *s: torch.zeros(*s, dtype=torch.float16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    pool = h(4, 16, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_attention_prefill(h(3, 4, 64), h(3, 4, 64), pool, pool, i32(1, 2), i32(1), i32(2), max_seq_len=3)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_kv_gather(h(3, 2, 64), h(3, 2, 64), pool, pool, i32(1, 2), i32(1), i32(2))
    f = lambda *s: torch.zeros(*s)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.speculative_accept(torch.zeros(1, 3, dtype=torch.int64), i32(1), torch.zeros(1, 2, dtype=torch.int64), f(1, 3, 9),
                               f(1, 3))
    with pytest.raises(ValueError, match="more than one device"):
        pkv.paged_kv_gather(on(h(3, 2, 64)), on(h(3, 2, 64)), on(pool, 1), on(pool, 1), on(i32(1, 2)), on(i32(1)), on(i32(2)))


@pytest.fixture
def no_device(monkeypatch):
    """The shape checks of the binding alone: placement accepted, no device switched."""
    class Nothing:
        def __init__(self, *a):
            pass

        def __enter__(self):
            return self

        def __exit__(self, *a):
            return False
    monkeypatch.setattr(torch.cuda, "device", Nothing)


def test_binding_checks_shapes_and_types(no_device):
    h = lambda *s: on(torch.zeros(*s, dtype=torch.float16))
    i32 = lambda *s: on(torch.zeros(*s, dtype=torch.int32))
    i64 = lambda *s: on(torch.zeros(*s, dtype=torch.int64))
    f = lambda *s: on(torch.zeros(*s))
    pool = h(4, 16, 2, 64)

    def prefill(out=h(3, 4, 64), q=h(3, 4, 64), k=pool, v=pool, tables=i32(1, 2), lens=i32(1), starts=i32(2), **kw):
        pkv.paged_attention_prefill(out, q, k, v, tables, lens, starts, max_seq_len=3, **kw)

    for kw in (dict(q=h(3, 4, 32)), dict(out=h(2, 4, 64)), dict(q=h(3, 1, 4, 64)), dict(v=h(5, 16, 2, 64)),
               dict(tables=i32(2, 2)), dict(starts=i32(3)), dict(starts=i64(2)), dict(lens=i64(1)), dict(planned=True),
               dict(q=f(3, 4, 64)), dict(tables=i32(2))):
        with pytest.raises(ValueError):
            prefill(**kw)
    with pytest.raises(ValueError):                      # E4M3 pools need their scales
        pool8 = on(torch.zeros(4, 16, 2, 128, dtype=torch.uint8))
        pkv.paged_attention_prefill(h(3, 4, 128), h(3, 4, 128), pool8, pool8, i32(1, 2), i32(1), i32(2), max_seq_len=3,
                                    workspace=i32(4))

    def gather(k=h(3, 2, 64), v=h(3, 2, 64), pool=pool, tables=i32(1, 2), lens=i32(1), starts=i32(2)):
        pkv.paged_kv_gather(k, v, pool, pool, tables, lens, starts)

    for kw in (dict(k=h(3, 2, 32)), dict(v=h(4, 2, 64)), dict(k=f(3, 2, 64)), dict(starts=i32(3)), dict(tables=i32(2, 2)),
               dict(lens=i64(1))):
        with pytest.raises(ValueError):
            gather(**kw)

    def accept(tokens=i64(2, 4), acc=i32(2), drafts=i64(2, 3), target=f(2, 4, 9), uniform=f(2, 4), **kw):
        pkv.speculative_accept(tokens, acc, drafts, target, uniform, **kw)

    for kw in (dict(tokens=i64(2, 3)), dict(acc=i32(3)), dict(target=f(2, 3, 9)), dict(uniform=f(2, 3)),
               dict(drafts=i32(2, 3)), dict(draft_probs=f(2, 4, 9)), dict(draft_probs=h(2, 3, 9)), dict(num_drafts=i32(3)),
               dict(num_drafts=i64(2)), dict(uniform=h(2, 4))):
        with pytest.raises(ValueError):
            accept(**kw)


def test_scales_are_refused_over_16_bit_pools(no_device):
    h = lambda *s: on(torch.zeros(*s, dtype=torch.float16))
    i32 = lambda *s: on(torch.zeros(*s, dtype=torch.int32))
    pool, scale = h(4, 16, 2, 64), on(torch.ones(2))
    for kw in (dict(k_scale=scale), dict(v_scale=scale), dict(k_scale=scale, v_scale=scale)):
        with pytest.raises(ValueError, match="E4M3"):
            pkv.paged_attention_prefill(h(3, 4, 64), h(3, 4, 64), pool, pool, i32(1, 2), i32(1), i32(2), max_seq_len=3, **kw)
        with pytest.raises(ValueError, match="E4M3"):
            pkv.paged_kv_gather(h(3, 2, 64), h(3, 2, 64), pool, pool, i32(1, 2), i32(1), i32(2), **kw)
