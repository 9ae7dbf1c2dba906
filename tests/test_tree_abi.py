"""Host-side validation of the rotated append and of the tree calls: bad arguments are refused before any CUDA call, empty
work is accepted without touching the device, and the binding checks shapes and types.  No GPU."""
import ctypes
import os
import re

import pytest
import torch

import paged_kv_cache_156_gb300 as pkv
from paged_kv_cache_156_gb300 import _build
from test_prefill_abi import no_device, on  # noqa: F401  (a fixture, and stand-ins that report a CUDA device)

null = ctypes.c_void_p(0)
fake = ctypes.c_void_p(256)             # a non-null, aligned address that nothing dereferences
odd = ctypes.c_void_p(258)
half = ctypes.c_void_p(264)             # 8-byte aligned


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkv.load()


def test_header_and_binding_agree_on_the_tree_limit():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "pkv.h")).read()
    assert int(re.search(r"#define\s+PKV_TREE_MAX_NODES\s+(\d+)", text).group(1)) == pkv.TREE_MAX_NODES == 64


def test_append_rotary_refusals(lib):
    def call(q_out=fake, q=ctypes.c_void_p(512), kv=fake, pool=fake, slots=fake, pos=fake, cs=fake, T=3, qos=1024, qs=1024,
             ks=256, vs=256, P=100, r=128, il=0, nb=10, bs=16, Hq=8, Hkv=2, d=128, dt=1, kvdt=1, scale=null):
        return lib.pkv_paged_kv_append_rotary(q_out, q, kv, kv, pool, pool, slots, pos, cs, T, qos, qs, ks, vs, P, r, il, nb,
                                              bs, Hq, Hkv, d, dt, kvdt, scale, scale, null)

    for kw in (dict(dt=2), dict(dt=3), dict(dt=7), dict(kvdt=0), dict(kvdt=3), dict(dt=0)):
        assert call(**kw) == pkv.PKV_ERR_UNSUPPORTED, kw
    for kw in (dict(T=-1), dict(T=1 << 31), dict(P=0), dict(P=-5), dict(r=0), dict(r=-16), dict(r=24), dict(r=144), dict(d=0),
               dict(d=120, r=112), dict(d=4112, r=16), dict(Hq=-1), dict(Hq=4097), dict(Hkv=0), dict(Hkv=4097), dict(nb=0),
               dict(bs=0), dict(qos=1016), dict(qs=1020), dict(qs=0), dict(qos=-1024), dict(ks=248), dict(vs=260),
               dict(q_out=null), dict(q=null), dict(kv=null), dict(pool=null), dict(slots=null), dict(pos=null), dict(cs=null),
               dict(q_out=half), dict(kv=half), dict(pool=half), dict(slots=ctypes.c_void_p(260)), dict(pos=odd), dict(cs=half),
               dict(q=fake, qs=2048), dict(kvdt=2), dict(kvdt=2, scale=odd), dict(kvdt=2, scale=fake, pool=ctypes.c_void_p(260))):
        assert call(**kw) == pkv.PKV_ERR_INVALID, kw
    assert call(T=0) == pkv.PKV_OK and call(T=0, q=null, q_out=null, Hq=0, qs=0, qos=0) == pkv.PKV_OK
    assert call(T=0, kv=null, pool=null) == pkv.PKV_OK


def test_tree_attention_refusals(lib):
    def call(ptr=fake, B=2, T=10, max_len=40, Hq=8, Hkv=2, d=128, bs=16, nb=10, scale=1.0, dt=0, kvdt=0, ws=null, ws_bytes=0,
             planned=0, width=4, starts=fake, lens=fake, mask=fake, ks=null, vs=null, tables=fake):
        return lib.pkv_paged_attention_tree(ptr, ptr, ptr, ptr, tables, width, lens, starts, mask, B, T, max_len, Hq, Hkv, d, bs,
                                            nb, scale, dt, kvdt, ks, vs, ws, ws_bytes, planned, null), lib.pkv_last_error()

    ok_ws = dict(ws=fake, ws_bytes=1 << 40)
    for kw, status, word in (
            (dict(d=96), pkv.PKV_ERR_UNSUPPORTED, b"head_dim"), (dict(bs=12), pkv.PKV_ERR_UNSUPPORTED, b"block_size"),
            (dict(dt=2, kvdt=2, ks=fake, vs=fake), pkv.PKV_ERR_UNSUPPORTED, b"dtype"), (dict(dt=3, kvdt=3), pkv.PKV_ERR_UNSUPPORTED, b"dtype"),
            (dict(kvdt=1), pkv.PKV_ERR_UNSUPPORTED, b"kv_dt"), (dict(kvdt=3), pkv.PKV_ERR_UNSUPPORTED, b"kv_dt"),
            (dict(kvdt=2), pkv.PKV_ERR_INVALID, b"k_scale"), (dict(kvdt=2, ks=fake), pkv.PKV_ERR_INVALID, b"k_scale"),
            (dict(kvdt=2, ks=odd, vs=fake), pkv.PKV_ERR_INVALID, b"aligned"),
            (dict(kvdt=2, ks=fake, vs=fake, d=64), pkv.PKV_ERR_UNSUPPORTED, b"128"),
            (dict(mask=null), pkv.PKV_ERR_INVALID, b"tree_mask"), (dict(mask=ctypes.c_void_p(260)), pkv.PKV_ERR_INVALID, b"tree_mask"),
            (dict(Hq=7), pkv.PKV_ERR_INVALID, b"num_heads"), (dict(B=-1), pkv.PKV_ERR_INVALID, b"num_seqs"),
            (dict(T=-1), pkv.PKV_ERR_INVALID, b"num_tokens"), (dict(T=1 << 27), pkv.PKV_ERR_INVALID, b"num_tokens"),
            (dict(max_len=65), pkv.PKV_ERR_INVALID, b"max_seq_len"), (dict(nb=0), pkv.PKV_ERR_INVALID, b"num_blocks"),
            (dict(scale=float("nan")), pkv.PKV_ERR_INVALID, b"scale"), (dict(planned=2), pkv.PKV_ERR_INVALID, b"planned"),
            (dict(starts=null), pkv.PKV_ERR_INVALID, b"null"), (dict(lens=odd), pkv.PKV_ERR_INVALID, b"aligned"),
            (dict(), pkv.PKV_ERR_WORKSPACE, b"workspace"), (dict(ws=odd, ws_bytes=1 << 40), pkv.PKV_ERR_WORKSPACE, b"workspace"),
            (dict(ptr=null, **ok_ws), pkv.PKV_ERR_INVALID, b"null"), (dict(tables=null, **ok_ws), pkv.PKV_ERR_INVALID, b"null"),
            (dict(ptr=half, **ok_ws), pkv.PKV_ERR_INVALID, b"16-byte")):
        st, msg = call(**kw)
        assert st == status and word in msg, (kw, st, msg)
    assert call(B=0)[0] == pkv.PKV_OK and call(T=0)[0] == pkv.PKV_OK and call(T=0, mask=null)[0] == pkv.PKV_OK


def test_accept_tree_refusals(lib):
    def call(tokens=fake, path=fake, count=fake, drafts=fake, parents=fake, starts=fake, probs=fake, uniform=fake, B=2, T=9, W=4,
             V=100, dt=3):
        return lib.pkv_speculative_accept_tree(tokens, path, count, drafts, parents, starts, probs, uniform, B, T, W, V, dt, null)

    assert call(dt=2) == pkv.PKV_ERR_UNSUPPORTED and call(dt=4) == pkv.PKV_ERR_UNSUPPORTED
    for kw in (dict(B=-1), dict(B=(1 << 24) + 1), dict(T=-1), dict(T=1 << 31), dict(W=0), dict(W=1025), dict(W=-1), dict(V=0),
               dict(V=pkv.ACCEPT_MAX_VOCAB + 1), dict(tokens=null), dict(path=null), dict(count=null), dict(drafts=null),
               dict(parents=null), dict(starts=null), dict(probs=null), dict(uniform=null), dict(tokens=ctypes.c_void_p(260)),
               dict(drafts=ctypes.c_void_p(260)), dict(path=odd), dict(count=odd), dict(parents=odd), dict(starts=odd),
               dict(uniform=odd), dict(probs=odd), dict(probs=ctypes.c_void_p(257), dt=1)):
        assert call(**kw) == pkv.PKV_ERR_INVALID, kw
    assert call(B=0) == pkv.PKV_OK


def test_keep_path_refusals(lib):
    def call(layers=2, pool=fake, tables=fake, width=4, lens=fake, starts=fake, path=fake, count=fake, B=2, W=4, nb=10, bs=16,
             Hkv=2, d=64, dt=0, arr=True):
        ptrs = (ctypes.c_void_p * max(layers, 1))(*[fake] * max(layers - 1, 0), pool)
        return lib.pkv_paged_kv_keep_path(ptrs if arr else None, ptrs, layers, tables, width, lens, starts, path, count, B, W, nb,
                                          bs, Hkv, d, dt, null)

    assert call(dt=3) == pkv.PKV_ERR_UNSUPPORTED
    for kw in (dict(layers=-1), dict(B=-1), dict(W=0), dict(W=1025), dict(nb=0), dict(bs=0), dict(Hkv=0), dict(d=0), dict(d=3, Hkv=1),
               dict(d=8, Hkv=1, dt=2), dict(width=-1), dict(pool=null), dict(pool=half), dict(tables=null), dict(lens=null),
               dict(starts=null), dict(path=null), dict(count=null), dict(tables=odd), dict(lens=odd), dict(starts=odd),
               dict(path=odd), dict(count=odd), dict(arr=False), dict(Hkv=1 << 15, d=1 << 15)):
        assert call(**kw) == pkv.PKV_ERR_INVALID, kw
    assert call(B=0) == pkv.PKV_OK and call(layers=0) == pkv.PKV_OK


def test_binding_refuses_cpu_tensors_and_two_devices():
    h = lambda *s: torch.zeros(*s, dtype=torch.float16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    i64 = lambda *s: torch.zeros(*s, dtype=torch.int64)
    f = lambda *s: torch.zeros(*s)
    pool = h(4, 16, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_kv_append_rotary(h(3, 4, 64), h(3, 4, 64), h(3, 2, 64), h(3, 2, 64), pool, pool, i64(3), i32(3), f(9, 64))
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_attention_tree(h(3, 4, 64), h(3, 4, 64), pool, pool, i32(1, 2), i32(1), i32(2), i64(3), max_seq_len=3)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.speculative_accept_tree(i64(1, 3), i32(1, 3), i32(1), i64(4), i32(4), i32(2), f(4, 9), f(4))
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_kv_keep_path(pool, pool, i32(1, 2), i32(1), i32(2), i32(1, 3), i32(1))
    with pytest.raises(ValueError, match="more than one device"):
        pkv.paged_kv_append_rotary(on(h(3, 4, 64)), on(h(3, 4, 64)), on(h(3, 2, 64)), on(h(3, 2, 64)), on(pool, 1), on(pool, 1),
                                   on(i64(3)), on(i32(3)), on(f(9, 64)))
    with pytest.raises(ValueError, match="more than one device"):
        pkv.paged_attention_tree(on(h(3, 4, 64)), on(h(3, 4, 64)), on(pool), on(pool), on(i32(1, 2)), on(i32(1)), on(i32(2)),
                                 on(i64(3), 1), max_seq_len=3)
    with pytest.raises(ValueError, match="more than one device"):
        pkv.speculative_accept_tree(on(i64(1, 3)), on(i32(1, 3)), on(i32(1)), on(i64(4)), on(i32(4)), on(i32(2)), on(f(4, 9)),
                                    on(f(4), 1))
    with pytest.raises(ValueError, match="more than one device"):
        pkv.paged_kv_keep_path([on(pool)], [on(pool, 1)], on(i32(1, 2)), on(i32(1)), on(i32(2)), on(i32(1, 3)), on(i32(1)))


def test_binding_checks_shapes_and_types(no_device):  # noqa: F811
    h = lambda *s: on(torch.zeros(*s, dtype=torch.float16))
    b16 = lambda *s: on(torch.zeros(*s, dtype=torch.bfloat16))
    u8 = lambda *s: on(torch.zeros(*s, dtype=torch.uint8))
    i32 = lambda *s: on(torch.zeros(*s, dtype=torch.int32))
    i64 = lambda *s: on(torch.zeros(*s, dtype=torch.int64))
    f = lambda *s: on(torch.zeros(*s))
    pool = h(4, 16, 2, 64)

    def append(q_out=h(3, 4, 64), q=h(3, 4, 64), k=h(3, 2, 64), v=h(3, 2, 64), kc=pool, vc=pool, slots=i64(3), pos=i32(3),
               cs=f(9, 64), **kw):
        pkv.paged_kv_append_rotary(q_out, q, k, v, kc, vc, slots, pos, cs, **kw)

    wide = torch.zeros(3, 4, 128, dtype=torch.float16)
    for kw in (dict(q=None), dict(q_out=None), dict(q=h(2, 4, 64)), dict(q_out=h(3, 3, 64)), dict(q=b16(3, 4, 64)),
               dict(k=h(3, 3, 64)), dict(k=h(3, 2, 32)), dict(v=h(4, 2, 64)), dict(v=b16(3, 2, 64)), dict(k=b16(3, 2, 64)),
               dict(k=h(3, 128)), dict(q=on(wide[:, :, :64])), dict(q=on(wide[:, :, ::2])), dict(vc=h(5, 16, 2, 64)), dict(slots=i32(3)),
               dict(slots=i64(2)), dict(pos=i64(3)), dict(pos=i32(4)), dict(cs=h(9, 64)), dict(cs=f(64)),
               dict(k_scale=f(2)), dict(kc=u8(4, 16, 2, 64), vc=u8(4, 16, 2, 64)),
               dict(kc=u8(4, 16, 2, 64), vc=u8(4, 16, 2, 64), k_scale=f(3), v_scale=f(2)), dict(q=3, q_out=4)):
        with pytest.raises(ValueError):
            append(**kw)

    def attend(out=h(3, 4, 64), q=h(3, 4, 64), k=pool, v=pool, tables=i32(1, 2), lens=i32(1), starts=i32(2), mask=i64(3), **kw):
        pkv.paged_attention_tree(out, q, k, v, tables, lens, starts, mask, max_seq_len=3, **kw)

    for kw in (dict(q=h(3, 4, 32)), dict(out=h(2, 4, 64)), dict(q=h(3, 1, 4, 64)), dict(v=h(5, 16, 2, 64)), dict(tables=i32(2, 2)),
               dict(starts=i32(3)), dict(starts=i64(2)), dict(lens=i64(1)), dict(planned=True), dict(q=f(3, 4, 64)),
               dict(mask=i32(3)), dict(mask=i64(4)), dict(mask=i64(3, 1)), dict(k_scale=f(2)),
               dict(k=u8(4, 16, 2, 64), v=u8(4, 16, 2, 64), workspace=i32(4))):
        with pytest.raises(ValueError):
            attend(**kw)

    def accept(tokens=i64(2, 4), path=i32(2, 4), count=i32(2), drafts=i64(7), parents=i32(7), starts=i32(3), probs=f(7, 9),
               uniform=f(7)):
        pkv.speculative_accept_tree(tokens, path, count, drafts, parents, starts, probs, uniform)

    for kw in (dict(tokens=i32(2, 4)), dict(path=i32(2, 3)), dict(path=i64(2, 4)), dict(count=i32(3)), dict(drafts=i64(6)),
               dict(drafts=i32(7)), dict(parents=i64(7)), dict(parents=i32(8)), dict(starts=i32(2)), dict(probs=f(6, 9)),
               dict(probs=i32(7, 9)), dict(uniform=f(8)), dict(uniform=h(7))):
        with pytest.raises(ValueError):
            accept(**kw)

    def keep(k=[pool, pool], v=[pool, pool], tables=i32(2, 3), lens=i32(2), starts=i32(3), path=i32(2, 4), count=i32(2)):
        pkv.paged_kv_keep_path(k, v, tables, lens, starts, path, count)

    for kw in (dict(k=[pool]), dict(k=[], v=[]), dict(v=[pool, h(5, 16, 2, 64)]), dict(v=[pool, b16(4, 16, 2, 64)]),
               dict(tables=i32(3, 3)), dict(tables=i64(2, 3)), dict(lens=i32(3)), dict(starts=i32(2)), dict(path=i32(8)),
               dict(path=i64(2, 4)), dict(count=i32(1)), dict(count=i64(2))):
        with pytest.raises(ValueError):
            keep(**kw)
