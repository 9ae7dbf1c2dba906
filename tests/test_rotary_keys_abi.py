"""A rotated append of keys and values alone: with num_heads 0 the query pointers are not looked at, whatever they are."""
import ctypes

import pytest
import torch

import paged_kv_cache_156_gb300 as pkv
from paged_kv_cache_156_gb300 import _build

null = ctypes.c_void_p(0)
fake = ctypes.c_void_p(256)             # a non-null, aligned address that nothing dereferences


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkv.load()


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up: nothing may be launched with them")
@pytest.mark.parametrize("addr", [1, 2, 8, 258, 264])
def test_query_pointers_are_ignored_without_heads(lib, addr):
    def call(q_out, q, heads=0, stride=0, kv=fake):
        return lib.pkv_paged_kv_append_rotary(q_out, q, kv, kv, fake, fake, fake, fake, fake, 3, stride, stride, 256, 256, 100,
                                              128, 0, 10, 16, heads, 2, 128, 1, 1, null, null, null)

    at = ctypes.c_void_p(addr)
    for q_out, q in ((at, fake), (fake, at), (at, at), (null, at), (at, null), (null, null)):
        assert call(q_out, q) == pkv.PKV_ERR_CUDA             # past every check: there is no device to launch on
    assert call(at, at, kv=at) == pkv.PKV_ERR_INVALID         # keys and values are looked at all the same
    for q_out, q in ((at, fake), (fake, at)):
        assert call(q_out, q, heads=1, stride=128) == pkv.PKV_ERR_INVALID


@pytest.mark.gpu
def test_keys_and_values_beside_odd_query_pointers(lib):
    T, Hkv, d, bs, P = 5, 2, 64, 16, 40
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(T, Hkv, d, generator=g).half().cuda() for _ in "kv")
    angles = torch.rand(P, d // 2, generator=g, dtype=torch.float64)
    cos_sin = torch.cat([angles.cos(), angles.sin()], 1).float().cuda()
    slots, pos = torch.tensor([3, 40, 17, -1, 5]).cuda(), torch.arange(T, dtype=torch.int32).cuda()
    junk = torch.full((64,), 7, dtype=torch.uint8, device="cuda")
    got, want = ([torch.zeros(4, bs, Hkv, d, dtype=torch.float16, device="cuda") for _ in "kv"] for _ in range(2))
    at = junk.data_ptr() + 1
    st = lib.pkv_paged_kv_append_rotary(at, at, k.data_ptr(), v.data_ptr(), got[0].data_ptr(), got[1].data_ptr(), slots.data_ptr(),
                                        pos.data_ptr(), cos_sin.data_ptr(), T, 0, 0, Hkv * d, Hkv * d, P, d, 0, 4, bs, 0, Hkv, d,
                                        0, 0, None, None, torch.cuda.current_stream().cuda_stream)
    assert st == pkv.PKV_OK, lib.pkv_last_error()
    pkv.paged_kv_append_rotary(None, None, k, v, *want, slots, pos, cos_sin)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and float(want[0].abs().sum()) > 0
    assert (junk == 7).all() and pkv.device_error(reset=True) == 0
