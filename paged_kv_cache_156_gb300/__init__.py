"""Python binding of the paged KV-cache decode library (``_lib/libpkv.so``).

Argument marshalling only: every function checks tensor placement (all of a
call's CUDA tensors on one device, made current for the call), dtype, shape
and contiguity, then passes raw device pointers and that device's current
CUDA stream to the C ABI declared in ``include/pkv.h``.  All work runs in the
library's CUDA kernels; there is no CPU path.  A missing library raises.

    paged_kv_append(k, v, key_cache, value_cache, slot_mapping)
    paged_attention_decode(out, q, key_cache, value_cache, block_tables, seq_lens, scale, ...)
    copy_blocks(key_caches, value_caches, src_dst_pairs)
"""
from __future__ import annotations

import array
import ctypes
import functools
import math
import operator
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libpkv.so")

PKV_OK, PKV_ERR_INVALID, PKV_ERR_UNSUPPORTED, PKV_ERR_WORKSPACE, PKV_ERR_CUDA, PKV_ERR_OOM = range(6)
_DT = {torch.float16: 0, torch.bfloat16: 1}
_POOL_DT = {torch.float16: 0, torch.bfloat16: 1, torch.uint8: 2}   # uint8 pools hold E4M3 codes
PLAN_MAX_SEQS = 1024        # PKV_PLAN_MAX_SEQS: batches up to this size run through the plan kernel
PLANNED = 1                 # PKV_PLANNED: run over the plan an earlier call wrote
_PROB_DT = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 3}   # PKV_F32: probabilities only
_HALF_DTS, _POOL_DTS, _PROB_DTS = tuple(_DT), tuple(_POOL_DT), tuple(_PROB_DT)
ACCEPT_MAX_VOCAB = 524288   # PKV_ACCEPT_MAX_VOCAB
TREE_MAX_NODES = 64         # PKV_TREE_MAX_NODES
INPUTS_READY = 2            # PKV_INPUTS_READY: nothing pending writes the pools, tables, lengths or plan

# every symbol include/pkv.h declares
ABI_SYMBOLS = ("pkv_version", "pkv_last_error", "pkv_paged_kv_append", "pkv_decode_workspace_bytes",
               "pkv_decode_partition_tokens", "pkv_decode_plan_partition_tokens", "pkv_paged_attention_decode", "pkv_copy_blocks", "pkv_device_error",
               "pkv_paged_attention_decode_static", "pkv_swap_blocks", "pkv_paged_attention_verify", "pkv_bm_create", "pkv_bm_destroy",
               "pkv_bm_num_free_blocks", "pkv_bm_seq_len", "pkv_bm_refcount", "pkv_bm_allocate", "pkv_bm_fork",
               "pkv_bm_free", "pkv_bm_append_slots", "pkv_bm_block_tables", "pkv_paged_kv_append_fp8",
               "pkv_paged_attention_decode_fp8", "pkv_decode_plan", "pkv_paged_attention_decode_planned",
               "pkv_paged_attention_decode_fp8_planned", "pkv_paged_kv_append_decode",
               "pkv_paged_attention_verify_fp8", "pkv_prefill_workspace_bytes", "pkv_prefill_plan",
               "pkv_paged_attention_prefill", "pkv_paged_attention_prefill_fp8", "pkv_paged_kv_gather",
               "pkv_paged_kv_gather_fp8", "pkv_speculative_accept", "pkv_paged_kv_append_rotary",
               "pkv_paged_attention_tree", "pkv_speculative_accept_tree", "pkv_paged_kv_keep_path")

_lib = None


class PkvError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"pkv status {status}: {message}")
        self.status = status


def load() -> ctypes.CDLL:
    """Load the built library (build it with ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run `python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(LIB_PATH)
    c_i, c_i64, c_p, c_sz, c_f = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
    lib.pkv_version.restype = c_i
    lib.pkv_version.argtypes = []
    lib.pkv_last_error.restype = ctypes.c_char_p
    lib.pkv_last_error.argtypes = []
    lib.pkv_paged_kv_append.restype = c_i
    lib.pkv_paged_kv_append.argtypes = [c_p, c_p, c_p, c_p, c_p, c_i64, c_i64, c_i, c_i, c_i, c_i, c_p]
    lib.pkv_decode_workspace_bytes.restype = c_sz
    lib.pkv_decode_workspace_bytes.argtypes = [c_i, c_i, c_i, c_i, c_i, c_i]
    lib.pkv_decode_partition_tokens.restype = c_i
    lib.pkv_decode_partition_tokens.argtypes = [c_i, c_i, c_i, c_i, c_i]
    lib.pkv_decode_plan_partition_tokens.restype = c_i
    lib.pkv_decode_plan_partition_tokens.argtypes = [c_p, c_i, c_i, c_i, c_p]
    lib.pkv_paged_attention_decode.restype = c_i
    lib.pkv_paged_attention_decode.argtypes = [c_p, c_p, c_p, c_p, c_p, c_i, c_p, c_i, c_i, c_i, c_i, c_i, c_i,
                                               c_i64, c_f, c_i, c_p, c_sz, c_i, c_p]
    lib.pkv_paged_attention_verify.restype = c_i
    lib.pkv_paged_attention_verify.argtypes = [c_p, c_p, c_p, c_p, c_p, c_i, c_p, c_i, c_i, c_i64, c_i, c_i, c_i,
                                               c_i, c_i64, c_f, c_i, c_i, c_p, c_sz, c_i, c_p]
    lib.pkv_paged_kv_append_fp8.restype = c_i
    lib.pkv_paged_kv_append_fp8.argtypes = [c_p, c_p, c_p, c_p, c_p, c_i64, c_i64, c_i, c_i, c_i, c_i, c_p, c_p, c_p]
    lib.pkv_paged_attention_decode_fp8.restype = c_i
    lib.pkv_paged_attention_decode_fp8.argtypes = [c_p, c_p, c_p, c_p, c_p, c_i, c_p, c_i, c_i, c_i, c_i, c_i, c_i,
                                                   c_i64, c_f, c_i, c_p, c_p, c_p, c_sz, c_i, c_p]
    lib.pkv_paged_attention_decode_fp8_planned.restype = c_i
    lib.pkv_paged_attention_decode_fp8_planned.argtypes = [c_p, c_p, c_p, c_p, c_p, c_i, c_p, c_i, c_i, c_i64, c_i,
                                                           c_i, c_i, c_i, c_i64, c_f, c_i, c_p, c_p, c_p, c_sz, c_i,
                                                           c_p]
    lib.pkv_paged_attention_decode_planned.restype = c_i
    lib.pkv_paged_attention_decode_planned.argtypes = [c_p, c_p, c_p, c_p, c_p, c_i, c_p, c_i, c_i, c_i64, c_i, c_i,
                                                       c_i, c_i, c_i64, c_f, c_i, c_p, c_sz, c_i, c_p]
    lib.pkv_paged_attention_verify_fp8.restype = c_i
    lib.pkv_paged_attention_verify_fp8.argtypes = [c_p, c_p, c_p, c_p, c_p, c_i, c_p, c_i, c_i, c_i64, c_i, c_i, c_i,
                                                   c_i, c_i64, c_f, c_i, c_p, c_p, c_i, c_p, c_sz, c_i, c_p]
    lib.pkv_paged_kv_append_decode.restype = c_i
    lib.pkv_paged_kv_append_decode.argtypes = [c_p, c_p, c_p, c_p, c_p, c_p, c_p, c_p, c_i, c_p, c_i, c_i, c_i64, c_i,
                                               c_i, c_i, c_i, c_i64, c_f, c_i, c_i, c_p, c_p, c_p, c_sz, c_i, c_i, c_p]
    lib.pkv_decode_plan.restype = c_i
    lib.pkv_decode_plan.argtypes = [c_p, c_i, c_p, c_i, c_i, c_i64, c_i, c_i, c_i, c_i, c_i, c_p, c_sz, c_i, c_p]
    lib.pkv_prefill_workspace_bytes.restype = c_sz
    lib.pkv_prefill_workspace_bytes.argtypes = [c_i, c_i64, c_i, c_i, c_i]
    lib.pkv_prefill_plan.restype = c_i
    lib.pkv_prefill_plan.argtypes = [c_p, c_p, c_i, c_i64, c_i, c_i, c_i, c_i, c_p, c_sz, c_p]
    lib.pkv_paged_attention_prefill.restype = c_i
    lib.pkv_paged_attention_prefill.argtypes = [c_p, c_p, c_p, c_p, c_p, c_i, c_p, c_p, c_i, c_i64, c_i, c_i, c_i, c_i,
                                                c_i, c_i64, c_f, c_i, c_p, c_sz, c_i, c_p]
    lib.pkv_paged_attention_prefill_fp8.restype = c_i
    lib.pkv_paged_attention_prefill_fp8.argtypes = [c_p, c_p, c_p, c_p, c_p, c_i, c_p, c_p, c_i, c_i64, c_i, c_i, c_i,
                                                    c_i, c_i, c_i64, c_f, c_i, c_p, c_p, c_p, c_sz, c_i, c_p]
    lib.pkv_paged_kv_gather.restype = c_i
    lib.pkv_paged_kv_gather.argtypes = [c_p, c_p, c_p, c_p, c_p, c_i, c_p, c_p, c_i, c_i64, c_i64, c_i, c_i, c_i, c_i,
                                        c_p]
    lib.pkv_paged_kv_gather_fp8.restype = c_i
    lib.pkv_paged_kv_gather_fp8.argtypes = [c_p, c_p, c_p, c_p, c_p, c_i, c_p, c_p, c_i, c_i64, c_i64, c_i, c_i, c_i,
                                            c_i, c_p, c_p, c_p]
    lib.pkv_speculative_accept.restype = c_i
    lib.pkv_speculative_accept.argtypes = [c_p, c_p, c_p, c_p, c_p, c_p, c_p, c_i, c_i, c_i64, c_i, c_p]
    lib.pkv_paged_kv_append_rotary.restype = c_i
    lib.pkv_paged_kv_append_rotary.argtypes = [c_p] * 9 + [c_i64] * 5 + [c_i, c_i, c_i, c_i64, c_i, c_i, c_i, c_i, c_i, c_i,
                                                                         c_p, c_p, c_p]
    lib.pkv_paged_attention_tree.restype = c_i
    lib.pkv_paged_attention_tree.argtypes = [c_p, c_p, c_p, c_p, c_p, c_i, c_p, c_p, c_p, c_i, c_i64, c_i, c_i, c_i, c_i, c_i,
                                             c_i64, c_f, c_i, c_i, c_p, c_p, c_p, c_sz, c_i, c_p]
    lib.pkv_speculative_accept_tree.restype = c_i
    lib.pkv_speculative_accept_tree.argtypes = [c_p] * 8 + [c_i, c_i64, c_i, c_i64, c_i, c_p]
    lib.pkv_paged_kv_keep_path.restype = c_i
    lib.pkv_paged_kv_keep_path.argtypes = [c_p, c_p, c_i, c_p, c_i, c_p, c_p, c_p, c_p, c_i,
                                           c_i, c_i64, c_i, c_i, c_i, c_i, c_p]
    lib.pkv_copy_blocks.restype = c_i
    lib.pkv_copy_blocks.argtypes = [ctypes.POINTER(c_p), ctypes.POINTER(c_p), c_i, c_p, c_i64, c_i64, c_i, c_i,
                                    c_i, c_i, c_p]
    lib.pkv_device_error.restype = c_i
    lib.pkv_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint), c_i]
    lib.pkv_swap_blocks.restype = c_i
    lib.pkv_swap_blocks.argtypes = [ctypes.POINTER(c_p)] * 4 + [c_i, c_p, c_i64, c_i64, c_i64, c_i, c_i, c_i, c_i, c_p]
    lib.pkv_bm_create.restype = c_p
    lib.pkv_bm_create.argtypes = [c_i64, c_i, c_p]
    lib.pkv_bm_destroy.restype = None
    lib.pkv_bm_destroy.argtypes = [c_p]
    lib.pkv_bm_num_free_blocks.restype = c_i64
    lib.pkv_bm_num_free_blocks.argtypes = [c_p]
    lib.pkv_bm_seq_len.restype = c_i64
    lib.pkv_bm_seq_len.argtypes = [c_p, c_i64]
    lib.pkv_bm_refcount.restype = c_i
    lib.pkv_bm_refcount.argtypes = [c_p, c_i64]
    for name, args in (("pkv_bm_allocate", [c_p, c_i64, c_i64]), ("pkv_bm_fork", [c_p, c_i64, c_i64]),
                       ("pkv_bm_free", [c_p, c_i64]),
                       ("pkv_bm_append_slots", [c_p, c_p, c_i64, c_p, c_p, c_i64, c_p]),
                       ("pkv_bm_block_tables", [c_p, c_p, c_i64, c_p, c_i, ctypes.c_int32, c_p])):
        getattr(lib, name).restype = c_i
        getattr(lib, name).argtypes = args
    lib.pkv_paged_attention_decode_static.restype = c_i
    lib.pkv_paged_attention_decode_static.argtypes = [c_p, c_p, c_p, c_p, c_p, c_i, c_p, c_i, c_i, c_i, c_i, c_i, c_i,
                                                      c_i64, c_f, c_i, c_i, c_p]
    _lib = lib
    return lib


def _check(status: int):
    if status != PKV_OK:
        raise PkvError(status, load().pkv_last_error().decode(errors="replace"))


_Tensor = torch.Tensor
_NESTED = (list, tuple, torch.Tensor)


def _current_device() -> int:
    return torch._C._cuda_getDevice()


def _cuda_devices(values):
    """The CUDA devices of the tensors among ``values`` (tensors, or lists / tuples of them)."""
    devs = set()
    for v in values:
        for t in (v if isinstance(v, (list, tuple)) else (v,)):
            if isinstance(t, torch.Tensor) and t.is_cuda:
                devs.add(t.device)
    return devs


def _one_device(fn):
    """Every CUDA tensor of the call on one device, and that device current while
    the library runs: the kernels launch on the current device, on the stream of
    the tensors' device, and dereference every pointer there."""
    @functools.wraps(fn)
    def call(*args, **kwargs):
        # the usual call: plain tensors of the current device
        dev = None
        for v in (*args, *kwargs.values()) if kwargs else args:
            if type(v) is _Tensor:
                d = v.get_device()
                if d != dev and d >= 0:
                    if dev is not None:
                        break
                    dev = d
            elif v is not None and isinstance(v, _NESTED):
                break
        else:
            # (a CUDA tensor exists: the runtime is up, and the raw call answers in a tenth of the public one's time)
            if dev is None or dev == _current_device():
                return fn(*args, **kwargs)
        devs = _cuda_devices(list(args) + list(kwargs.values()))
        if len(devs) > 1:
            raise ValueError(f"{fn.__name__}: tensors on more than one device: {sorted(str(d) for d in devs)}")
        if not devs:
            return fn(*args, **kwargs)
        with torch.cuda.device(devs.pop()):
            return fn(*args, **kwargs)
    return call


def _stream(t: torch.Tensor):
    # (the raw handle: building the Stream object costs 2 us of a call)
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _cuda(name, t, dtype=None, ndim=None):
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype is not dtype and (type(dtype) is not tuple or t.dtype not in dtype):
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    return t.data_ptr()


def _usual(*tensors) -> bool:
    """Plain contiguous tensors of the current device.  The calls below take such arguments without the checks that
    name what is wrong (which cost a third of a small call's host time); whatever else they meet goes through those."""
    dev = tensors[0].get_device() if type(tensors[0]) is _Tensor else -1
    if dev < 0:
        return False
    for t in tensors:
        if type(t) is not _Tensor or t.get_device() != dev or not t.is_contiguous():
            return False
    return dev == _current_device()


def _pool(name, c, dtypes=(torch.float16, torch.bfloat16)):
    _cuda(name, c, dtypes, 4)
    return c.shape  # num_blocks, block_size, num_kv_heads, head_dim


@_one_device
def paged_kv_append(k, v, key_cache, value_cache, slot_mapping) -> None:
    """Write k[t], v[t] ([T, Hkv, d]) into slot slot_mapping[t] (int64; < 0 = skip)."""
    NB, bs, Hkv, d = _pool("key_cache", key_cache)
    if value_cache.shape != key_cache.shape or value_cache.dtype != key_cache.dtype:
        raise ValueError("value_cache must match key_cache")
    args = [_cuda("k", k, key_cache.dtype, 3), _cuda("v", v, key_cache.dtype, 3), _cuda("key_cache", key_cache),
            _cuda("value_cache", value_cache), _cuda("slot_mapping", slot_mapping, torch.int64, 1)]
    T = k.shape[0]
    if tuple(k.shape) != (T, Hkv, d) or tuple(v.shape) != (T, Hkv, d) or slot_mapping.shape[0] != T:
        raise ValueError("k, v must be [T, num_kv_heads, head_dim] and slot_mapping [T]")
    _check(load().pkv_paged_kv_append(*args, T, NB, bs, Hkv, d, _DT[key_cache.dtype], _stream(key_cache)))


def _rows_stride(name, t, dtypes, heads, dim):
    """Rows of [heads, dim] whose elements are dense, a stride of elements apart (views of a packed projection)."""
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtypes}")
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim:
        raise ValueError(f"{name} must be [num_tokens, {heads}, {dim}], got {tuple(t.shape)}")
    if (dim > 1 and t.stride(2) != 1) or (heads > 1 and t.stride(1) != dim):
        raise ValueError(f"{name}: a token's row must be dense")
    return t.stride(0) if t.shape[0] > 1 else heads * dim


def paged_kv_append_rotary(q_out, q, k, v, key_cache, value_cache, slot_mapping, positions, cos_sin, interleaved=False,
                           k_scale=None, v_scale=None) -> None:
    """paged_kv_append with the position rotation on the way: q_out = q turned, and K = k turned, V = v in the caches.

    q_out, q [T, Hq, d] (q_out may be q; both None: no queries), k, v [T, Hkv, d]: rows may be a stride apart (views of a
    packed projection), a multiple of 8 elements.  slot_mapping int64 [T] (< 0: nothing is cached).  positions int32 [T];
    cos_sin float32 [P, r]: row p holds the cosines, then the sines, of position p's r / 2 angles.  A head's first r
    elements turn, as pairs (i, i + r / 2), or (2 i, 2 i + 1) when ``interleaved``.  uint8 pools hold E4M3 codes and take
    k_scale / v_scale (float32 [Hkv]) as paged_kv_append_fp8 does."""
    if _usual(key_cache, value_cache, slot_mapping, positions, cos_sin) and type(k) is _Tensor:
        dev, dt, pool, kdt = key_cache.get_device(), key_cache.dtype, key_cache.shape, k.dtype
        kv8 = dt is torch.uint8
        T, h, d = k.shape if k.dim() == 3 else (0, 0, 0)
        if T > 0 and type(v) is type(q) is type(q_out) is _Tensor and len(pool) == 4 and pool[2] == h and \
                pool[3] == d and k.get_device() == v.get_device() == q.get_device() == q_out.get_device() == dev and \
                (kv8 or dt is kdt) and v.dtype is q.dtype is q_out.dtype is kdt and kdt in _DT and value_cache.dtype is dt and \
                value_cache.shape == pool and v.shape == (T, h, d) and slot_mapping.dtype is torch.int64 and \
                positions.dtype is torch.int32 and cos_sin.dtype is torch.float32 and cos_sin.dim() == 2 and \
                slot_mapping.shape == positions.shape == (T,) and \
                (k_scale is None and v_scale is None if not kv8 else _usual(key_cache, k_scale, v_scale) and
                 k_scale.dtype is v_scale.dtype is torch.float32 and k_scale.shape == v_scale.shape == (h,)):
            rows = q.shape
            ks, vs, qs, os_ = k.stride(), v.stride(), q.stride(), q_out.stride()
            if len(rows) == 3 and rows[0] == T and rows[2] == d and q_out.shape == rows and \
                    ks[2] == vs[2] == qs[2] == os_[2] == 1 and ks[1] == vs[1] == qs[1] == os_[1] == d:
                return _check(load().pkv_paged_kv_append_rotary(
                    q_out.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(),
                    slot_mapping.data_ptr(), positions.data_ptr(), cos_sin.data_ptr(), T,
                    *((os_[0], qs[0], ks[0], vs[0]) if T > 1 else (rows[1] * d, rows[1] * d, h * d, h * d)), *cos_sin.shape,
                    1 if interleaved else 0, pool[0], pool[1], rows[1], h, d, _DT[kdt], _POOL_DT[dt],
                    k_scale.data_ptr() if kv8 else None, v_scale.data_ptr() if kv8 else None, _stream(key_cache)))
    _append_rotary(q_out, q, k, v, key_cache, value_cache, slot_mapping, positions, cos_sin, interleaved, k_scale, v_scale)


@_one_device
def _append_rotary(q_out, q, k, v, key_cache, value_cache, slot_mapping, positions, cos_sin, interleaved, k_scale,
                   v_scale) -> None:
    dt = key_cache.dtype
    kc = _cuda("key_cache", key_cache, _POOL_DTS, 4)
    kv8 = dt is torch.uint8
    NB, bs, Hkv, d = key_cache.shape
    if value_cache.shape != key_cache.shape or value_cache.dtype is not dt:
        raise ValueError("value_cache must match key_cache")
    if not kv8 and (k_scale is not None or v_scale is not None):
        raise ValueError("k_scale / v_scale belong to E4M3 (uint8) pools")
    ks = _rows_stride("k", k, _HALF_DTS if kv8 else (dt,), Hkv, d)
    T, own = k.shape[0], (k.dtype,)
    vs = _rows_stride("v", v, own, Hkv, d)
    Hq, qo, qi, qos, qis = 0, None, None, 0, 0
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    if q is not None:
        if not isinstance(q, _Tensor) or q.dim() != 3:
            raise ValueError("q must be a tensor [num_tokens, num_heads, head_dim]")
        Hq = q.shape[1]
        qis, qos = _rows_stride("q", q, own, Hq, d), _rows_stride("q_out", q_out, own, Hq, d)
        qo, qi = q_out.data_ptr(), q.data_ptr()
        if q.shape[0] != T or q_out.shape[0] != T:
            raise ValueError("q, q_out, k and v must have the same tokens")
    vc, sm = _cuda("value_cache", value_cache), _cuda("slot_mapping", slot_mapping, torch.int64, 1)
    ps, cs = _cuda("positions", positions, torch.int32, 1), _cuda("cos_sin", cos_sin, torch.float32, 2)
    if v.shape[0] != T or slot_mapping.shape[0] != T or positions.shape[0] != T:
        raise ValueError("k, v, slot_mapping and positions must have the same tokens")
    scales = (_scales("k_scale", k_scale, Hkv), _scales("v_scale", v_scale, Hkv)) if kv8 else (None, None)
    P, r = cos_sin.shape
    _check(load().pkv_paged_kv_append_rotary(qo, qi, k.data_ptr(), v.data_ptr(), kc, vc, sm, ps, cs, T, qos, qis, ks, vs, P, r,
                                             1 if interleaved else 0, NB, bs, Hq, Hkv, d, _DT[k.dtype], _POOL_DT[dt],
                                             *scales, _stream(key_cache)))


def decode_partition_tokens(num_seqs, num_heads, num_kv_heads, head_dim, max_seq_len) -> int:
    return int(load().pkv_decode_partition_tokens(num_seqs, num_heads, num_kv_heads, head_dim, max_seq_len))


@_one_device
def decode_plan_partition_tokens(workspace, num_seqs, num_heads, num_kv_heads) -> int:
    """Partition size the last decode call with ``workspace`` used (-1: unplanned batch); synchronises."""
    return int(load().pkv_decode_plan_partition_tokens(_cuda("workspace", workspace), num_seqs, num_heads,
                                                       num_kv_heads, _stream(workspace)))


def decode_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim, max_seq_len, partition_tokens=0) -> int:
    n = load().pkv_decode_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim, max_seq_len, partition_tokens)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("invalid decode shape")
    return int(n)


def alloc_workspace(num_seqs, num_heads, num_kv_heads, head_dim, max_seq_len, partition_tokens=0, device="cuda"):
    """A device buffer of the size the decode call needs."""
    n = decode_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim, max_seq_len, partition_tokens)
    return torch.empty(n, dtype=torch.uint8, device=device)


@_one_device
def decode_plan(workspace, block_tables, seq_lens, num_heads, key_cache, max_seq_len, partition_tokens=0,
                sum_seq_lens=0) -> None:
    """The work list of a decode batch, once per step (``pkv_decode_plan``): the runs that pass
    ``planned=True`` over the same batch then skip the plan kernel.  ``key_cache`` gives the pool's
    shape and element type (uint8: E4M3).  ``sum_seq_lens``: the lengths' sum if known (sizes the
    grid tighter; the runs must pass the same value)."""
    NB, bs, Hkv, d = _pool("key_cache", key_cache, tuple(_POOL_DT))
    B = seq_lens.shape[0]
    _cuda("block_tables", block_tables, torch.int32, 2)
    _cuda("seq_lens", seq_lens, torch.int32, 1)
    _check(load().pkv_decode_plan(ctypes.c_void_p(block_tables.data_ptr()), block_tables.shape[1],
                                  ctypes.c_void_p(seq_lens.data_ptr()), B, int(max_seq_len), int(sum_seq_lens),
                                  num_heads, Hkv, d, bs,
                                  _POOL_DT[key_cache.dtype], _cuda("workspace", workspace),
                                  workspace.numel() * workspace.element_size(), int(partition_tokens),
                                  _stream(workspace)))


@_one_device
def paged_attention_decode(out, q, key_cache, value_cache, block_tables, seq_lens, scale=None, block_size=None,
                           num_kv_heads=None, max_seq_len=None, workspace=None, partition_tokens=0,
                           planned=False, sum_seq_lens=0) -> None:
    """out[s, h] = softmax(scale * q[s, h] . K) V over positions [0, seq_lens[s]) of KV head h // G.

    q, out: [B, Hq, d]; caches [NB, bs, Hkv, d]; block_tables int32 [B, W]; seq_lens int32 [B].
    ``max_seq_len`` is the host-known bound of seq_lens (read from the device
    if omitted, which synchronises).  ``workspace``: see ``alloc_workspace``
    (allocated here when omitted).  ``planned``: run over the work list
    ``decode_plan`` put in ``workspace`` for this batch (no plan kernel).
    """
    NB, bs, Hkv, d = _pool("key_cache", key_cache)
    if block_size is not None and block_size != bs:
        raise ValueError(f"block_size {block_size} != cache block size {bs}")
    if num_kv_heads is not None and num_kv_heads != Hkv:
        raise ValueError(f"num_kv_heads {num_kv_heads} != cache heads {Hkv}")
    if value_cache.shape != key_cache.shape or value_cache.dtype != key_cache.dtype:
        raise ValueError("value_cache must match key_cache")
    B, Hq, dq = q.shape
    if dq != d or tuple(out.shape) != (B, Hq, d):
        raise ValueError("q and out must be [B, num_heads, head_dim]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if max_seq_len is None:
        max_seq_len = int(seq_lens.max().item()) if B else 0
    ptrs = [_cuda("out", out, key_cache.dtype), _cuda("q", q, key_cache.dtype), _cuda("key_cache", key_cache),
            _cuda("value_cache", value_cache), _cuda("block_tables", block_tables, torch.int32, 2)]
    _cuda("seq_lens", seq_lens, torch.int32, 1)
    if block_tables.shape[0] != B or seq_lens.shape[0] != B:
        raise ValueError("block_tables / seq_lens batch mismatch")
    if workspace is None:
        workspace = alloc_workspace(B, Hq, Hkv, d, int(max_seq_len), partition_tokens, q.device)
    ws_ptr = _cuda("workspace", workspace)
    ws_bytes = workspace.numel() * workspace.element_size()
    lens_arg = [ctypes.c_void_p(seq_lens.data_ptr()), B, int(max_seq_len)]
    if planned:
        _check(load().pkv_paged_attention_decode_planned(
            *ptrs, block_tables.shape[1], *lens_arg, int(sum_seq_lens), Hq, Hkv, d, bs, NB, float(scale),
            _DT[key_cache.dtype], ws_ptr, ws_bytes, int(partition_tokens), _stream(q)))
    else:
        _check(load().pkv_paged_attention_decode(
            *ptrs, block_tables.shape[1], *lens_arg, Hq, Hkv, d, bs, NB, float(scale), _DT[key_cache.dtype], ws_ptr,
            ws_bytes, int(partition_tokens), _stream(q)))


def _scales(name, t, Hkv):
    _cuda(name, t, torch.float32, 1)
    if t.shape[0] != Hkv:
        raise ValueError(f"{name} must have num_kv_heads = {Hkv} entries")
    return t.data_ptr()


@_one_device
def paged_kv_append_fp8(k, v, key_cache, value_cache, slot_mapping, k_scale, v_scale) -> None:
    """Quantize k[t], v[t] ([T, Hkv, d], fp16 / bf16) into slot slot_mapping[t] of uint8 E4M3 pools:
    code = e4m3(float32(x) / scale[head]) (nearest even, saturating); k_scale, v_scale float32 [Hkv]."""
    NB, bs, Hkv, d = _pool("key_cache", key_cache, (torch.uint8,))
    if value_cache.shape != key_cache.shape or value_cache.dtype != torch.uint8:
        raise ValueError("value_cache must match key_cache")
    T = k.shape[0]
    if tuple(k.shape) != (T, Hkv, d) or v.shape != k.shape or v.dtype != k.dtype:
        raise ValueError("k and v must be [T, num_kv_heads, head_dim] of one dtype")
    args = [_cuda("k", k, (torch.float16, torch.bfloat16)), _cuda("v", v, k.dtype), _cuda("key_cache", key_cache),
            _cuda("value_cache", value_cache), _cuda("slot_mapping", slot_mapping, torch.int64, 1)]
    if slot_mapping.shape[0] != T:
        raise ValueError("slot_mapping must have T entries")
    _check(load().pkv_paged_kv_append_fp8(*args, T, NB, bs, Hkv, d, _DT[k.dtype], _scales("k_scale", k_scale, Hkv),
                                          _scales("v_scale", v_scale, Hkv), _stream(key_cache)))


@_one_device
def paged_attention_decode_fp8(out, q, key_cache, value_cache, block_tables, seq_lens, k_scale, v_scale, scale=None,
                               max_seq_len=None, workspace=None, partition_tokens=0, planned=False,
                               sum_seq_lens=0) -> None:
    """paged_attention_decode over uint8 E4M3 pools: K = e4m3(code) * k_scale[g], V = e4m3(code) * v_scale[g];
    q, out fp16 / bf16 [B, Hq, 128]; k_scale, v_scale float32 [Hkv]."""
    NB, bs, Hkv, d = _pool("key_cache", key_cache, (torch.uint8,))
    if value_cache.shape != key_cache.shape or value_cache.dtype != torch.uint8:
        raise ValueError("value_cache must match key_cache")
    B, Hq, dq = q.shape
    if dq != d or tuple(out.shape) != (B, Hq, d):
        raise ValueError("q and out must be [B, num_heads, head_dim]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if max_seq_len is None:
        max_seq_len = int(seq_lens.max().item()) if B else 0
    ptrs = [_cuda("out", out, (torch.float16, torch.bfloat16)), _cuda("q", q, out.dtype), _cuda("key_cache", key_cache),
            _cuda("value_cache", value_cache), _cuda("block_tables", block_tables, torch.int32, 2)]
    _cuda("seq_lens", seq_lens, torch.int32, 1)
    if block_tables.shape[0] != B or seq_lens.shape[0] != B:
        raise ValueError("block_tables / seq_lens batch mismatch")
    if workspace is None:
        workspace = alloc_workspace(B, Hq, Hkv, d, int(max_seq_len), partition_tokens, q.device)
    ws_ptr = _cuda("workspace", workspace)
    ws_bytes = workspace.numel() * workspace.element_size()
    lens_arg = [ctypes.c_void_p(seq_lens.data_ptr()), B, int(max_seq_len)]
    rest = [Hq, Hkv, d, bs, NB, float(scale), _DT[q.dtype], _scales("k_scale", k_scale, Hkv),
            _scales("v_scale", v_scale, Hkv), ws_ptr, ws_bytes, int(partition_tokens), _stream(q)]
    if planned:
        _check(load().pkv_paged_attention_decode_fp8_planned(*ptrs, block_tables.shape[1], *lens_arg,
                                                             int(sum_seq_lens), *rest))
    else:
        _check(load().pkv_paged_attention_decode_fp8(*ptrs, block_tables.shape[1], *lens_arg, *rest))


@_one_device
def paged_kv_append_decode(out, q, k, v, key_cache, value_cache, slot_mapping, block_tables, seq_lens, scale=None,
                           max_seq_len=None, workspace=None, partition_tokens=0, planned=False, sum_seq_lens=0,
                           k_scale=None, v_scale=None, inputs_ready=False) -> None:
    """paged_kv_append of one new token per sequence (k, v [B, Hkv, d]; slot_mapping int64 [B], the slot of
    position seq_lens[s] - 1, or < 0 for none) then paged_attention_decode, in one launch.  uint8 pools hold
    E4M3 codes and take k_scale / v_scale as paged_kv_append_fp8 does.  ``inputs_ready`` (with ``planned``):
    the caller guarantees that no work still pending on the stream writes the pools, block tables, seq_lens or
    the workspace's plan (every layer of a step after the first), so the tile loads may start while the
    preceding kernel finishes (``PKV_INPUTS_READY``)."""
    if inputs_ready and not planned:
        raise ValueError("inputs_ready needs planned=True (a plan written by an earlier call)")
    kv8 = key_cache.dtype == torch.uint8
    NB, bs, Hkv, d = _pool("key_cache", key_cache, tuple(_POOL_DT))
    if value_cache.shape != key_cache.shape or value_cache.dtype != key_cache.dtype:
        raise ValueError("value_cache must match key_cache")
    B, Hq, dq = q.shape
    if dq != d or tuple(out.shape) != (B, Hq, d):
        raise ValueError("q and out must be [B, num_heads, head_dim]")
    if tuple(k.shape) != (B, Hkv, d) or tuple(v.shape) != (B, Hkv, d):
        raise ValueError("k and v must be [B, num_kv_heads, head_dim]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if max_seq_len is None:
        max_seq_len = int(seq_lens.max().item()) if B else 0
    qdt = (torch.float16, torch.bfloat16) if kv8 else key_cache.dtype
    ptrs = [_cuda("out", out, qdt), _cuda("q", q, out.dtype), _cuda("k", k, out.dtype, 3), _cuda("v", v, out.dtype, 3),
            _cuda("key_cache", key_cache), _cuda("value_cache", value_cache),
            _cuda("slot_mapping", slot_mapping, torch.int64, 1), _cuda("block_tables", block_tables, torch.int32, 2)]
    _cuda("seq_lens", seq_lens, torch.int32, 1)
    if block_tables.shape[0] != B or seq_lens.shape[0] != B or slot_mapping.shape[0] != B:
        raise ValueError("block_tables / seq_lens / slot_mapping batch mismatch")
    if kv8:
        scales = [_scales("k_scale", k_scale, Hkv), _scales("v_scale", v_scale, Hkv)]
    else:
        scales = [None, None]
    if workspace is None:
        workspace = alloc_workspace(B, Hq, Hkv, d, int(max_seq_len), partition_tokens, q.device)
    ws_ptr = _cuda("workspace", workspace)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(load().pkv_paged_kv_append_decode(
        *ptrs, block_tables.shape[1], ctypes.c_void_p(seq_lens.data_ptr()), B, int(max_seq_len), int(sum_seq_lens),
        Hq, Hkv, d, bs, NB, float(scale), _DT[q.dtype], _POOL_DT[key_cache.dtype], *scales, ws_ptr, ws_bytes,
        int(partition_tokens), (PLANNED if planned else 0) | (INPUTS_READY if inputs_ready else 0), _stream(q)))


@_one_device
def paged_attention_verify(out, q, key_cache, value_cache, block_tables, seq_lens, scale=None, max_seq_len=None,
                           workspace=None, partition_tokens=0, sum_seq_lens=0, k_scale=None, v_scale=None) -> None:
    """Multi-query paged attention: q, out [B, nq, Hq, d]; query token i of sequence s attends over
    positions [0, seq_lens[s] - nq + i] (the last nq positions are the queries' own K/V).  uint8 pools
    hold E4M3 codes and take k_scale / v_scale (float32 [Hkv]) as paged_attention_decode_fp8 does."""
    kv8 = key_cache.dtype == torch.uint8
    NB, bs, Hkv, d = _pool("key_cache", key_cache, tuple(_POOL_DT))
    if value_cache.shape != key_cache.shape or value_cache.dtype != key_cache.dtype:
        raise ValueError("value_cache must match key_cache")
    if q.dim() != 4:
        raise ValueError("q must be [B, num_queries, num_heads, head_dim]")
    B, nq, Hq, dq = q.shape
    if dq != d or tuple(out.shape) != tuple(q.shape):
        raise ValueError("q and out must be [B, num_queries, num_heads, head_dim]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if max_seq_len is None:
        max_seq_len = int(seq_lens.max().item()) if B else 0
    qdt = (torch.float16, torch.bfloat16) if kv8 else key_cache.dtype
    ptrs = [_cuda("out", out, qdt), _cuda("q", q, out.dtype), _cuda("key_cache", key_cache),
            _cuda("value_cache", value_cache), _cuda("block_tables", block_tables, torch.int32, 2)]
    _cuda("seq_lens", seq_lens, torch.int32, 1)
    if block_tables.shape[0] != B or seq_lens.shape[0] != B:
        raise ValueError("block_tables / seq_lens batch mismatch")
    if workspace is None:
        workspace = alloc_workspace(B, Hq * nq, Hkv, d, int(max_seq_len), partition_tokens, q.device)
    ws_ptr = _cuda("workspace", workspace)
    ws_bytes = workspace.numel() * workspace.element_size()
    lens_arg = [ctypes.c_void_p(seq_lens.data_ptr()), B, int(max_seq_len), int(sum_seq_lens)]
    if kv8:
        _check(load().pkv_paged_attention_verify_fp8(
            *ptrs, block_tables.shape[1], *lens_arg, Hq, Hkv, d, bs, NB, float(scale), _DT[q.dtype],
            _scales("k_scale", k_scale, Hkv), _scales("v_scale", v_scale, Hkv), nq, ws_ptr, ws_bytes,
            int(partition_tokens), _stream(q)))
    else:
        _check(load().pkv_paged_attention_verify(
            *ptrs, block_tables.shape[1], *lens_arg, Hq, Hkv, d, bs, NB, float(scale), _DT[key_cache.dtype], nq,
            ws_ptr, ws_bytes, int(partition_tokens), _stream(q)))


def prefill_workspace_bytes(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim) -> int:
    n = load().pkv_prefill_workspace_bytes(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("invalid prefill shape")
    return int(n)


def alloc_prefill_workspace(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim, device="cuda"):
    """A device buffer of the size the prefill call needs (for this many new tokens in all)."""
    n = prefill_workspace_bytes(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim)
    return torch.empty(n, dtype=torch.uint8, device=device)


@_one_device
def prefill_plan(workspace, seq_lens, query_starts, num_tokens, num_heads, num_kv_heads, head_dim,
                 max_seq_len) -> None:
    """The work list of a prefill batch, once per step (``pkv_prefill_plan``): the layers that pass
    ``planned=True`` with the same batch and workspace then skip the plan kernel."""
    B = seq_lens.shape[0]
    args = [_cuda("seq_lens", seq_lens, torch.int32, 1), _cuda("query_starts", query_starts, torch.int32, 1)]
    if query_starts.shape[0] != B + 1:
        raise ValueError("query_starts must have num_seqs + 1 entries")
    _check(load().pkv_prefill_plan(*args, B, int(num_tokens), int(max_seq_len), num_heads, num_kv_heads, head_dim,
                                   _cuda("workspace", workspace), workspace.numel() * workspace.element_size(),
                                   _stream(workspace)))


def paged_attention_prefill(out, q, key_cache, value_cache, block_tables, seq_lens, query_starts, scale=None,
                            max_seq_len=None, workspace=None, planned=False, k_scale=None, v_scale=None) -> None:
    """Attention of a ragged batch of new tokens over the paged cache.  q, out: [T, Hq, d]; sequence s owns rows
    query_starts[s] .. query_starts[s + 1] - 1 (int32 [B + 1]), whose K/V are its last positions in the pools; row i
    of n attends over positions [0, seq_lens[s] - n + i].  Rows of no sequence are left as they are.  ``workspace``:
    see ``alloc_prefill_workspace`` (allocated here when omitted); ``planned``: run over the list ``prefill_plan``
    put there for this batch.  ``max_seq_len`` is read from the device if omitted, which synchronises.  uint8 pools hold
    E4M3 codes and take k_scale / v_scale (float32 [Hkv]) as paged_attention_decode_fp8 does."""
    if _usual(q, out, key_cache, value_cache, block_tables, seq_lens, query_starts, workspace) and scale is not None and \
            max_seq_len is not None:
        dt, qdt, pool, rows, table = key_cache.dtype, q.dtype, key_cache.shape, q.shape, block_tables.shape
        kv8 = dt is torch.uint8
        if (kv8 or dt is qdt) and qdt in _DT and out.dtype is qdt and value_cache.dtype is dt and \
                block_tables.dtype is seq_lens.dtype is query_starts.dtype is torch.int32 and len(pool) == 4 and \
                len(rows) == 3 and len(table) == 2 and value_cache.shape == pool and out.shape == rows and \
                seq_lens.shape == table[:1] and query_starts.shape == (table[0] + 1,) and rows[2] == pool[3] and \
                (k_scale is None and v_scale is None if not kv8 else _usual(q, k_scale, v_scale) and
                 k_scale.dtype is v_scale.dtype is torch.float32 and k_scale.shape == v_scale.shape == pool[2:3]):
            args = (out.data_ptr(), q.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(), block_tables.data_ptr(),
                    table[1], seq_lens.data_ptr(), query_starts.data_ptr(), table[0], rows[0], int(max_seq_len), rows[1],
                    pool[2], pool[3], pool[1], pool[0], float(scale), _DT[qdt])
            end = (workspace.data_ptr(), workspace.nbytes, PLANNED if planned else 0, _stream(q))
            if kv8:
                status = load().pkv_paged_attention_prefill_fp8(*args, k_scale.data_ptr(), v_scale.data_ptr(), *end)
            else:
                status = load().pkv_paged_attention_prefill(*args, *end)
            return _check(status)
    _prefill(out, q, key_cache, value_cache, block_tables, seq_lens, query_starts, scale, max_seq_len, workspace, planned,
             k_scale, v_scale)


@_one_device
def _prefill(out, q, key_cache, value_cache, block_tables, seq_lens, query_starts, scale, max_seq_len, workspace, planned,
             k_scale, v_scale) -> None:
    dt = key_cache.dtype
    kv8 = dt is torch.uint8
    if not kv8 and (k_scale is not None or v_scale is not None):
        raise ValueError("k_scale / v_scale belong to E4M3 (uint8) pools")
    kc = _cuda("key_cache", key_cache, _POOL_DTS, 4)
    NB, bs, Hkv, d = key_cache.shape
    if value_cache.shape != key_cache.shape or value_cache.dtype is not dt:
        raise ValueError("value_cache must match key_cache")
    qp = _cuda("q", q, _HALF_DTS if kv8 else dt)
    if q.dim() != 3:
        raise ValueError("q must be [num_tokens, num_heads, head_dim]")
    T, Hq, dq = q.shape
    if dq != d or out.shape != q.shape:
        raise ValueError("q and out must be [num_tokens, num_heads, head_dim]")
    op, vc, bt = _cuda("out", out, q.dtype), _cuda("value_cache", value_cache), _cuda("block_tables", block_tables, torch.int32, 2)
    sl, qs = _cuda("seq_lens", seq_lens, torch.int32, 1), _cuda("query_starts", query_starts, torch.int32, 1)
    B = seq_lens.shape[0]
    NT, W = block_tables.shape
    if NT != B or query_starts.shape[0] != B + 1:
        raise ValueError("block_tables must have num_seqs rows and query_starts num_seqs + 1 entries")
    if workspace is None:
        if planned:
            raise ValueError("planned=True needs the workspace that prefill_plan wrote")
        workspace = alloc_prefill_workspace(B, T, Hq, Hkv, d, q.device)
    if max_seq_len is None:
        max_seq_len = int(seq_lens.max().item()) if B else 0
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    wp, flags = _cuda("workspace", workspace), PLANNED if planned else 0
    if kv8:
        ks, vs = _scales("k_scale", k_scale, Hkv), _scales("v_scale", v_scale, Hkv)
        _check(load().pkv_paged_attention_prefill_fp8(op, qp, kc, vc, bt, W, sl, qs, B, T, int(max_seq_len), Hq, Hkv, d, bs, NB,
                                                      scale, _DT[q.dtype], ks, vs, wp, workspace.nbytes, flags, _stream(q)))
    else:
        _check(load().pkv_paged_attention_prefill(op, qp, kc, vc, bt, W, sl, qs, B, T, int(max_seq_len), Hq, Hkv, d, bs, NB,
                                                  scale, _DT[dt], wp, workspace.nbytes, flags, _stream(q)))


def paged_attention_tree(out, q, key_cache, value_cache, block_tables, seq_lens, query_starts, tree_mask, scale=None,
                         max_seq_len=None, workspace=None, planned=False, k_scale=None, v_scale=None) -> None:
    """Attention of drafted trees over the paged cache.  q, out: [T, Hq, d]; sequence s's nodes (up to 64) are rows
    query_starts[s] .. query_starts[s + 1] - 1 (int32 [B + 1]), whose K/V are its last n positions in the pools, in that
    order; node i attends over every position before them and over node j where bit j <= i of its int64 tree_mask entry
    is set (its ancestors' and its own).  ``workspace``, ``planned``, ``max_seq_len``, E4M3 pools and their scales: as
    paged_attention_prefill, whose plan it shares."""
    if _usual(q, out, key_cache, value_cache, block_tables, seq_lens, query_starts, tree_mask, workspace) and \
            scale is not None and max_seq_len is not None:
        dt, qdt, pool, rows, table = key_cache.dtype, q.dtype, key_cache.shape, q.shape, block_tables.shape
        kv8 = dt is torch.uint8
        if (kv8 or dt is qdt) and qdt in _DT and out.dtype is qdt and value_cache.dtype is dt and \
                block_tables.dtype is seq_lens.dtype is query_starts.dtype is torch.int32 and len(pool) == 4 and \
                tree_mask.dtype is torch.int64 and len(rows) == 3 and len(table) == 2 and value_cache.shape == pool and \
                out.shape == rows and seq_lens.shape == table[:1] and query_starts.shape == (table[0] + 1,) and \
                rows[2] == pool[3] and tree_mask.shape == rows[:1] and \
                (k_scale is None and v_scale is None if not kv8 else _usual(q, k_scale, v_scale) and
                 k_scale.dtype is v_scale.dtype is torch.float32 and k_scale.shape == v_scale.shape == pool[2:3]):
            return _check(load().pkv_paged_attention_tree(
                out.data_ptr(), q.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(), block_tables.data_ptr(), table[1],
                seq_lens.data_ptr(), query_starts.data_ptr(), tree_mask.data_ptr(), table[0], rows[0], int(max_seq_len),
                rows[1], pool[2], pool[3], pool[1], pool[0], float(scale), _DT[qdt], _POOL_DT[dt],
                k_scale.data_ptr() if kv8 else None, v_scale.data_ptr() if kv8 else None, workspace.data_ptr(),
                workspace.nbytes, PLANNED if planned else 0, _stream(q)))
    _tree(out, q, key_cache, value_cache, block_tables, seq_lens, query_starts, tree_mask, scale, max_seq_len, workspace,
          planned, k_scale, v_scale)


@_one_device
def _tree(out, q, key_cache, value_cache, block_tables, seq_lens, query_starts, tree_mask, scale, max_seq_len, workspace,
          planned, k_scale, v_scale) -> None:
    dt = key_cache.dtype
    kv8 = dt is torch.uint8
    if not kv8 and (k_scale is not None or v_scale is not None):
        raise ValueError("k_scale / v_scale belong to E4M3 (uint8) pools")
    kc = _cuda("key_cache", key_cache, _POOL_DTS, 4)
    NB, bs, Hkv, d = key_cache.shape
    if value_cache.shape != key_cache.shape or value_cache.dtype is not dt:
        raise ValueError("value_cache must match key_cache")
    qp = _cuda("q", q, _HALF_DTS if kv8 else dt, 3)
    T, Hq, dq = q.shape
    if dq != d or out.shape != q.shape:
        raise ValueError("q and out must be [num_tokens, num_heads, head_dim]")
    op, vc, bt = _cuda("out", out, q.dtype), _cuda("value_cache", value_cache), _cuda("block_tables", block_tables, torch.int32, 2)
    sl, qs = _cuda("seq_lens", seq_lens, torch.int32, 1), _cuda("query_starts", query_starts, torch.int32, 1)
    tm = _cuda("tree_mask", tree_mask, torch.int64, 1)
    B = seq_lens.shape[0]
    NT, W = block_tables.shape
    if NT != B or query_starts.shape[0] != B + 1:
        raise ValueError("block_tables must have num_seqs rows and query_starts num_seqs + 1 entries")
    if tree_mask.shape[0] != T:
        raise ValueError("tree_mask must have num_tokens entries")
    if workspace is None:
        if planned:
            raise ValueError("planned=True needs the workspace that prefill_plan wrote")
        workspace = alloc_prefill_workspace(B, T, Hq, Hkv, d, q.device)
    if max_seq_len is None:
        max_seq_len = int(seq_lens.max().item()) if B else 0
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    wp = _cuda("workspace", workspace)
    scales = (_scales("k_scale", k_scale, Hkv), _scales("v_scale", v_scale, Hkv)) if kv8 else (None, None)
    _check(load().pkv_paged_attention_tree(op, qp, kc, vc, bt, W, sl, qs, tm, B, T, int(max_seq_len), Hq, Hkv, d, bs, NB, scale,
                                           _DT[q.dtype], _POOL_DT[dt], *scales, wp, workspace.nbytes, PLANNED if planned else 0,
                                           _stream(q)))


def paged_kv_gather(k_out, v_out, key_cache, value_cache, block_tables, seq_lens, row_starts, k_scale=None,
                    v_scale=None) -> None:
    """Rows row_starts[s] + t of k_out, v_out ([R, Hkv, d]) = position t < seq_lens[s] of sequence s (row_starts
    int32 [B + 1]; other rows are left as they are).  uint8 pools hold E4M3 codes and take k_scale / v_scale
    (float32 [Hkv]): the rows are then code value * scale, rounded to the outputs' fp16 / bf16."""
    if _usual(key_cache, value_cache, k_out, v_out, block_tables, seq_lens, row_starts):
        dt, odt, pool, rows, table = key_cache.dtype, k_out.dtype, key_cache.shape, k_out.shape, block_tables.shape
        kv8 = dt is torch.uint8
        if (kv8 or dt is odt) and odt in _DT and v_out.dtype is odt and value_cache.dtype is dt and \
                block_tables.dtype is seq_lens.dtype is row_starts.dtype is torch.int32 and len(pool) == 4 and \
                len(rows) == 3 and len(table) == 2 and value_cache.shape == pool and v_out.shape == rows and \
                seq_lens.shape == table[:1] and row_starts.shape == (table[0] + 1,) and rows[1:] == pool[2:] and \
                (k_scale is None and v_scale is None if not kv8 else _usual(k_out, k_scale, v_scale) and
                 k_scale.dtype is v_scale.dtype is torch.float32 and k_scale.shape == v_scale.shape == pool[2:3]):
            args = (k_out.data_ptr(), v_out.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(), block_tables.data_ptr(),
                    table[1], seq_lens.data_ptr(), row_starts.data_ptr(), table[0], rows[0], *pool, _DT[odt])
            if kv8:
                status = load().pkv_paged_kv_gather_fp8(*args, k_scale.data_ptr(), v_scale.data_ptr(), _stream(k_out))
            else:
                status = load().pkv_paged_kv_gather(*args, _stream(k_out))
            return _check(status)
    _gather(k_out, v_out, key_cache, value_cache, block_tables, seq_lens, row_starts, k_scale, v_scale)


@_one_device
def _gather(k_out, v_out, key_cache, value_cache, block_tables, seq_lens, row_starts, k_scale, v_scale) -> None:
    dt = key_cache.dtype
    kv8 = dt is torch.uint8
    if not kv8 and (k_scale is not None or v_scale is not None):
        raise ValueError("k_scale / v_scale belong to E4M3 (uint8) pools")
    kc = _cuda("key_cache", key_cache, _POOL_DTS, 4)
    NB, bs, Hkv, d = key_cache.shape
    if value_cache.shape != key_cache.shape or value_cache.dtype is not dt:
        raise ValueError("value_cache must match key_cache")
    ko = _cuda("k_out", k_out, _HALF_DTS if kv8 else dt, 3)
    vo, vc = _cuda("v_out", v_out, k_out.dtype, 3), _cuda("value_cache", value_cache)
    bt = _cuda("block_tables", block_tables, torch.int32, 2)
    R, Hr, dr = k_out.shape
    if Hr != Hkv or dr != d or v_out.shape != k_out.shape:
        raise ValueError("k_out and v_out must be [rows, num_kv_heads, head_dim]")
    sl, rs = _cuda("seq_lens", seq_lens, torch.int32, 1), _cuda("row_starts", row_starts, torch.int32, 1)
    B = seq_lens.shape[0]
    NT, W = block_tables.shape
    if NT != B or row_starts.shape[0] != B + 1:
        raise ValueError("block_tables must have num_seqs rows and row_starts num_seqs + 1 entries")
    if kv8:
        _check(load().pkv_paged_kv_gather_fp8(ko, vo, kc, vc, bt, W, sl, rs, B, R, NB, bs, Hkv, d, _DT[k_out.dtype],
                                              _scales("k_scale", k_scale, Hkv), _scales("v_scale", v_scale, Hkv),
                                              _stream(key_cache)))
    else:
        _check(load().pkv_paged_kv_gather(ko, vo, kc, vc, bt, W, sl, rs, B, R, NB, bs, Hkv, d, _DT[dt], _stream(key_cache)))


def speculative_accept(tokens, num_accepted, draft_tokens, target_probs, uniform, draft_probs=None,
                       num_drafts=None) -> None:
    """Accept drafted tokens against the target's probabilities and draw the token that follows.

    draft_tokens int64 [B, K]; target_probs [B, K + 1, V] and draft_probs [B, K, V] (None: drafts without
    probabilities, taken as certain) float32 / float16 / bfloat16; uniform float32 [B, K + 1] in [0, 1): entry
    i < K decides draft i, entry K the draw; num_drafts int32 [B] (None: K each).  tokens int64 [B, K + 1]
    receives the accepted drafts, the drawn token, then -1; num_accepted int32 [B] the count of drafts kept."""
    if _usual(tokens, num_accepted, draft_tokens, target_probs, uniform) and \
            (draft_probs is None or _usual(tokens, draft_probs)) and (num_drafts is None or _usual(tokens, num_drafts)):
        dt, drafts, target, rows = target_probs.dtype, draft_tokens.shape, target_probs.shape, tokens.shape
        if dt in _PROB_DT and tokens.dtype is draft_tokens.dtype is torch.int64 and num_accepted.dtype is torch.int32 and \
                uniform.dtype is torch.float32 and len(drafts) == 2 and len(target) == 3 and \
                rows == (drafts[0], drafts[1] + 1) and target[:2] == rows and uniform.shape == rows and \
                num_accepted.shape == drafts[:1] and \
                (draft_probs is None or draft_probs.dtype is dt and draft_probs.shape == (*drafts, target[2])) and \
                (num_drafts is None or num_drafts.dtype is torch.int32 and num_drafts.shape == drafts[:1]):
            return _check(load().pkv_speculative_accept(
                tokens.data_ptr(), num_accepted.data_ptr(), draft_tokens.data_ptr(),
                None if num_drafts is None else num_drafts.data_ptr(), target_probs.data_ptr(),
                None if draft_probs is None else draft_probs.data_ptr(), uniform.data_ptr(), *drafts, target[2],
                _PROB_DT[dt], _stream(tokens)))
    _accept(tokens, num_accepted, draft_tokens, target_probs, uniform, draft_probs, num_drafts)


@_one_device
def _accept(tokens, num_accepted, draft_tokens, target_probs, uniform, draft_probs, num_drafts) -> None:
    ptrs = [_cuda("tokens", tokens, torch.int64, 2), _cuda("num_accepted", num_accepted, torch.int32, 1),
            _cuda("draft_tokens", draft_tokens, torch.int64, 2)]
    target = _cuda("target_probs", target_probs, _PROB_DTS, 3)
    B, K = draft_tokens.shape
    V = target_probs.shape[2]
    if target_probs.shape != (B, K + 1, V) or tokens.shape != (B, K + 1) or num_accepted.shape[0] != B:
        raise ValueError("target_probs must be [B, K + 1, V], tokens [B, K + 1] and num_accepted [B]")
    if uniform.shape != tokens.shape:
        raise ValueError("uniform must be [B, K + 1]")
    counts = draft = None
    if num_drafts is not None:
        counts = _cuda("num_drafts", num_drafts, torch.int32, 1)
        if num_drafts.shape[0] != B:
            raise ValueError("num_drafts must be [B]")
    if draft_probs is not None:
        draft = _cuda("draft_probs", draft_probs, target_probs.dtype, 3)
        if draft_probs.shape != (B, K, V):
            raise ValueError("draft_probs must be [B, K, V]")
    _check(load().pkv_speculative_accept(*ptrs, counts, target, draft, _cuda("uniform", uniform, torch.float32, 2), B, K,
                                         V, _PROB_DT[target_probs.dtype], _stream(tokens)))


def speculative_accept_tree(tokens, path, num_accepted, draft_tokens, parents, query_starts, target_probs, uniform) -> None:
    """The path through each sequence's drafted tree that follows the target's distribution, and the token after it.

    Nodes are rows query_starts[s] .. query_starts[s + 1] - 1 (int32 [B + 1]; up to 64 a sequence, the first its root) of
    draft_tokens int64 [T], parents int32 [T] (an index within the sequence, before the node's own), target_probs [T, V]
    float32 / float16 / bfloat16 and uniform float32 [T] in [0, 1).  tokens int64 [B, W] receives the accepted drafts, the
    token drawn after them, then -1; path int32 [B, W] the root 0, the accepted nodes, then -1; num_accepted int32 [B] how
    many drafts were accepted, up to W - 1."""
    if _usual(tokens, path, num_accepted, draft_tokens, parents, query_starts, target_probs, uniform):
        dt, rows, shape = target_probs.dtype, target_probs.shape, tokens.shape
        if dt in _PROB_DT and tokens.dtype is draft_tokens.dtype is torch.int64 and uniform.dtype is torch.float32 and \
                path.dtype is num_accepted.dtype is parents.dtype is query_starts.dtype is torch.int32 and len(rows) == 2 and \
                len(shape) == 2 and path.shape == shape and num_accepted.shape == shape[:1] and \
                query_starts.shape == (shape[0] + 1,) and draft_tokens.shape == parents.shape == uniform.shape == rows[:1]:
            return _check(load().pkv_speculative_accept_tree(
                tokens.data_ptr(), path.data_ptr(), num_accepted.data_ptr(), draft_tokens.data_ptr(), parents.data_ptr(),
                query_starts.data_ptr(), target_probs.data_ptr(), uniform.data_ptr(), shape[0], rows[0], shape[1], rows[1],
                _PROB_DT[dt], _stream(tokens)))
    _accept_tree(tokens, path, num_accepted, draft_tokens, parents, query_starts, target_probs, uniform)


@_one_device
def _accept_tree(tokens, path, num_accepted, draft_tokens, parents, query_starts, target_probs, uniform) -> None:
    ptrs = [_cuda("tokens", tokens, torch.int64, 2), _cuda("path", path, torch.int32, 2),
            _cuda("num_accepted", num_accepted, torch.int32, 1), _cuda("draft_tokens", draft_tokens, torch.int64, 1),
            _cuda("parents", parents, torch.int32, 1), _cuda("query_starts", query_starts, torch.int32, 1),
            _cuda("target_probs", target_probs, _PROB_DTS, 2), _cuda("uniform", uniform, torch.float32, 1)]
    (B, W), (T, V) = tokens.shape, target_probs.shape
    if path.shape != tokens.shape or num_accepted.shape[0] != B or query_starts.shape[0] != B + 1:
        raise ValueError("tokens and path must be [B, W], num_accepted [B] and query_starts [B + 1]")
    if draft_tokens.shape[0] != T or parents.shape[0] != T or uniform.shape[0] != T:
        raise ValueError("draft_tokens, parents and uniform must be [T], target_probs [T, V]")
    _check(load().pkv_speculative_accept_tree(*ptrs, B, T, W, V, _PROB_DT[target_probs.dtype], _stream(tokens)))


_get_dtype, _get_shape = operator.attrgetter("dtype"), operator.attrgetter("shape")


def paged_kv_keep_path(key_caches, value_caches, block_tables, seq_lens, query_starts, path, num_accepted) -> None:
    """The cache after a tree step: of sequence s's last n = query_starts[s + 1] - query_starts[s] positions, its tree's
    nodes, those of path[s] (int32 [B, W], 0 = path[s, 0] < .. < path[s, num_accepted[s]]) move to the first
    num_accepted[s] + 1, in every layer's pools.  seq_lens: the lengths with all nodes, as the attention had them; the
    sequence then has seq_lens[s] - n + num_accepted[s] + 1 positions."""
    if _usual(block_tables, seq_lens, query_starts, path, num_accepted) and type(key_caches) is type(value_caches) is list and \
            len(key_caches) == len(value_caches) and key_caches:
        # (map and set over the pools: statements of its own for each of 32 layers' took three times as long)
        pools = key_caches + value_caches
        first, table, shape = pools[0], block_tables.shape, path.shape
        if set(map(type, pools)) == {_Tensor} and set(map(_Tensor.get_device, pools)) == {block_tables.get_device()} and \
                all(map(_Tensor.is_contiguous, pools)) and len(set(map(_get_dtype, pools))) == 1 and \
                list(map(_get_shape, pools)).count(first.shape) == len(pools) and first.dim() == 4 and first.dtype in _POOL_DT and \
                block_tables.dtype is seq_lens.dtype is query_starts.dtype is path.dtype is num_accepted.dtype is torch.int32 and \
                len(table) == len(shape) == 2 and seq_lens.shape == num_accepted.shape == table[:1] == shape[:1] and \
                query_starts.shape == (shape[0] + 1,):
            n, (NB, bs, Hkv, d) = len(key_caches), first.shape
            ptrs = array.array("Q", map(_Tensor.data_ptr, pools))
            at = ptrs.buffer_info()[0]
            return _check(load().pkv_paged_kv_keep_path(
                at, at + 8 * n, n, block_tables.data_ptr(), table[1], seq_lens.data_ptr(), query_starts.data_ptr(),
                path.data_ptr(), num_accepted.data_ptr(), shape[0], shape[1], NB, bs, Hkv, d, _POOL_DT[first.dtype],
                _stream(path)))
    _keep_path(key_caches, value_caches, block_tables, seq_lens, query_starts, path, num_accepted)


@_one_device
def _keep_path(key_caches, value_caches, block_tables, seq_lens, query_starts, path, num_accepted) -> None:
    if isinstance(key_caches, torch.Tensor):
        key_caches, value_caches = [key_caches], [value_caches]
    if len(key_caches) != len(value_caches) or not key_caches:
        raise ValueError("need the same non-zero number of key and value caches")
    shape, dt = key_caches[0].shape, key_caches[0].dtype
    for i, (kc, vc) in enumerate(zip(key_caches, value_caches)):
        _pool(f"key_caches[{i}]", kc, tuple(_POOL_DT))
        _pool(f"value_caches[{i}]", vc, tuple(_POOL_DT))
        if kc.shape != shape or vc.shape != shape or kc.dtype != dt or vc.dtype != dt:
            raise ValueError("all caches must share shape and dtype")
    args = [_cuda("block_tables", block_tables, torch.int32, 2), _cuda("seq_lens", seq_lens, torch.int32, 1),
            _cuda("query_starts", query_starts, torch.int32, 1), _cuda("path", path, torch.int32, 2),
            _cuda("num_accepted", num_accepted, torch.int32, 1)]
    B, W = path.shape
    if block_tables.shape[0] != B or seq_lens.shape[0] != B or query_starts.shape[0] != B + 1 or num_accepted.shape[0] != B:
        raise ValueError("block_tables, seq_lens, path and num_accepted must have num_seqs rows, query_starts one more")
    n = len(key_caches)
    karr = (ctypes.c_void_p * n)(*[kc.data_ptr() for kc in key_caches])
    varr = (ctypes.c_void_p * n)(*[vc.data_ptr() for vc in value_caches])
    NB, bs, Hkv, d = shape
    _check(load().pkv_paged_kv_keep_path(ctypes.addressof(karr), ctypes.addressof(varr), n, args[0], block_tables.shape[1],
                                         *args[1:], B, W, NB, bs, Hkv, d, _POOL_DT[dt], _stream(key_caches[0])))


@_one_device
def copy_blocks(key_caches, value_caches, src_dst_pairs) -> None:
    """For each (src, dst) row of src_dst_pairs (int64 [Np, 2]): every layer's block dst = block src."""
    if isinstance(key_caches, torch.Tensor):
        key_caches, value_caches = [key_caches], [value_caches]
    if len(key_caches) != len(value_caches) or not key_caches:
        raise ValueError("need the same non-zero number of key and value caches")
    shape, dt = key_caches[0].shape, key_caches[0].dtype
    for i, (kc, vc) in enumerate(zip(key_caches, value_caches)):
        _pool(f"key_caches[{i}]", kc, tuple(_POOL_DT))
        _pool(f"value_caches[{i}]", vc, tuple(_POOL_DT))
        if kc.shape != shape or vc.shape != shape or kc.dtype != dt or vc.dtype != dt:
            raise ValueError("all caches must share shape and dtype")
    _cuda("src_dst_pairs", src_dst_pairs, torch.int64, 2)
    if src_dst_pairs.shape[1] != 2:
        raise ValueError("src_dst_pairs must be [Np, 2]")
    n = len(key_caches)
    karr = (ctypes.c_void_p * n)(*[kc.data_ptr() for kc in key_caches])
    varr = (ctypes.c_void_p * n)(*[vc.data_ptr() for vc in value_caches])
    NB, bs, Hkv, d = shape
    _check(load().pkv_copy_blocks(karr, varr, n, ctypes.c_void_p(src_dst_pairs.data_ptr()), src_dst_pairs.shape[0],
                                  NB, bs, Hkv, d, _POOL_DT[dt], _stream(key_caches[0])))


def _addressable_pool(name, t):
    """A pool the GPU can address: a CUDA tensor or a pinned CPU tensor."""
    if not isinstance(t, torch.Tensor) or t.dim() != 4 or t.dtype not in _POOL_DT:
        raise ValueError(f"{name} must be a 4-D fp16 / bf16 / uint8 (E4M3) tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not t.is_cuda and not t.is_pinned():
        raise ValueError(f"{name} must be a CUDA tensor or pinned host memory")
    return t.data_ptr()


@_one_device
def swap_blocks(src_key_caches, src_value_caches, dst_key_caches, dst_value_caches, src_dst_pairs) -> None:
    """dst[dst_i] = src[src_i] for every (src_i, dst_i) row of src_dst_pairs (int64 [Np, 2], on the GPU),
    for every layer's K and V pool.  Pools are CUDA tensors or pinned host tensors (swap out / swap in)."""
    lists = [src_key_caches, src_value_caches, dst_key_caches, dst_value_caches]
    lists = [[x] if isinstance(x, torch.Tensor) else list(x) for x in lists]
    n = len(lists[0])
    if n == 0 or any(len(x) != n for x in lists):
        raise ValueError("need the same non-zero number of pools in every list")
    src_shape, dst_shape, dt = lists[0][0].shape, lists[2][0].shape, lists[0][0].dtype
    ptrs = []
    for li, (name, pools) in enumerate(zip(("src_key", "src_value", "dst_key", "dst_value"), lists)):
        want = src_shape if li < 2 else dst_shape
        for i, t in enumerate(pools):
            ptrs.append(_addressable_pool(f"{name}[{i}]", t))
            if t.shape != want or t.dtype != dt:
                raise ValueError("pools must share dtype; source pools one shape, destination pools another")
    if tuple(src_shape[1:]) != tuple(dst_shape[1:]):
        raise ValueError("source and destination blocks must have the same shape")
    _cuda("src_dst_pairs", src_dst_pairs, torch.int64, 2)
    if src_dst_pairs.shape[1] != 2:
        raise ValueError("src_dst_pairs must be [Np, 2]")
    arrs = [(ctypes.c_void_p * n)(*ptrs[k * n:(k + 1) * n]) for k in range(4)]
    _, bs, Hkv, d = src_shape
    _check(load().pkv_swap_blocks(*arrs, n, ctypes.c_void_p(src_dst_pairs.data_ptr()), src_dst_pairs.shape[0],
                                  src_shape[0], dst_shape[0], bs, Hkv, d, _POOL_DT[dt], _stream(src_dst_pairs)))


class BlockManager:
    """The library's host block manager (``pkv_bm_*``): free list, reference
    counts, copy-on-write at a fork.  Host only; it produces the inputs of the
    decode step (tables, lengths, slots) and the copy pairs for copy_blocks."""

    def __init__(self, num_blocks: int, block_size: int, free_order=None):
        import numpy as np

        self._np = np
        self.block_size = int(block_size)
        self._order = None if free_order is None else np.ascontiguousarray(free_order, dtype=np.int64)
        ptr = None if self._order is None else self._order.ctypes.data
        self._h = load().pkv_bm_create(int(num_blocks), self.block_size, ptr)
        if not self._h:
            raise ValueError("bad block manager arguments")

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            load().pkv_bm_destroy(h)
            self._h = None

    @property
    def num_free_blocks(self) -> int:
        return int(load().pkv_bm_num_free_blocks(self._h))

    def seq_len(self, seq_id) -> int:
        return int(load().pkv_bm_seq_len(self._h, int(seq_id)))

    def refcount(self, block) -> int:
        return int(load().pkv_bm_refcount(self._h, int(block)))

    def allocate(self, seq_id, num_tokens) -> None:
        _check(load().pkv_bm_allocate(self._h, int(seq_id), int(num_tokens)))

    def fork(self, parent_id, child_id) -> None:
        _check(load().pkv_bm_fork(self._h, int(parent_id), int(child_id)))

    def free(self, seq_id) -> None:
        _check(load().pkv_bm_free(self._h, int(seq_id)))

    def append_slots(self, seq_ids):
        """One new token per sequence: (slots int64 [n], cow_pairs int64 [k, 2])."""
        np = self._np
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        slots = np.empty(len(ids), dtype=np.int64)
        cow = np.empty((max(1, len(ids)), 2), dtype=np.int64)
        n = ctypes.c_int64(0)
        _check(load().pkv_bm_append_slots(self._h, ids.ctypes.data, len(ids), slots.ctypes.data, cow.ctypes.data,
                                          cow.shape[0], ctypes.byref(n)))
        return slots, cow[:n.value].copy()

    def block_tables(self, seq_ids, max_blocks_per_seq, pad=-1):
        """(int32 [n, max_blocks_per_seq] tables padded with `pad`, int32 [n] lengths)."""
        np = self._np
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        tables = np.empty((len(ids), max_blocks_per_seq), dtype=np.int32)
        lens = np.empty(len(ids), dtype=np.int32)
        _check(load().pkv_bm_block_tables(self._h, ids.ctypes.data, len(ids), tables.ctypes.data,
                                          int(max_blocks_per_seq), int(pad), lens.ctypes.data))
        return tables, lens


def device_error(reset: bool = True) -> int:
    """The device error word (synchronises the device): bit 0 out-of-range id skipped, bit 1 wait timeout."""
    v = ctypes.c_uint(0)
    _check(load().pkv_device_error(ctypes.byref(v), 1 if reset else 0))
    return int(v.value)
