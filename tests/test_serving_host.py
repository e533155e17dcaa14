"""Refusals of the serving operators: argument checks on the host, nothing launched."""
import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIBPATH = os.path.join(ROOT, "chunk_level_kv_gb300", "libchunkkv.so")
OK, INVALID, UNSUPPORTED, SMALL = 0, 1, 2, 3


@pytest.fixture(scope="module")
def ckv():
    if not os.path.exists(LIBPATH):
        import __graft_entry__
        __graft_entry__.build()
    import chunk_level_kv_gb300 as m
    return m


def _prefill(ckv, cu_q=(0, 40), cu_k=None, dtype=torch.bfloat16, Hq=4, Hkv=2, d=64, **kw):
    q = torch.zeros(cu_q[-1] if cu_q else 0, Hq, d, dtype=dtype)
    k = torch.zeros((cu_k or cu_q)[-1] if cu_q else 0, Hkv, d, dtype=dtype)
    p, keep = ckv.prefill_params_for(q, k, list(cu_q), list(cu_k) if cu_k else None)
    for name, x in kw.items():
        setattr(p, name, x)
    return p, keep


@pytest.mark.parametrize("kw,code", [
    (dict(Hq=3, Hkv=2), INVALID),
    (dict(d=12), INVALID),                          # 24-byte rows
    (dict(d=264), UNSUPPORTED),
    (dict(scale=0.0), INVALID),
    (dict(scale=-1.0), INVALID),
    (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID),
    (dict(dtype=torch.bfloat16, q_stride_t=257), INVALID),
    (dict(kv_stride_h=-64), INVALID),
    (dict(o_stride_t=12), INVALID),
    (dict(B=-1), INVALID),
    (dict(B=1025), UNSUPPORTED),
])
def test_prefill_parameters(ckv, kw, code):
    from chunk_level_kv_gb300._lib import LIB
    p, keep = _prefill(ckv, **kw)
    n = ctypes.c_size_t()
    assert LIB.chunkkv_prefill_workspace_size(ctypes.byref(p), ctypes.byref(n)) == code
    assert LIB.chunkkv_prefill_path(ctypes.byref(p)) == -1
    assert LIB.chunkkv_prefill_attention(ctypes.byref(p), 0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 1 << 20, None) == code


def test_prefill_offsets_pointers_and_workspace(ckv):
    from chunk_level_kv_gb300._lib import LIB
    n0 = ckv.chunkkv_launch_count()

    def call(p, q=0x1000, k=0x2000, v=0x3000, out=0x4000, ws=0x5000, size=1 << 20):
        return LIB.chunkkv_prefill_attention(ctypes.byref(p), q, k, v, out, ws, size, None)
    p, keep = _prefill(ckv)
    size = ckv.chunkkv_prefill_workspace_size(p)
    assert call(p, q=None) == call(p, k=None) == call(p, v=0x3008) == call(p, out=0x4004) == call(p, ws=None) == INVALID
    assert call(p, size=size - 1) == SMALL
    assert LIB.chunkkv_prefill_attention(None, None, None, None, None, None, 0, None) == INVALID
    for cu in ([1, 40], [0, -1]):
        q, keep_q = _prefill(ckv)
        arr = (ctypes.c_int32 * 2)(*cu)
        q.cu_k = ctypes.cast(arr, ctypes.POINTER(ctypes.c_int32))
        assert call(q) == INVALID
    null, keep_n = _prefill(ckv)
    null.cu_q = None
    assert call(null) == INVALID
    empty, keep_e = _prefill(ckv, cu_q=(0, 0))
    assert call(empty, q=None, k=None, v=None, out=None, ws=None, size=0) == OK        # nothing to do
    assert ckv.chunkkv_launch_count() == n0


def test_prefill_binding_checks(ckv):
    z = torch.zeros
    with pytest.raises(ValueError):
        ckv.prefill_params_for(z(4, 2, 64), z(4, 2, 32), [0, 4])
    with pytest.raises(ValueError):
        ckv.prefill_params_for(z(4, 2, 64), z(4, 2, 64), [0, 5])
    with pytest.raises(ValueError):
        ckv.prefill_params_for(z(4, 2, 64).half(), z(4, 2, 64).half(), [0, 4])
    with pytest.raises(ValueError):
        ckv.prefill_params_for(z(4, 64, 2).transpose(1, 2), z(4, 2, 64), [0, 4])
    with pytest.raises(ValueError):
        ckv.prefill_params_for(z(4, 2, 64), z(4, 2, 64), [0, 4], [0, 2, 4])
    with pytest.raises(ValueError):
        ckv.prefill_attention(z(4, 2, 64), z(4, 2, 64), z(4, 2, 128)[:, :, :64], [0, 4])
    with pytest.raises(ckv.ChunkKVError):
        ckv.prefill_attention(z(4, 3, 64), z(4, 2, 64), z(4, 2, 64), [0, 4])


def _struct(**kw):
    from chunk_level_kv_gb300._lib import Q8CacheStruct
    args = dict(B=2, Hkv=2, d=64, n_pages=10, max_pages=4, k_pages=0x10000, v_pages=0x20000, scales=0x30000, table=0x40000,
                lens=0x50000, ring=0x60000, state=0x70000)
    args.update(kw)
    return Q8CacheStruct(**args)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INVALID), (dict(Hkv=0), INVALID), (dict(d=0), INVALID), (dict(d=60), INVALID), (dict(d=264), UNSUPPORTED),
    (dict(B=40000), UNSUPPORTED), (dict(n_pages=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(max_pages=1 << 26), UNSUPPORTED), (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(lens=0x50001), INVALID),
])
def test_cache_structs(ckv, kw, code):
    from chunk_level_kv_gb300._lib import LIB
    c = ctypes.byref(_struct(**kw))
    n = ctypes.c_size_t()
    assert LIB.chunkkv_q8_workspace_size(c, 2, ctypes.byref(n)) == code
    assert LIB.chunkkv_q8_resize(c, 0x1000, None, 0, None) == code
    assert LIB.chunkkv_q8_append(c, 1, 0x1000, 0x1000, 64, 64, 64, 0x1000, 0x1000, 1, None) == code
    assert LIB.chunkkv_q8_load(c, 1, 0x1000, 1, 0x1000, 0x1000, 64, None) == code
    assert LIB.chunkkv_q8_attention(c, 1, 2, 0.1, 0x1000, 64, 64, 0x1000, 64, 64, 0x1000, 1 << 30, None) == code


def test_cache_call_arguments(ckv):
    from chunk_level_kv_gb300._lib import LIB
    n0 = ckv.chunkkv_launch_count()
    c = ctypes.byref(_struct())
    n = ctypes.c_size_t()
    assert LIB.chunkkv_q8_workspace_size(c, 0, ctypes.byref(n)) == INVALID
    assert LIB.chunkkv_q8_workspace_size(c, 1, None) == INVALID
    assert LIB.chunkkv_q8_workspace_size(c, 4, ctypes.byref(n)) == OK and n.value >= 256
    # resize
    assert LIB.chunkkv_q8_resize(c, None, None, 0, None) == INVALID
    assert LIB.chunkkv_q8_resize(c, 0x50000, None, 0, None) == INVALID             # the lengths themselves
    assert LIB.chunkkv_q8_resize(c, 0x1000, 0x2004, 4, None) == INVALID
    assert LIB.chunkkv_q8_resize(c, 0x1000, 0x2000, -1, None) == INVALID
    assert LIB.chunkkv_q8_resize(ctypes.byref(_struct(state=None)), 0x1000, None, 0, None) == INVALID
    # append
    def append(dtype=1, k=0x1000, v=0x2000, st=(64, 64, 64), counts=0x3000, slots=0x4000, cap=3, cache=c):
        return LIB.chunkkv_q8_append(cache, dtype, k, v, *st, counts, slots, cap, None)
    assert append(dtype=2) == append(k=None) == append(v=0x2008) == append(st=(64, 64, 7)) == append(counts=None) == INVALID
    assert append(slots=0x4004) == append(cap=-1) == append(st=(-64, 64, 64)) == INVALID
    assert append(cache=ctypes.byref(_struct(k_pages=None))) == append(cache=ctypes.byref(_struct(scales=0x30004))) == INVALID
    assert append(cap=2147483647) == UNSUPPORTED
    assert append(cap=0, k=None, v=None) == OK
    # load
    assert LIB.chunkkv_q8_load(c, 1, None, 3, 0x1000, 0x1000, 64, None) == INVALID
    assert LIB.chunkkv_q8_load(c, 1, 0x1000, 3, None, 0x1000, 64, None) == INVALID
    assert LIB.chunkkv_q8_load(c, 1, 0x1000, 3, 0x1000, 0x1000, 9, None) == INVALID
    assert LIB.chunkkv_q8_load(c, 0, 0x1000, -2, 0x1000, 0x1000, 64, None) == INVALID
    # attention
    def attend(dtype=1, G=2, scale=0.1, q=0x1000, qs=(256, 64), out=0x2000, os_=(256, 64), ws=0x3000, size=1 << 30):
        return LIB.chunkkv_q8_attention(c, dtype, G, scale, q, *qs, out, *os_, ws, size, None)
    assert attend(dtype=5) == attend(G=0) == attend(scale=0.0) == attend(scale=float("nan")) == attend(q=None) == INVALID
    assert attend(qs=(256, 7)) == attend(os_=(-256, 64)) == attend(out=0x2002) == attend(ws=None) == INVALID
    assert attend(size=16) == SMALL
    assert attend(G=70000) == UNSUPPORTED
    assert LIB.chunkkv_q8_attention(None, 1, 2, 0.1, 0x1000, 64, 64, 0x1000, 64, 64, 0x1000, 1 << 30, None) == INVALID
    assert ckv.chunkkv_launch_count() == n0


def test_cache_binding_checks(ckv):
    cache = ckv.q8_cache(2, 2, 64, n_pages=8, max_pages=3, device="cpu")
    assert cache.k_pages[0].shape == (8, 1, 64, 64) and cache.v_pages[0].shape == (8, 64, 64)
    assert ckv.q8_cache(1, 1, 80, n_pages=2, max_pages=3, device="cpu").k_pages[0].shape == (2, 2, 64, 64)
    i32 = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        ckv.chunkkv_q8_resize(cache, i32.long())
    with pytest.raises(ValueError):
        ckv.chunkkv_q8_resize(cache, i32[:3])
    with pytest.raises(ValueError):
        ckv.chunkkv_q8_resize(cache, i32, torch.zeros(4, 3, dtype=torch.int32))
    k = torch.zeros(2, 2, 5, 64)
    with pytest.raises(ValueError):
        ckv.chunkkv_q8_append(cache, 0, k, k, i32, torch.zeros(4, 4, dtype=torch.int64))
    with pytest.raises(ValueError):
        ckv.chunkkv_q8_append(cache, 0, k, k.half(), i32, torch.zeros(4, 5, dtype=torch.int64))
    with pytest.raises(ValueError):
        ckv.chunkkv_q8_append(cache, 0, k[..., :32], k[..., :32], i32, torch.zeros(4, 5, dtype=torch.int64))
    with pytest.raises(ValueError):
        ckv.chunkkv_q8_load(cache, 0, torch.zeros(4, dtype=torch.int64), 5, k[0, 0], k[0, 0].half())
    q = torch.zeros(2, 3, 64)
    with pytest.raises(ValueError):
        ckv.q8_attention(cache, 0, q)               # 3 query heads for 2 KV heads
    with pytest.raises(ValueError):
        ckv.Q8Cache(B=2, Hkv=2, d=64, k_pages=cache.k_pages, v_pages=[], scales=cache.scales, table=cache.table,
                    lens=cache.lens, ring=cache.ring, state=cache.state)
    with pytest.raises(ValueError):
        ckv.Q8Cache(B=2, Hkv=3, d=64, k_pages=[], v_pages=[], scales=[], table=cache.table, lens=cache.lens,
                    ring=cache.ring, state=cache.state)
