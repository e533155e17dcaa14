"""Refusals of the 4-bit cache's calls: argument checks on the host, nothing launched."""
import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, SMALL = 0, 1, 2, 3


@pytest.fixture(scope="module")
def ckv():
    if not os.path.exists(os.path.join(ROOT, "chunk_level_kv_gb300", "libchunkkv.so")):
        import __graft_entry__
        __graft_entry__.build()
    import chunk_level_kv_gb300 as m
    return m


def _struct(**kw):
    from chunk_level_kv_gb300._lib import Q4CacheStruct
    args = dict(B=2, Hkv=2, d=64, n_pages=10, max_pages=4, pages=0x10000, table=0x40000, lens=0x50000, ring=0x60000,
                state=0x70000)
    args.update(kw)
    return Q4CacheStruct(**args)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INVALID), (dict(Hkv=0), INVALID), (dict(d=0), INVALID), (dict(d=60), INVALID), (dict(d=264), UNSUPPORTED),
    (dict(B=40000), UNSUPPORTED), (dict(n_pages=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(max_pages=1 << 26), UNSUPPORTED), (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(lens=0x50001), INVALID),
])
def test_cache_structs(ckv, kw, code):
    from chunk_level_kv_gb300._lib import LIB
    c = ctypes.byref(_struct(**kw))
    n = ctypes.c_size_t()
    before = ckv.chunkkv_launch_count()
    assert LIB.chunkkv_q4_workspace_size(c, 1, 2, 1, ctypes.byref(n)) == code
    assert LIB.chunkkv_q4_path(c, 1, 2, 1) == -1
    assert LIB.chunkkv_q4_resize(c, 0x1000, None, 0, None) == code
    assert LIB.chunkkv_q4_append(c, 1, 0x1000, 0x1000, 64, 64, 64, 0x1000, 0x1000, 1, None) == code
    assert LIB.chunkkv_q4_load(c, 1, 0x1000, 1, 9, 0x1000, 0x1000, 64, None) == code
    assert LIB.chunkkv_q4_attention(c, 1, 2, 1, None, 0.1, 0x1000, 64, 64, 64, 0x1000, 64, 64, 64, 0x1000, 1 << 30, None) == code
    assert ckv.chunkkv_launch_count() == before


def test_call_arguments(ckv):
    from chunk_level_kv_gb300._lib import LIB
    n0 = ckv.chunkkv_launch_count()
    c = ctypes.byref(_struct())
    n = ctypes.c_size_t()

    def size(dtype=1, G=2, n_q=1, to=ctypes.byref(n)):
        return LIB.chunkkv_q4_workspace_size(c, dtype, G, n_q, to)
    assert size(G=0) == size(n_q=0) == size(dtype=2) == size(to=None) == INVALID
    assert size(G=1 << 16, n_q=1 << 15) == UNSUPPORTED
    assert size(G=1 << 30) == UNSUPPORTED                                          # 2^31 query heads
    assert size() == OK and n.value >= 256
    assert LIB.chunkkv_q4_path(c, 1, 2, 1) in (0, 1) and LIB.chunkkv_q4_path(c, 1, 2, 0) == LIB.chunkkv_q4_path(c, 3, 2, 1) == -1
    # resize
    assert LIB.chunkkv_q4_resize(c, None, None, 0, None) == INVALID
    assert LIB.chunkkv_q4_resize(c, 0x50000, None, 0, None) == INVALID             # the lengths themselves
    assert LIB.chunkkv_q4_resize(c, 0x1000, 0x2004, 4, None) == INVALID
    assert LIB.chunkkv_q4_resize(c, 0x1000, 0x2000, -1, None) == INVALID
    assert LIB.chunkkv_q4_resize(c, 0x1000, 0x2000, 2147483647, None) == UNSUPPORTED
    assert LIB.chunkkv_q4_resize(ctypes.byref(_struct(state=None)), 0x1000, None, 0, None) == INVALID

    # append
    def append(dtype=1, k=0x1000, v=0x2000, st=(64, 64, 64), counts=0x3000, slots=0x4000, cap=3, cache=c):
        return LIB.chunkkv_q4_append(cache, dtype, k, v, *st, counts, slots, cap, None)
    assert append(dtype=2) == append(k=None) == append(v=0x2008) == append(st=(64, 64, 7)) == append(counts=None) == INVALID
    assert append(slots=0x4004) == append(cap=-1) == append(st=(-64, 64, 64)) == append(k=0x1008) == INVALID
    assert append(cache=ctypes.byref(_struct(pages=None))) == append(cache=ctypes.byref(_struct(pages=0x10008))) == INVALID
    assert append(cap=2147483647) == UNSUPPORTED
    assert append(cap=0, k=None, v=None) == OK

    # load
    def load(dtype=1, start=0x1000, cap=3, rows=10, k=0x1000, v=0x1000, st=64):
        return LIB.chunkkv_q4_load(c, dtype, start, cap, rows, k, v, st, None)
    assert load(start=None) == load(k=None) == load(v=0x1002) == load(st=9) == load(cap=-2) == load(rows=-1) == load(dtype=7) == INVALID
    assert load(cap=2147483647) == UNSUPPORTED
    assert load(rows=0, k=None) == load(cap=0, k=None) == OK                       # nothing to write

    # attention
    def attend(dtype=1, G=2, n_q=3, lens=0x9000, scale=0.1, q=0x1000, qs=(768, 256, 64), out=0x2000, os_=(768, 256, 64), ws=0x3000,
               room=1 << 30, cache=c):
        return LIB.chunkkv_q4_attention(cache, dtype, G, n_q, lens, scale, q, *qs, out, *os_, ws, room, None)
    assert attend(dtype=5) == attend(G=0) == attend(n_q=0) == attend(scale=0.0) == attend(scale=float("nan")) == INVALID
    assert attend(q=None) == attend(q=0x1002) == attend(out=None) == attend(ws=None) == attend(ws=0x3004) == attend(lens=0x9002) == INVALID
    assert attend(qs=(768, 7, 64)) == attend(qs=(768, 256, -64)) == attend(os_=(4, 256, 64)) == INVALID
    assert attend(cache=ctypes.byref(_struct(pages=None))) == attend(cache=None) == INVALID
    assert attend(room=16) == SMALL
    assert attend(G=1 << 16, n_q=1 << 15) == UNSUPPORTED
    empty = ctypes.byref(_struct(B=0))
    assert attend(cache=empty, q=None, out=None, ws=None) == OK                    # nothing to do
    assert ckv.chunkkv_launch_count() == n0


def test_binding_checks(ckv):
    cache = ckv.q4_cache(2, 2, 64, n_pages=8, max_pages=3, device="cpu")
    assert cache.pages[0].shape == (8, 4608) and ckv.q4_page_bytes(64) == 4608 and ckv.q4_page_bytes(65) == 9216
    assert ckv.q4_cache(1, 1, 80, n_pages=2, max_pages=3, device="cpu").pages[0].shape == (2, 9216)
    i32 = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: ckv.chunkkv_q4_resize(cache, i32.long()),
                 lambda: ckv.chunkkv_q4_resize(cache, i32[:3]),
                 lambda: ckv.chunkkv_q4_resize(cache, i32, torch.zeros(4, 3, dtype=torch.int32)),
                 lambda: ckv.chunkkv_q4_resize(cache, i32)):                       # host tensors
        with pytest.raises(ValueError):
            call()
    k, s5 = torch.zeros(2, 2, 5, 64), torch.zeros(4, 5, dtype=torch.int64)
    for a in ((k, k, i32, s5[:, :4]), (k, k.half(), i32, s5), (k[..., :32], k[..., :32], i32, s5), (k[0], k[0], i32, s5),
              (k, k.transpose(1, 2), i32, s5), (k, k, i32[:2], s5), (k, k, i32, s5)):
        with pytest.raises(ValueError):
            ckv.chunkkv_q4_append(cache, 0, *a)
    start = torch.zeros(4, dtype=torch.int64)
    for a in ((start, 5, k[0, 0], k[0, 0].half()), (start[:2], 5, k[0, 0], k[0, 0]), (start, 5, k[0], k[0]),
              (start, 5, k[0, 0], k[0, 0])):
        with pytest.raises(ValueError):
            ckv.chunkkv_q4_load(cache, 0, *a)
    q, ws = torch.zeros(2, 4, 64), torch.zeros(1 << 20, dtype=torch.uint8)
    q5 = torch.zeros(2, 5, 4, 64)
    for a in ((q[:, :3], q[:, :3]), (q, q[:, :2]), (q, q.half()), (q[0], q[0]), (q[..., :32], q[..., :32]), (q[:1], q[:1]),
              (q5, q5[:, :4]), (q5.transpose(2, 3), q5.transpose(2, 3)), (q, q)):
        with pytest.raises(ValueError):
            ckv.chunkkv_q4_attention(cache, 0, *a, ws)
    for lens in (torch.zeros(2), torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int64), torch.zeros(2, dtype=torch.int32)):
        with pytest.raises(ValueError):
            ckv.chunkkv_q4_attention(cache, 0, q5, q5, ws, q_lens=lens)
    with pytest.raises(ValueError):
        ckv.chunkkv_q4_workspace_size(cache, 4, 1, torch.float16)
    far = torch.zeros(4, dtype=torch.int32, device="meta")
    for kw in (dict(Hkv=3), dict(pages=[cache.pages[0][:, :4000]]), dict(pages=[cache.pages[0].to(torch.int8)]), dict(lens=far),
               dict(table=cache.table.long()), dict(d=128)):
        args = dict(B=2, Hkv=2, d=64, pages=cache.pages, table=cache.table, lens=cache.lens, ring=cache.ring, state=cache.state)
        args.update(kw)
        with pytest.raises(ValueError):
            ckv.Q4Cache(**args)
