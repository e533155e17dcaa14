"""Refusals of the serving operators that keep a call from memory it must not touch; nothing is launched."""
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ckv():
    if not os.path.exists(os.path.join(ROOT, "chunk_level_kv_gb300", "libchunkkv.so")):
        import __graft_entry__
        __graft_entry__.build()
    import chunk_level_kv_gb300 as m
    return m


class On:
    """A tensor as far as its device goes."""

    def __init__(self, device: int):
        self.device = device

    def get_device(self) -> int:
        return self.device


def test_a_call_takes_tensors_of_the_current_gpu(ckv, monkeypatch):
    from chunk_level_kv_gb300 import serve
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 100 + dev, raising=False)
    assert serve._stream(On(1), On(1), On(1)) == 101
    for tensors in ([On(-1)], [On(1), On(-1)], [On(1), On(1), On(0)], [On(0)], [On(0), On(0)]):
        with pytest.raises(ValueError):
            serve._stream(*tensors)


def test_a_cache_lies_on_one_device(ckv):
    c = ckv.q8_cache(2, 2, 64, n_pages=8, max_pages=3, device="cpu")
    far = torch.zeros(4, dtype=torch.int32, device="meta")
    with pytest.raises(ValueError):
        ckv.Q8Cache(B=2, Hkv=2, d=64, k_pages=c.k_pages, v_pages=c.v_pages, scales=c.scales, table=c.table, lens=far,
                    ring=c.ring, state=c.state)


def test_load_bounded_arguments(ckv):
    import ctypes

    from chunk_level_kv_gb300._lib import LIB, Q8CacheStruct
    OK, INVALID = 0, 1
    before = ckv.chunkkv_launch_count()
    c = Q8CacheStruct(B=2, Hkv=2, d=64, n_pages=10, max_pages=4, k_pages=0x10000, v_pages=0x20000, scales=0x30000,
                      table=0x40000, lens=0x50000, ring=0x60000, state=0x70000)

    def load(start=0x1000, n_cap=3, n_rows=10, k=0x1000, st=64):
        return LIB.chunkkv_q8_load_bounded(ctypes.byref(c), 1, start, n_cap, n_rows, k, 0x2000, st, None)
    assert load(start=None) == load(n_cap=-1) == load(n_rows=-1) == load(k=None) == load(st=9) == INVALID
    assert load(n_rows=0, k=None) == OK                                      # nothing to write
    assert ckv.chunkkv_launch_count() == before


def test_slot_maps_beyond_the_counters(ckv):
    # as for the append: runs of a row are counted in 32 bits
    import ctypes

    from chunk_level_kv_gb300._lib import LIB, Q8CacheStruct
    UNSUPPORTED = 2
    c = Q8CacheStruct(B=2, Hkv=2, d=64, n_pages=10, max_pages=4, k_pages=0x10000, v_pages=0x20000, scales=0x30000,
                      table=0x40000, lens=0x50000, ring=0x60000, state=0x70000)
    for n_cap in (2147483647, 2147483647 - 255):
        assert LIB.chunkkv_q8_resize(ctypes.byref(c), 0x1000, 0x2000, n_cap, None) == UNSUPPORTED


def test_offsets_that_pass_32_bits(ckv):
    # an offset must not wrap into a small one on its way into the library
    q = torch.zeros(10, 2, 64)
    for cu in ([0, (1 << 32) + 3, 10], [0, -(1 << 32) + 3, 10]):
        with pytest.raises(ValueError):
            ckv.prefill_params_for(q, q, cu)
        with pytest.raises(ValueError):
            ckv.prefill_params_for(q, q, [0, 3, 10], cu)
    ckv.prefill_params_for(q, q, [0, 3, 10])
