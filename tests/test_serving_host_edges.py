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
