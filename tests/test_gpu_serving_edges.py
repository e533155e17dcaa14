"""The serving operators where a call's neighbours, earlier calls or extreme values could reach its results.

Formulas, helpers and tolerances are those of test_gpu_serving.py.
"""
import math

import pytest
import torch

from test_gpu_serving import BF, DEV, F32, check_prefill, ckv, make_qkv, offsets  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ prefill attention

@pytest.mark.parametrize("Hq,Hkv,d,long", [(1, 1, 128, 0), (4, 4, 64, 0), (8, 2, 128, 0), (2, 2, 128, 4)])
def test_prefill_masked_items_after_unmasked_ones(ckv, Hq, Hkv, d, long):  # noqa: F811
    # Items whose blocks hold no hidden key (a position on exactly 256 keys, or on 19200) come before items
    # that share their last block with rows of non-finite values: those rows belong to sequences without queries
    # and reach nobody, whatever a CTA did before.
    n = 300
    tq, tk, dirty = [], [], []
    for i in range(n):
        tq += [1, 1, 0]
        tk += [256, 200, 60]
        dirty.append(3 * i + 2)
    tq += [1] * long
    tk += [19200] * long
    q, k, v = make_qkv(tq, tk, Hq, Hkv, d, BF, seed=41)
    cq, ck = offsets(tq), offsets(tk)
    clean = ckv.prefill_attention(q, k, v, cq, ck)
    check_prefill(clean, q, k, v, cq, ck, 1 / math.sqrt(d), 1)
    for bad in (float("nan"), float("inf")):
        vb = v.clone()
        for i in dirty:
            vb[ck[i]:ck[i + 1]] = bad
        for _ in range(20):
            assert torch.equal(ckv.prefill_attention(q, k, vb, cq, ck), clean)
