"""The 4-bit cache's operators where hidden tokens, far apart values or extreme numbers could reach their results.

The definition, helpers and tolerances are those of test_gpu_q4.py; tolerances go by the tokens that a query sees.
"""
import math

import pytest
import torch

from test_gpu_q4 import BF, DEV, F32, ckv, fill, held  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ weights and sums at far apart scales

@pytest.mark.parametrize("dtype,G,n_q", [(BF, 4, 1), (F32, 2, 1), (BF, 4, 3), (BF, 4, 20), (BF, 4, 150)])
def test_the_largest_of_huge_logits_wins(ckv, dtype, G, n_q):  # noqa: F811
    # logits of about 2^power (as exponents of 2) at one token a row and a half of it and less at the others: its value is the
    # output, wherever it lies
    d, n = 128, 2500
    powers = [18, 22, 24, 26, 28, 30, 34, 60, 100]
    at = [0, 127, 128, 500, 1279, 1600, 2000, 2303, 2304, n - n_q]
    rows = len(powers) * len(at)
    g = torch.Generator(device=DEV).manual_seed(9)
    cache = ckv.q4_cache(rows, 1, d, n_pages=rows * 40, max_pages=40)
    k = 0.5 * torch.rand(rows, 1, n, 1, generator=g, device=DEV)
    r = torch.arange(rows, device=DEV)
    k[r, 0, torch.tensor(at, device=DEV).repeat(len(powers))] = 1.0
    k = k * (0.9 + 0.2 * torch.rand(rows, 1, 1, d, generator=g, device=DEV))
    v = torch.randn(rows, 1, n, d, generator=g, device=DEV).to(dtype)
    fill(ckv, cache, [n] * rows, k.to(dtype), v)
    q = 0.9 + 0.2 * torch.rand(rows, n_q, G, d, generator=g, device=DEV)
    q *= 2.0 ** torch.tensor(powers, device=DEV).repeat_interleave(len(at))[:, None, None, None]
    out = ckv.q4_attention(cache, 0, q.to(dtype), scale=1.3 * math.log(2.0) / d).double()
    for i in range(rows):
        vs, vm = held(cache, i, 1)
        want = (vs + vm)[at[i % len(at)]]
        tol = ((2.0 ** -8 + 2.0 ** -10 if dtype == BF else 0) + 2.0 ** -18) * (vs + vm.abs())[at[i % len(at)]]
        err = (out[i] - want).abs()
        assert bool((err <= tol).all()), (powers[i // len(at)], at[i % len(at)], float((err / tol).max()))
