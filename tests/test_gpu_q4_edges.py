"""The 4-bit cache's operators where hidden tokens, far apart values or extreme numbers could reach their results.

The definition, helpers and tolerances are those of test_gpu_q4.py; tolerances go by the tokens that a query sees.
"""
import math

import pytest
import torch

from test_gpu_q4 import BF, DEV, F32, ckv, fill, held, random_cache  # noqa: F401

pytestmark = pytest.mark.gpu


def check_query(ckv, cache, r, q, out, n, scale, path, spread=0, count=None):  # noqa: F811
    """One query token's heads q, out [G, d] against 64 bits over the first n tokens of cache row r.

    spread: in the kernel for many query rows, what shares a block of 128 tokens with the seen ones may raise its
    powers of two by this many bits (2^8 of the largest seen value, and one for where in an octave the two lie), so an
    element's error below f16's normal numbers is 2^(spread - 39) of the largest, a weight's 2^(spread - 28).
    count: of the n tokens, those whose weight counts (None: all).
    """
    (ks, km), (vs, vm) = held(cache, r, 0), held(cache, r, 1)
    ks, km, vs, vm = ks[:n], km[:n], vs[:n], vm[:n]
    qr, d = q.double(), q.shape[-1]
    p = torch.softmax(qr @ (ks + km).T * scale, -1)
    ref, A = p @ (vs + vm), p @ (vs + vm.abs())
    at = slice(None) if count is None else count
    E = (qr.abs() @ (ks + km.abs())[at].T * scale).amax(1, keepdim=True)
    tol = (2 * (d + 8) * 2.0 ** -22 * E + (n + 16) * 2.0 ** -22) * A + 1e-30
    if q.dtype == BF:
        tol = tol + 2.0 ** -8 * ref.abs() + (2.0 ** -11 + n * 2.0 ** -35) * A
    if path:
        kmax, vmax = (ks + km.abs())[at].max(), (vs + vm.abs())[at].max()
        small = 2.0 ** (spread - 39) * scale * qr.abs().sum(1, keepdim=True) * kmax
        tol = tol + (2 * (2.0 ** -11 * E + small) + 2.0 ** -11) * A + n * 2.0 ** (spread - 28) * vmax
    err = (out.double() - ref).abs()
    assert bool(torch.isfinite(out).all()) and bool((err <= tol).all()), \
        f"row {r}, {n} tokens: {float((err / tol).max())} of the tolerance"


# ------------------------------------------------------------------ what a query does not see

@pytest.mark.parametrize("power", [6, 20, 35, 60, 100])
@pytest.mark.parametrize("dtype,n_q,d,G", [(BF, 3, 128, 4), (BF, 5, 128, 4), (BF, 60, 128, 4), (BF, 90, 64, 2), (BF, 17, 80, 1), (F32, 5, 64, 2)])
def test_hidden_tokens_of_any_size_cost_the_others_nothing(ckv, dtype, n_q, d, G, power):  # noqa: F811
    lens = [300, n_q, 130, n_q + 1]
    at = n_q // 2                                     # the query token from which the large one is seen
    g = torch.Generator(device=DEV).manual_seed(n_q + d)
    q = torch.randn(2, n_q, 2 * G, d, generator=g, device=DEV).to(dtype)
    for which in (0, 1, 2):
        kv = [torch.randn(2, 2, 300, d, generator=g, device=DEV) for _ in range(2)]
        for r, n in enumerate(lens):
            for i in range(2):
                if which in (i, 2):
                    kv[i][r // 2, r % 2, n - n_q + at] *= 2.0 ** power
        cache = ckv.q4_cache(2, 2, d, n_pages=20, max_pages=6)
        fill(ckv, cache, lens, kv[0].to(dtype), kv[1].to(dtype))
        out = ckv.q4_attention(cache, 0, q)
        assert bool(torch.isfinite(out).all())
        path = ckv.chunkkv_q4_path(cache, G, n_q, dtype)
        for r, n in enumerate(lens):
            b, h = divmod(r, 2)
            for i in range(at):
                if n - n_q + 1 + i > 0:
                    heads = slice(h * G, (h + 1) * G)
                    check_query(ckv, cache, r, q[b, i, heads], out[b, i, heads], n - n_q + 1 + i, 1 / math.sqrt(d), path, spread=9)


@pytest.mark.parametrize("dtype,n_q,G", [(BF, 4, 4), (BF, 5, 4), (BF, 40, 7), (F32, 5, 2)])
def test_every_query_sees_a_larger_value_than_the_one_before(ckv, dtype, n_q, G):  # noqa: F811
    d, n = 128, 200
    g = torch.Generator(device=DEV).manual_seed(n_q)
    k, v = (torch.randn(1, 2, n, d, generator=g, device=DEV) for _ in range(2))
    v[:, :, n - n_q:] *= 2.0 ** (3.0 * torch.arange(n_q, device=DEV))[:, None]
    cache = ckv.q4_cache(1, 2, d, n_pages=10, max_pages=4)
    fill(ckv, cache, [n, n], k.to(dtype), v.to(dtype))
    q = torch.randn(1, n_q, 2 * G, d, generator=g, device=DEV).to(dtype)
    out = ckv.q4_attention(cache, 0, q)
    for h in range(2):
        for i in range(n_q):
            heads = slice(h * G, (h + 1) * G)
            check_query(ckv, cache, h, q[0, i, heads], out[0, i, heads], n - n_q + 1 + i, 1 / math.sqrt(d),
                        ckv.chunkkv_q4_path(cache, G, n_q, dtype), spread=9)


@pytest.mark.parametrize("dtype,G,n_q", [(BF, 4, 1), (F32, 4, 1), (BF, 4, 3), (BF, 4, 20), (BF, 4, 200)])
@pytest.mark.parametrize("cut", [384 + 37, 70, 600])
def test_value_steps_far_apart_inside_a_block(ckv, dtype, G, n_q, cut):  # noqa: F811
    # tokens up to `cut` (or from there on) hold values 2^r times the others' under weights below 2^-150 of theirs: one
    # block of 128 tokens holds both kinds
    d, n, powers = 64, 1000, [0, 20, 40, 60, 80]
    rows = 2 * len(powers)
    g = torch.Generator(device=DEV).manual_seed(62)
    cache = ckv.q4_cache(rows, 1, d, n_pages=rows * 16, max_pages=16)
    k = 0.1 * torch.randn(rows, 1, n, d, generator=g, device=DEV)
    v = torch.randn(rows, 1, n, d, generator=g, device=DEV)
    far = (torch.arange(n, device=DEV)[None] < cut) ^ (torch.arange(rows, device=DEV) % 2 == 1)[:, None]
    k[:, 0, :, 0] = torch.where(far, -150.0, 1.0)
    k[:, 0, :, 1] = torch.where(far, 150.0, 1.0)
    v *= torch.where(far, 2.0 ** torch.tensor(powers, device=DEV).repeat_interleave(2)[:, None], 1.0)[:, None, :, None]
    fill(ckv, cache, [n] * rows, k, v)
    q = torch.zeros(rows, n_q, G, d, device=DEV)
    q[..., 0] = 1 + torch.arange(G, device=DEV) / 16
    q = q.to(dtype)
    out = ckv.q4_attention(cache, 0, q, scale=1.0)
    for r in range(rows):
        for i in range(n_q):
            seen = n - n_q + 1 + i
            check_query(ckv, cache, r, q[r, i], out[r, i], seen, 1.0, ckv.chunkkv_q4_path(cache, G, n_q, dtype),
                        spread=9, count=~far[r, :seen])


# ------------------------------------------------------------------ weights and sums at far apart scales

@pytest.mark.parametrize("dtype,G,n_q", [(BF, 4, 1), (F32, 2, 1), (BF, 4, 3), (BF, 4, 20), (BF, 7, 60)])
@pytest.mark.parametrize("rows", [1, 40])
def test_equal_weights_of_values_far_apart(ckv, dtype, G, n_q, rows):  # noqa: F811
    # keys of zero, so equal weights: tokens up to `cut` (or from there on) hold 0 or small values and the others values of
    # 2^power; the former add nothing to the sum, and as much weight as the latter.  One row is cut into parts
    d, n = 128, 5120 if rows == 1 else 900
    for power in (0, 60, 66, 67, 70, 90, 100):
        for cut, low in ((n // 2 // 128 * 128, 0.0), (n // 2 // 128 * 128, 1.0), (200, 0.0), (n - 300, 2.0 ** -70)):
            for swap in (False, True):
                g = torch.Generator(device=DEV).manual_seed(power)
                cache = ckv.q4_cache(rows, 1, d, n_pages=rows * -(-n // 64), max_pages=-(-n // 64))
                v = 1.0 + torch.rand(1, 1, n, d, generator=g, device=DEV)
                small = (torch.arange(n, device=DEV) < cut) ^ swap
                v = (v * torch.where(small, low, 2.0 ** power)[:, None]).expand(rows, 1, n, d).contiguous().to(dtype)
                fill(ckv, cache, [n] * rows, torch.zeros_like(v), v)
                q = torch.randn(rows, n_q, G, d, generator=g, device=DEV).to(dtype)
                out = ckv.q4_attention(cache, 0, q).double()
                vs, vm = held(cache, 0, 1)
                total = (vs + vm).cumsum(0)
                seen = torch.arange(n - n_q, n, device=DEV)
                want = (total[seen] / (seen + 1)[:, None])[None, :, None]
                # weights and values in f16 (2^-11 each), the output's rounding (2^-8), n terms in fp32
                tol = ((n + 16) * 2.0 ** -22 + (2.0 ** -8 + 2.0 ** -10 if dtype == BF else 0)) * want
                assert bool(((out - want).abs() <= tol).all()), (power, cut, low, swap, float(((out - want).abs() / want).max()))


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


# ------------------------------------------------------------------ writing near the ends of the types

def step_of(lo, hi):
    """(m, s) of a group with these ends, by the definition: s is lowered where 15 s + m would be infinite."""
    m = lo.to(BF)
    m = torch.where(m.float() > lo, torch.nextafter(m, torch.full_like(m, -math.inf)), m).float()
    want = (hi - m) * torch.tensor(1.0 / 15.0, dtype=F32, device=lo.device)
    s = want.to(BF)
    s = torch.where(s.float() < want, torch.nextafter(s, torch.full_like(s, math.inf)), s)
    end = torch.tensor((2.0 - 2.0 ** -8) * 2.0 ** 127, dtype=torch.float64, device=lo.device)      # rounds to infinity in bf16
    limit = torch.where(hi.double() < end, end, end.new_tensor(2.0 ** 128 - 2.0 ** 103))           # and in fp32
    for _ in range(2):
        over = 15 * s.double() + m.double() >= limit
        s = torch.where(over, torch.nextafter(s, torch.zeros_like(s)), s)
    return m, s.float()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_finite_groups_read_back_finite(ckv, dtype):  # noqa: F811
    # values up to the type's largest: 15 s + m must not pass it
    d, n = 64, 512
    top = torch.finfo(dtype).max
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.rand(n, d, generator=g, device=DEV, dtype=torch.float64)
    scale = top * (1 - torch.rand(n, 1, generator=g, device=DEV, dtype=torch.float64) * 2.0 ** -8 * (torch.arange(n, device=DEV) % 3)[:, None])
    shift = torch.rand(n, 1, generator=g, device=DEV, dtype=torch.float64) * (torch.arange(n, device=DEV) % 4 > 1)[:, None]
    x = (shift + x * (1 - shift)) * scale             # from shift * scale up
    x[:, 7] = scale[:, 0]                             # the largest
    x[:64, 9] = 0.0
    x[64:80, 9] = -1.0
    x[80:96, 9] = -1e30
    x = x.to(dtype)
    k = x.float()[None, None]
    cache = ckv.q4_cache(1, 1, d, n_pages=8, max_pages=8)
    fill(ckv, cache, [n], k.to(dtype), -k.to(dtype))
    m, s = step_of(x.float().min(1).values, x.float().max(1).values)
    sc, km = held(cache, 0, 0)
    assert torch.equal(km[:, 0], m.double())
    codes = torch.round((x.float() - m[:, None]) * (1.0 / s[:, None]))
    assert float(codes.max()) <= 15 and torch.equal(sc, codes.double() * s[:, None].double())
    # half a step, and the rounding of x - m and of its product with 1 / s
    assert bool(((sc + km - x.double()).abs() <= s[:, None].double() * (0.5 + 16 * 2.0 ** -22)).all())
    outs = [torch.empty(n, d, dtype=dtype, device=DEV) for _ in range(2)]
    ckv.chunkkv_q4_load(cache, 0, torch.zeros(1, dtype=torch.int64, device=DEV), n, *outs)
    assert bool(torch.isfinite(outs[0]).all())
    # the other sign: a group whose smallest value is below bf16's lowest has an infinite m (-2^128 < x < -(2 - 2^-7) 2^127
    # rounds down to -inf), and so reads as NaN by the definition; all others are finite
    below = torch.isinf(step_of(-x.float().max(1).values, -x.float().min(1).values)[0])
    assert bool(outs[1][below].isnan().all()) and bool(torch.isfinite(outs[1][~below]).all())
    assert bool(below.any()) == (dtype == F32) and not bool(below.all())


# ------------------------------------------------------------------ which kernel a call takes

@pytest.mark.parametrize("n_q", [5, 33])
def test_repeated_axes_take_the_kernel_for_few_rows(ckv, n_q):  # noqa: F811
    # no tensor map can address a stride of zero: the other kernel's tolerance holds, whatever chunkkv_q4_path says of
    # strides that one can
    cache, g = random_cache(ckv, 2, 2, 64, [200, 70, 64, 130], seed=24)
    for shape in ((2, n_q, 1, 64), (1, n_q, 8, 64), (2, 1, 8, 64)):
        q = torch.randn(*shape, generator=g, device=DEV).to(BF).expand(2, n_q, 8, 64)
        out = ckv.q4_attention(cache, 0, q, out=torch.empty(2, n_q, 8, 64, dtype=BF, device=DEV))
        for r in range(4):
            b, h = divmod(r, 2)
            for i in range(n_q):
                n = int(cache.lens[r]) - n_q + 1 + i
                heads = slice(4 * h, 4 * h + 4)
                check_query(ckv, cache, r, q[b, i, heads], out[b, i, heads], n, 1 / 8, 0)


# ------------------------------------------------------------------ long sums in fp32

@pytest.mark.parametrize("d,G,n_q", [(128, 3, 1), (64, 4, 1), (128, 2, 2), (192, 2, 1)])
def test_long_fp32_sums_keep_fp32(ckv, d, G, n_q):  # noqa: F811
    # rows that one CTA sums over a hundred pages: the output's error as a whole, relative.  Three sources, independent from
    # token to token like the values that they weigh, each of about 2^-21 and of 2^-20 at most: a logit's rounding (d
    # products under partial sums of 3, 2^-25 each: sqrt(128) 3 2^-25), a weight's (22 bits, the exponential's 2 ulp),
    # and a page's sum (8 products whose sums are cut off, not rounded: 8 2^-24); adding the pages is rounded and less
    rows, n = 128, 8000
    cache, g = random_cache(ckv, rows // 2, 2, d, [n] * rows, seed=d, dtype=F32)
    q = torch.randn(rows // 2, n_q, 2 * G, d, generator=g, device=DEV)
    out = ckv.q4_attention(cache, 0, q).double()
    err = size = 0.0
    for r in range(0, rows, 5):
        b, h = divmod(r, 2)
        (ks, km), (vs, vm) = held(cache, r, 0), held(cache, r, 1)
        hidden = torch.arange(n, device=DEV)[None] > n - n_q + torch.arange(n_q, device=DEV)[:, None]
        for i in range(h * G, (h + 1) * G):
            t = (q[b, :, i].double() @ (ks + km).T / math.sqrt(d)).masked_fill(hidden, -math.inf)
            want = torch.softmax(t, -1) @ (vs + vm)
            err += float((out[b, :, i] - want).square().sum())
            size += float(want.square().sum())
    assert math.sqrt(err / size) <= 3 * 2.0 ** -20, math.sqrt(err / size)
