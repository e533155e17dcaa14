"""The serving operators where a call's neighbours, earlier calls or extreme values could reach its results.

Formulas, helpers and tolerances are those of test_gpu_serving.py.
"""
import math

import pytest
import torch

from test_gpu_serving import (  # noqa: F401
    BF, DEV, F32, attention64, check_decode, check_prefill, ckv, fill, make_qkv, offsets, random_cache, read,
)

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


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("d,size", [(128, 4), (64, 4), (128, 8)])
def test_prefill_references_far_from_zero(ckv, d, size, split):  # noqa: F811
    # Exactly representable logits near size * 2^20 that differ by a few units between blocks of keys, so that
    # several blocks, and parts, of a row share the weight under references of their own.  In a row's last block
    # the last 32 keys lie 39 units lower (2^16.9 in weight), so a first reference taken there has to move.
    # Tolerance: logits exact, exponents below 40 in fp32 (2^-18 of a weight), sums and bf16 as elsewhere.
    T, rows, scale = 6000 if split else 960, 128, 0.3
    g = torch.Generator(device=DEV).manual_seed(size + d)
    q = torch.zeros(rows, 1, d, dtype=BF, device=DEV)
    k = torch.zeros(T, 1, d, dtype=BF, device=DEV)
    q[:, 0, 0] = 1024.0 * (1 + torch.arange(rows, device=DEV) / 128)
    q[:, 0, 1] = 1.0
    k[:, 0, 0] = 1024.0 * size
    blocks = (torch.arange(T, device=DEV) - (T - rows)).div(128, rounding_mode="floor") + T // 128 + 1
    up = torch.randint(0, 4, (T // 128 + 2,), generator=g, device=DEV)[blocks] + 40
    up[-32 - rows:] = 1
    k[:, 0, 1] = up.to(BF)
    v = torch.where(torch.rand(T // 128 + 2, 1, d, generator=g, device=DEV) < 0.5, -1.0, 1.0)[blocks].to(BF)
    cq, ck = [0, rows], [0, T]
    p, keep = ckv.prefill_params_for(q, k, cq, ck, scale=scale)
    ws = torch.zeros(ckv.chunkkv_prefill_workspace_size(p), dtype=torch.uint8, device=DEV)
    assert (ws.numel() > 1 << 16) == split
    out = torch.full_like(q, float("nan"))
    ckv.chunkkv_prefill_attention(p, q, k, v, out, ws)
    ckv.chunkkv_status_check(ws)
    ref, A, _ = attention64(q, k, v, scale)
    tol = (2.0 ** -18 + (T + 16) * 2.0 ** -23 + 2.0 ** -8) * A + 2.0 ** -8 * ref.abs()
    err = (out.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("dtype,d,T", [(BF, 128, 300), (BF, 64, 5000), (F32, 64, 300), (BF, 256, 100)])
def test_prefill_rows_of_minus_infinite_logits_alone(ckv, dtype, d, T):  # noqa: F811
    # the softmax of logits that are all -inf is NaN; a row without a key gives zeros
    rows = 40
    q, k, v = make_qkv([rows + 3], [T], 2, 1, d, dtype, seed=29)
    q = q.abs() + 0.01
    k = k.clone()
    k[:T - rows + 10, :, 0] = -float("inf")
    out = ckv.prefill_attention(q[:rows], k, v, [0, rows], [0, T])
    assert bool(out[:10].isnan().all()) and bool(torch.isfinite(out[10:]).all())
    # three queries more than keys
    k[:, :, 0] = -float("inf")
    out = ckv.prefill_attention(q, k[:rows], v[:rows], [0, rows + 3], [0, rows])
    assert bool((out[:3] == 0).all()) and bool(out[3:].isnan().all())


# ------------------------------------------------------------------ 8-bit cache

@pytest.mark.parametrize("dtype", [BF, F32])
def test_load_stays_inside_its_outputs(ckv, dtype):  # noqa: F811
    # rows that would end past the outputs, begin there, or begin nowhere near; the rows behind are left alone
    lens = [130, 70, 64, 5, 300]
    cache, _ = random_cache(ckv, 1, 5, 64, lens, seed=95)
    rows = read(ckv, cache, dtype)
    begin = [180, 0, 250, 1 << 40, 100]
    wide = torch.full((2, 1000, 64), 5.0, dtype=dtype, device=DEV)
    k, v = wide[0, 100:300], wide[1, 100:300]
    for r in range(5):
        wide.fill_(5.0)
        start = torch.tensor([b if i == r else -1 for i, b in enumerate(begin)], dtype=torch.int64, device=DEV)
        ckv.chunkkv_q8_load(cache, 0, start, 200, k, v)
        n = max(0, min(lens[r], 200, 200 - begin[r]))
        want = torch.full_like(wide, 5.0)
        if n:
            for i in range(2):
                want[i, 100 + begin[r]:100 + begin[r] + n] = rows[r][i][:n]
        assert torch.equal(wide, want), r


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_rows_of_no_sequence(ckv, dtype):  # noqa: F811
    # rows of q behind the last offset: zeros where the binding makes the output, whatever its memory held
    q, k, v = make_qkv([60], [60], 4, 2, 64, dtype, seed=33)
    for last in (40, 0):
        dirt = [torch.full_like(q, float("nan")) for _ in range(8)]
        del dirt
        out = ckv.prefill_attention(q, k, v, [0, last])
        check_prefill(out[:last], q[:last], k[:last], v[:last], [0, last], [0, last], 1 / 8, dtype == BF)
        assert bool((out[last:] == 0).all())
        mine = torch.full_like(q, 7.0)
        ckv.prefill_attention(q, k, v, [0, last], out=mine)
        assert torch.equal(mine[:last], out[:last]) and bool((mine[last:] == 7.0).all())


@pytest.mark.parametrize("tq,T,Hq,Hkv,d", [(1, 9000, 8, 2, 128), (3, 5000, 4, 1, 64), (130, 6000, 2, 1, 128), (40, 700, 2, 2, 128)])
def test_prefill_counts_every_key_once(ckv, tq, T, Hq, Hkv, d):  # noqa: F811
    # equal weights, and a value of 1 in column c for key w + c: each of the last row's outputs is 1 / T
    q = torch.zeros(tq, Hq, d, dtype=BF, device=DEV)
    k = torch.zeros(T, Hkv, d, dtype=BF, device=DEV)
    p, keep = ckv.prefill_params_for(q, k, [0, tq], [0, T])
    ws = torch.zeros(ckv.chunkkv_prefill_workspace_size(p), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(q)
    sees = torch.arange(tq, device=DEV) + (T - tq + 1)                       # keys that a row sees
    for w in range(0, T, d):
        n = min(d, T - w)
        v = torch.zeros(T, Hkv, d, dtype=BF, device=DEV)
        v[w + torch.arange(n), :, torch.arange(n)] = 1
        ckv.chunkkv_prefill_attention(p, q, k, v, out, ws)
        want = ((w + torch.arange(d, device=DEV) < sees[:, None]) & (torch.arange(d, device=DEV) < n)) / sees[:, None].double()
        # weights that are equal and exact in bf16, their sum in fp32, the output's rounding
        assert bool(((out.double() - want[:, None]).abs() <= (2.0 ** -8 + (T + 16) * 2.0 ** -23) * want[:, None]).all()), w


@pytest.mark.parametrize("tq,T", [(1, 9000), (70, 6000)])
def test_prefill_one_key_of_a_split_row_takes_all(ckv, tq, T):  # noqa: F811
    # the winner on both sides of every boundary of two blocks of keys, and so of two parts
    q = torch.zeros(tq, 2, 128, dtype=BF, device=DEV)
    q[:, :, 0] = 64.0
    v = torch.randn(T, 1, 128, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV).to(BF)
    k = torch.zeros(T, 1, 128, dtype=BF, device=DEV)
    p, keep = ckv.prefill_params_for(q, k, [0, tq], [0, T], scale=1.0)
    ws = torch.zeros(ckv.chunkkv_prefill_workspace_size(p), dtype=torch.uint8, device=DEV)
    assert ws.numel() > 1 << 16
    out = torch.empty_like(q)
    for at in [x for b in range(0, T - tq, 128) for x in (b - 1, b) if x >= 0] + [T - tq]:
        k[at, 0, 0] = 64.0
        ckv.chunkkv_prefill_attention(p, q, k, v, out, ws)
        assert torch.equal(out, v[at].expand(tq, 2, 128)), at
        k[at, 0, 0] = 0.0


@pytest.mark.parametrize("kind", ["large", "nan", "zero"])
@pytest.mark.parametrize("dtype,d,tq,tk", [(BF, 128, 700, 700), (BF, 64, 300, 900), (BF, 128, 40, 6000), (F32, 64, 200, 300)])
def test_prefill_rows_keep_their_bits_whatever_others_ask(ckv, dtype, d, tq, tk, kind):  # noqa: F811
    # another query for some rows (one that moves its reference, or has no finite logit) changes those rows alone
    q, k, v = make_qkv([tq], [tk], 4, 2, d, dtype, seed=43)
    want = ckv.prefill_attention(q, k, v, [0, tq], [0, tk])
    other = q.clone()
    hit = torch.zeros(tq, 4, dtype=torch.bool, device=DEV)
    hit[3::37, 1] = True
    hit[11::53] = True
    other[hit] = {"large": q[hit] * 60, "nan": torch.full_like(q[hit], float("nan")), "zero": q[hit] * 0}[kind]
    out = ckv.prefill_attention(other, k, v, [0, tq], [0, tk])
    assert torch.equal(out[~hit], want[~hit])
    assert bool(out[hit].isnan().all()) == (kind == "nan") and not torch.equal(out[hit], want[hit])


# ------------------------------------------------------------------ decode attention

@pytest.mark.parametrize("between,heads", [("prompt", (4, 12, 20, 130)), ("scoring", (4, 8, 1))])
def test_decode_workspace_serves_any_calls_in_turn(ckv, between, heads):  # noqa: F811
    # one workspace for caches of other shapes, other numbers of heads, and a split prompt (or, for up to 8 heads,
    # the compression's scoring) between them
    d = 128
    small, g = random_cache(ckv, 2, 4, d, [6000 + 100 * i for i in range(8)], seed=51)
    large, _ = random_cache(ckv, 64, 8, d, [600 + (i * 97) % 700 for i in range(512)], seed=52)
    narrow, _ = random_cache(ckv, 3, 1, 64, [5000, 40, 2000], seed=53)
    pq, pk, pv = make_qkv([20], [9000], 8, 2, d, BF, seed=54)
    p, keep = ckv.prefill_params_for(pq, pk, [0, 20], [0, 9000])
    want = ckv.prefill_attention(pq, pk, pv, [0, 20], [0, 9000])
    window, sk, _ = make_qkv([16], [3000], 8, 2, d, BF, seed=55)
    sp, keep_s = ckv.params_for(window[None], sk, [0, 3000], Hkv=2, w=16, c=10, L_max=100)
    scores = torch.zeros(1, 2, ckv.chunkkv_out_capacity(sp)[1], device=DEV)
    ws = torch.zeros(max([ckv.chunkkv_q8_workspace_size(c, G) for c in (small, large, narrow) for G in heads]
                         + [ckv.chunkkv_prefill_workspace_size(p), ckv.chunkkv_workspace_size(sp)]),
                     dtype=torch.uint8, device=DEV)
    for G in heads:
        for cache in (small, large, narrow, large):
            q = torch.randn(cache.B, cache.Hkv * G, cache.d, generator=g, device=DEV).to(BF)
            out = torch.full_like(q, float("nan"))
            ckv.chunkkv_q8_attention(cache, 0, q, out, ws)
            ckv.chunkkv_status_check(ws)
            check_decode(ckv, cache, q, out, 1 / math.sqrt(cache.d))
            if between == "prompt":
                prompt = torch.full_like(pq, float("nan"))
                ckv.chunkkv_prefill_attention(p, pq, pk, pv, prompt, ws)
                assert torch.equal(prompt, want)
            else:
                ckv.chunkkv_score(sp, window, sk, scores, ws)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,G", [(128, 4), (256, 2)])
def test_decode_value_scales_far_apart(ckv, dtype, d, G):  # noqa: F811
    # Half of a row's pages hold values 2^r times the others' under weights below 2^-190 of theirs; the pages of a
    # kind lie together (so that a warp has both kinds), in either order.  Tolerance as in check_decode with the
    # logits of the keys that count.
    rows, n = 320, 16 * 64
    g = torch.Generator(device=DEV).manual_seed(61)
    cache = ckv.q8_cache(rows, 1, d, n_pages=rows * 16, max_pages=16)
    k = torch.randn(rows, 1, n, d, generator=g, device=DEV)
    k[..., 0] = torch.rand(rows, 1, n, generator=g, device=DEV)
    v = torch.randn(rows, 1, n, d, generator=g, device=DEV)
    r = torch.tensor([0.0, 20.0, 30.0, 40.0, 60.0, 90.0], device=DEV)[torch.arange(rows, device=DEV) // 2 % 6]
    far = (torch.arange(n, device=DEV)[None] < n // 2) ^ (torch.arange(rows, device=DEV) % 2 == 1)[:, None]
    k[:, 0, :, 0] = torch.where(far, -140.0, k[:, 0, :, 0])
    v *= torch.where(far, 2.0 ** r[:, None], 1.0)[:, None, :, None]
    fill(ckv, cache, [n] * rows, k, v)
    q = torch.zeros(rows, G, d, device=DEV)
    q[:, :, 0] = 1 + torch.arange(G, device=DEV) / 4
    q = q.to(dtype)
    out = ckv.q8_attention(cache, 0, q, scale=1.0)
    for i, (kr, vr) in enumerate(read(ckv, cache, F32)):
        near = ~far[i]
        qi, ki, vi = q[i].double(), kr.double(), vr.double()
        p = torch.softmax(qi @ ki.T, -1)
        ref, A = p @ vi, p @ vi.abs()
        E = (qi.abs() @ ki[near].abs().T).amax(1, keepdim=True)
        tol = (2 * (d + 4) * 2.0 ** -22 * E + (n + 16) * 2.0 ** -22) * A + (2.0 ** -8 * ref.abs() if dtype == BF else 0)
        err = (out[i].double() - ref).abs()
        assert bool((err <= tol).all()), f"2^{int(r[i])}, row {i}: {float((err / tol).max())} of the tolerance"


def test_calls_refuse_tensors_outside_the_gpu(ckv):  # noqa: F811
    # one argument at a time in host memory: an error on the host, and nothing is launched
    cache, _ = random_cache(ckv, 1, 2, 64, [70, 5], seed=91)
    i32, i64 = torch.zeros(2, dtype=torch.int32, device=DEV), torch.zeros(2, 4, dtype=torch.int64, device=DEV)
    k = torch.zeros(1, 2, 4, 64, device=DEV)
    start, rows = torch.zeros(2, dtype=torch.int64, device=DEV), torch.zeros(100, 64, device=DEV)
    q, ws = torch.zeros(1, 4, 64, device=DEV), torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
    p, keep = ckv.prefill_params_for(rows[:, None], rows[:, None], [0, 100])
    calls = [(lambda n, s: ckv.chunkkv_q8_resize(cache, n, s), (i32, i64)),
             (lambda k, v, n, s: ckv.chunkkv_q8_append(cache, 0, k, v, n, s), (k, k, i32, i64)),
             (lambda s, k, v: ckv.chunkkv_q8_load(cache, 0, s, 4, k, v), (start, rows, rows)),
             (lambda q, o, w: ckv.chunkkv_q8_attention(cache, 0, q, o, w), (q, q.clone(), ws)),
             (lambda *a: ckv.chunkkv_prefill_attention(p, *a), (rows[:, None],) * 4 + (ws,))]
    torch.cuda.synchronize()
    before = ckv.chunkkv_launch_count()
    for call, args in calls:
        for i in range(len(args)):
            with pytest.raises(ValueError):
                call(*args[:i], args[i].cpu(), *args[i + 1:])
    assert ckv.chunkkv_launch_count() == before


@pytest.mark.parametrize("lens", [[6582] * 8, [800, 900], [577, 64, 4000, 1, 1300], [3000] * 40])
def test_decode_counts_every_token_once(ckv, lens):  # noqa: F811
    # zero keys, so equal weights; a value code of 127 in column c for token w + c gives 127 / n there
    d, rows = 128, len(lens)
    cache, g = random_cache(ckv, rows, 1, d, lens, seed=71)
    cache.k_pages[0].zero_()
    cache.scales[0].fill_(1.0)
    q = torch.randn(rows, 2, d, generator=g, device=DEV)
    ws = torch.zeros(ckv.chunkkv_q8_workspace_size(cache, 2), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(q)
    n = torch.tensor(lens, device=DEV)[:, None, None]
    for w in range(0, max(lens), d):
        cache.v_pages[0].zero_()
        for half in (0, 64):
            j = (w + half) // 64
            has = [r for r in range(rows) if lens[r] > w + half]
            if has:
                page = cache.table[has, j].long()
                cache.v_pages[0][page[:, None], torch.arange(64, device=DEV) + half, torch.arange(64, device=DEV)] = 127
        ckv.chunkkv_q8_attention(cache, 0, q, out, ws)
        want = (w + torch.arange(d, device=DEV) < n) * (127.0 / n.double())
        assert bool(((out.double() - want).abs() <= (n + 16) * 2.0 ** -22 * want).all()), w


@pytest.mark.parametrize("rows,n", [(8, 6582), (2, 800), (3, 2500)])
def test_decode_one_token_takes_all(ckv, rows, n):  # noqa: F811
    # the dominant key at the first and the last token of every page, and so of every run of pages
    d = 64
    cache, g = random_cache(ckv, rows, 1, d, [n] * rows, seed=81)
    cache.k_pages[0].zero_()
    cache.scales[0].fill_(1.0)
    q = torch.zeros(rows, 4, d, device=DEV)
    q[:, :, 0] = 4.0
    ws = torch.zeros(ckv.chunkkv_q8_workspace_size(cache, 4), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(q)
    spots = [x for j in range(-(-n // 64)) for x in (64 * j, min(64 * j + 63, n - 1))]
    row = torch.arange(rows, device=DEV)
    for i in range(len(spots)):
        at = torch.tensor([spots[(i + r * 31) % len(spots)] for r in range(rows)], device=DEV)
        page = cache.table[row, at // 64].long()
        cache.k_pages[0][page, 0, at % 64, 0] = 100
        ckv.chunkkv_q8_attention(cache, 0, q, out, ws, 1.0)
        want = cache.v_pages[0][page, :, at % 64].double()                   # [rows, d]
        assert bool(((out.double() - want[:, None]).abs() <= 2.0 ** -20 * want[:, None].abs()).all()), i
        cache.k_pages[0][page, 0, at % 64, 0] = 0


@pytest.mark.parametrize("kind", ["large", "nan"])
def test_decode_heads_keep_their_bits_whatever_others_ask(ckv, kind):  # noqa: F811
    cache, g = random_cache(ckv, 3, 2, 128, [3000, 70, 1, 900, 64, 2000], seed=97, spread=2.0)
    q = torch.randn(3, 12, 128, generator=g, device=DEV)
    want = ckv.q8_attention(cache, 0, q)
    other = q.clone()
    other[:, 2::6] = q[:, 2::6] * 60 if kind == "large" else float("nan")
    out = ckv.q8_attention(cache, 0, other)
    rest = [h for h in range(12) if h % 6 != 2]
    assert torch.equal(out[:, rest], want[:, rest])
