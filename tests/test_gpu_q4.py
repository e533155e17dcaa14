"""The 4-bit cache on the GPU, against plain implementations written from its definitions.

Codes, steps and smallest values are compared byte by byte with a restatement of the definition; what is read back
with s * c + m rounded once.  Attention is held to 64 bits over s * c + m; tolerances per output element, with
A = sum_j softmax_j (s c + |m|) and E = max_j scale * sum_e |q_e| (s c + |m|)_je over the tokens that the row sees:
  logits   fp32 sums of d products, the query in 22 bits (fp32) or exactly but for 2^-25 of its largest element (bf16):
           each off by at most (d + 8) 2^-22 E, which moves a weight and the row's sum by that factor each
  sums     n terms in fp32 and a few ulp of the exponential: (n + 16) 2^-22 A; fp32 weights in 22 bits are within that
  bf16     the weights p s rounded to f16: 2^-11 A (those below 2^-28 of the largest to 2^-39 of it: n 2^-35 A);
           the output's rounding 2^-8 |o|
  many query rows (chunkkv_q4_path 1): keys, values and weights rounded to f16, 2^-11 each: a logit is off by 2^-11 E
           more, and the output by 2 * 2^-11 A; what is below 2^-14 in f16 has an error of 2^-25 there: of a weight
           2^-29 of the reference's (times n and the largest value), of an element 2^-39 of its block's largest
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ckv():
    import chunk_level_kv_gb300 as m     # fails loudly if the library was not built
    return m


def offsets(ns):
    out = [0]
    for n in ns:
        out.append(out[-1] + n)
    return out


# ------------------------------------------------------------------ the definition, restated

def quantise(x):
    """(codes, m, s) of tokens x [n, d], group by group, in the arithmetic that the definition names."""
    codes, ms, steps = [], [], []
    for a in range(0, x.shape[1], 64):
        y = x[:, a:a + 64].float()
        lo, hi = y.min(1).values, y.max(1).values
        m = lo.to(BF)
        m = torch.where(m.float() > lo, torch.nextafter(m, torch.full_like(m, -math.inf)), m).float()
        span = hi - m
        want = span * torch.tensor(1.0 / 15.0, dtype=F32, device=x.device)
        s = want.to(BF)
        s = torch.where(s.float() < want, torch.nextafter(s, torch.full_like(s, math.inf)), s).float()
        s = torch.where(span >= 2.0 ** -100, s, 0.0)
        bad = ~torch.isfinite(span)
        c = torch.where(s[:, None] > 0, torch.round((y - m[:, None]) * (1.0 / s[:, None])).clamp(0, 15), 0.0)
        codes.append(torch.where(bad[:, None], 0.0, c))
        ms.append(torch.where(bad, math.nan, m))
        steps.append(torch.where(bad, 0.0, s))
    return codes, torch.stack(ms, 1), torch.stack(steps, 1)


def held(cache, r, which, layer=0):
    """Row r's keys (0) or values (1) from the bytes: s c and m for every element, [n, d] in 64 bits."""
    d, nd, n = cache.d, -(-cache.d // 64), int(cache.lens[r])
    raw = cache.pages[layer][cache.table[r, :-(-n // 64)].long()].long()
    item = torch.arange(16, device=DEV)
    w, p, e = item // 8, item % 8 // 2, item % 2
    nib = p + 4 * e
    byte, up = 4 * w + nib // 2, 4 * (nib % 2)
    token, col = torch.arange(64, device=DEV)[:, None], torch.arange(d, device=DEV)[None]
    if which == 0:
        at = ((token * 4 + col % 64 // 16) * nd + col // 64) * 8 + byte[col % 16]
        code = raw[:, at] >> up[col % 16] & 15
    else:
        at = 2304 * nd + (((col // 16 * 8 + col % 8) * 4 + token // 16) * 2 + col % 16 // 8) * 8 + byte[token % 16]
        code = raw[:, at] >> up[token % 16] & 15
    ms = (2048 if which == 0 else 4352) * nd + ((col // 64) * 64 + token) * 4

    def bf16(at):
        return ((raw[:, at] | raw[:, at + 1] << 8) << 16).to(torch.int32).view(F32).double()
    sc = (code.double() * bf16(ms + 2)).reshape(-1, d)[:n]
    return sc, bf16(ms).reshape(-1, d)[:n]


def fill(ckv, cache, new_lens, k, v, layer=0):
    """Grows the cache to new_lens with the rows of k, v [B, Hkv, n_cap, d]; returns the counts."""
    lens = cache.lens.clone()
    new = torch.tensor(new_lens, dtype=torch.int32, device=DEV)
    slots = torch.empty(cache.rows, k.shape[2], dtype=torch.int64, device=DEV)
    ckv.chunkkv_q4_resize(cache, new, slots)
    assert cache.state[2].item() == 0
    counts = (new - lens).contiguous()
    ckv.chunkkv_q4_append(cache, layer, k, v, counts, slots)
    return counts


def read(ckv, cache, dtype, layer=0):
    lens = cache.lens.tolist()
    at = offsets(lens)
    k = torch.full((max(at[-1], 1), cache.d), 9.0, dtype=dtype, device=DEV)
    v = torch.full_like(k, 9.0)
    start = torch.tensor(at[:-1], dtype=torch.int64, device=DEV)
    ckv.chunkkv_q4_load(cache, layer, start, max(max(lens), 1), k, v)
    return [(k[a:b], v[a:b]) for a, b in zip(at, at[1:])]


# ------------------------------------------------------------------ writing and reading back

@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (BF, 80), (BF, 8), (BF, 256), (F32, 128), (F32, 192), (F32, 72), (F32, 8)])
def test_append_and_load(ckv, dtype, d):
    B, Hkv = 2, 3
    g = torch.Generator(device=DEV).manual_seed(d)
    cache = ckv.q4_cache(B, Hkv, d, n_pages=40, max_pages=6)
    cache.ring.copy_(torch.randperm(40, generator=g, device=DEV).int())
    cache.pages[0].fill_(0xA5)                        # stale bytes
    rows = [(torch.empty(0, d, device=DEV), torch.empty(0, d, device=DEV)) for _ in range(B * Hkv)]
    for new in ([0, 1, 64, 65, 130, 200], [3, 2, 65, 65, 190, 331], [63, 64, 129, 70, 191, 332]):
        had = cache.lens.tolist()
        n = max(max(b - a for a, b in zip(had, new)), 1)
        grow = torch.exp(2 * torch.randn(B, Hkv, n, 1, generator=g, device=DEV))
        k = (torch.randn(B, Hkv, n, d, generator=g, device=DEV) * grow).to(dtype)
        v = (torch.randn(B, Hkv, n, d, generator=g, device=DEV) + 3.0).to(dtype)
        fill(ckv, cache, new, k, v)
        rows = [tuple(torch.cat([x, y[r // Hkv, r % Hkv, :new[r] - had[r]].float()]) for x, y in zip(rows[r], (k, v)))
                for r in range(B * Hkv)]
        for r in range(B * Hkv):
            for i in range(2):
                x = rows[r][i]
                if len(x) == 0:
                    continue
                sc, m = held(cache, r, i)
                codes, ms, steps = quantise(x)
                for p, a in enumerate(range(0, d, 64)):
                    s = steps[:, p:p + 1].double()
                    assert torch.equal(m[:, a:a + 64], ms[:, p:p + 1].double().expand_as(codes[p]))
                    assert torch.equal(sc[:, a:a + 64], codes[p].double() * s)
                    # half a step, and the rounding of x - m and of its product with 1 / s
                    err = (sc[:, a:a + 64] + m[:, a:a + 64] - x[:, a:a + 64].double()).abs()
                    assert bool((err <= s * (0.5 + 16 * 2.0 ** -22)).all())
        for out in (dtype, F32):
            for r, (kr, vr) in enumerate(read(ckv, cache, out)):
                for i, got in ((0, kr), (1, vr)):
                    if len(got):
                        sc, m = held(cache, r, i)
                        assert torch.equal(got, (sc.float() + m.float()).to(out)), (r, i)      # s c is exact in fp32


def test_append_token_by_token_is_append_at_once(ckv):
    B, Hkv, d, n = 2, 2, 80, 70
    g = torch.Generator(device=DEV).manual_seed(5)
    k, v = (torch.randn(B, Hkv, n, d, generator=g, device=DEV).to(BF) for _ in range(2))
    caches = [ckv.q4_cache(B, Hkv, d, n_pages=8, max_pages=2) for _ in range(2)]
    fill(ckv, caches[0], [n] * 4, k, v)
    fill(ckv, caches[1], [2] * 4, k[:, :, :2], v[:, :, :2])
    for i in range(2, n):
        fill(ckv, caches[1], [i + 1] * 4, k[:, :, i:i + 1], v[:, :, i:i + 1])
    for r in range(4):
        for i in range(2):
            for a, b in zip(held(caches[0], r, i), held(caches[1], r, i)):
                assert torch.equal(a, b)


def test_append_strides_and_slots_of_a_failed_resize(ckv):
    # k and v as parts of one projection, tokens before heads; and a map of -1 writes nothing
    B, Hkv, n, d = 2, 2, 70, 64
    g = torch.Generator(device=DEV).manual_seed(8)
    kv = torch.randn(B, n, 2 * Hkv, d, generator=g, device=DEV).to(BF)
    k, v = kv[:, :, :Hkv].transpose(1, 2), kv[:, :, Hkv:].transpose(1, 2)
    a, b = (ckv.q4_cache(B, Hkv, d, n_pages=8, max_pages=2) for _ in range(2))
    fill(ckv, a, [n, 3, 64, 0], k, v)
    fill(ckv, b, [n, 3, 64, 0], k.contiguous(), v.contiguous())
    assert torch.equal(a.pages[0], b.pages[0])
    before = a.pages[0].clone()
    slots = torch.empty(4, n, dtype=torch.int64, device=DEV)
    ckv.chunkkv_q4_resize(a, torch.full((4,), 10000, dtype=torch.int32, device=DEV), slots)
    assert a.state[2].item() == 2 and bool((slots == -1).all())
    ckv.chunkkv_q4_append(a, 0, k, v, torch.full((4,), n, dtype=torch.int32, device=DEV), slots)
    assert torch.equal(a.pages[0], before)


def test_append_constant_tiny_and_non_finite_groups(ckv):
    d = 128
    k = torch.zeros(1, 1, 9, d, device=DEV)
    k[0, 0, 0] = 5.25                                 # one value: step 0
    k[0, 0, 1, :64] = 2.0 ** -110 * torch.arange(64, device=DEV)             # spans less than 2^-100
    k[0, 0, 2, 3] = float("nan")                      # a group reads as NaN, the other does not
    k[0, 0, 3, 70] = float("inf")
    k[0, 0, 4, 5] = -float("inf")
    k[0, 0, 5, 0], k[0, 0, 5, 1] = 3.0e38, -3.0e38    # further apart than fp32 holds
    k[0, 0, 6] = -1.0e-38
    k[0, 0, 7] = torch.linspace(1e30, 2e30, d, device=DEV)
    k[0, 0, 8] = 1000.0 + torch.arange(d, device=DEV) / 1024                  # an offset that bf16 cannot hold
    cache = ckv.q4_cache(1, 1, d, n_pages=2, max_pages=1)
    fill(ckv, cache, [9], k, -k)
    for got, x in zip(read(ckv, cache, F32)[0], (k[0, 0], -k[0, 0])):
        codes, ms, steps = quantise(x)
        want = torch.cat([c * steps[:, p:p + 1] + ms[:, p:p + 1] for p, c in enumerate(codes)], 1)
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(nan=7.0), want.nan_to_num(nan=7.0))
        nan = torch.zeros(9, 2, dtype=torch.bool, device=DEV)
        nan[2, 0] = nan[3, 1] = nan[4, 0] = nan[5, 0] = True
        assert torch.equal(got.isnan(), nan.repeat_interleave(64, 1))
        assert bool((got[0] == x[0]).all())
        assert bool(((got[8] - x[8]).abs() <= 0.51 * steps[8].repeat_interleave(64)).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_load_packs_skips_and_stays_inside(ckv, dtype):
    lens, d = [100, 5, 130, 64], 64
    cache = ckv.q4_cache(2, 2, d, n_pages=10, max_pages=3)
    g = torch.Generator(device=DEV).manual_seed(2)
    k, v = (torch.randn(2, 2, 130, d, generator=g, device=DEV).to(dtype) for _ in range(2))
    fill(ckv, cache, lens, k, v)
    whole = read(ckv, cache, dtype)
    start = torch.tensor([40, -1, 190, 120], dtype=torch.int64, device=DEV)
    wide = torch.full((2, 260, 2 * d), 9.0, dtype=dtype, device=DEV)
    ko, vo = wide[0, :250, d:], wide[1, :250, d:]     # rows further apart, an end inside row 2's tokens
    ckv.chunkkv_q4_load(cache, 0, start, 70, ko, vo)
    want = torch.full_like(wide, 9.0)
    for r, at in ((0, 40), (2, 190), (3, 120)):
        n = min(lens[r], 70, 250 - at)
        for i in range(2):
            want[i, at:at + n, d:] = whole[r][i][:n]
    assert torch.equal(wide, want)


def test_resize_is_the_8_bit_caches(ckv):
    g = torch.Generator(device=DEV).manual_seed(3)
    a, b = ckv.q4_cache(3, 2, 64, n_pages=20, max_pages=6), ckv.q8_cache(3, 2, 64, n_pages=20, max_pages=6)
    for step in range(8):
        new = torch.randint(0, 300, (6,), generator=g, device=DEV).int()
        sa, sb = (torch.empty(6, 200, dtype=torch.int64, device=DEV) for _ in range(2))
        ckv.chunkkv_q4_resize(a, new, sa)
        ckv.chunkkv_q8_resize(b, new, sb)
        for x, y in ((sa, sb), (a.table, b.table), (a.lens, b.lens), (a.ring, b.ring), (a.state, b.state)):
            assert torch.equal(x, y), step


# ------------------------------------------------------------------ attention

def many_rows_tol(q, ka, va, E, A, n, scale):
    return (2 * (2.0 ** -11 * E + 2.0 ** -39 * scale * q.abs().sum(1, keepdim=True) * ka.max()) + 2.0 ** -11) * A + n * 2.0 ** -28 * va.max()


def check(ckv, cache, q, out, scale, layer=0, q_lens=None, share=1.0):
    """Holds every live output row to 64 bits."""
    path = ckv.chunkkv_q4_path(cache, q.shape[-2] // cache.Hkv, q.shape[1] if q.dim() == 4 else 1, q.dtype)
    if q.dim() == 3:
        q, out = q[:, None], out[:, None]
    B, nq, Hq, d = q.shape
    G = Hq // cache.Hkv
    for r in range(cache.rows):
        b, h = divmod(r, cache.Hkv)
        n = int(cache.lens[r])
        m = nq if q_lens is None else min(max(int(q_lens[b]), 0), nq)
        sees = n - m + 1 + torch.arange(m, device=DEV)
        o = out[b, :m, h * G:(h + 1) * G].double()
        none = sees <= 0
        assert bool((o[none] == 0).all()), r
        if n == 0 or m == 0:
            continue
        (ks, km), (vs, vm) = held(cache, r, 0, layer), held(cache, r, 1, layer)
        hidden = torch.arange(n, device=DEV)[None] >= sees[:, None]
        for g in range(G):
            qr = q[b, :m, h * G + g].double()
            p = torch.softmax((qr @ (ks + km).T * scale).masked_fill(hidden, -math.inf), -1).masked_fill(none[:, None], 0.0)
            ref, A = p @ (vs + vm), p @ (vs + vm.abs())
            E = (qr.abs() @ (ks + km.abs()).T * scale).masked_fill(hidden, 0.0).amax(1, keepdim=True)
            tol = (2 * (d + 8) * 2.0 ** -22 * E + (n + 16) * 2.0 ** -22) * A + 1e-30
            if q.dtype == BF:
                tol = tol + 2.0 ** -8 * ref.abs() + (2.0 ** -11 + n * 2.0 ** -35) * A
            if path:
                tol = tol + many_rows_tol(qr, ks + km.abs(), vs + vm.abs(), E, A, n, scale)
            err = (o[:, g] - ref).abs()
            assert torch.isfinite(o[:, g]).all(), r
            assert bool((err <= share * tol).all()), f"row {r} ({n} tokens, {m} queries), head {g}: {float((err / tol).max())} of the tolerance"


def random_cache(ckv, B, Hkv, d, lens, seed, dtype=BF, spread=0.0, offset=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    pages = sum(-(-n // 64) for n in lens)
    cache = ckv.q4_cache(B, Hkv, d, n_pages=pages + 5, max_pages=max(1, max(-(-n // 64) for n in lens)))
    cache.ring.copy_(torch.randperm(pages + 5, generator=g, device=DEV).int())
    cache.pages[0].fill_(0xFF)                        # stale codes, steps and smallest values (NaN) that must not count
    n = max(max(lens), 1)
    grow = torch.exp(spread * torch.randn(1, 1, n, 1, generator=g, device=DEV))
    k = (torch.randn(B, Hkv, n, d, generator=g, device=DEV) + offset).to(dtype)
    v = (torch.randn(B, Hkv, n, d, generator=g, device=DEV) * grow - offset).to(dtype)
    fill(ckv, cache, lens, k, v)
    return cache, g


LENS = {
    "short": lambda rows: [(i * 37) % 130 for i in range(rows)],                # zero and one among them
    "one": lambda rows: [1] * rows,
    "pages": lambda rows: [64 * (i % 4) for i in range(rows)],
    "long": lambda rows: [3001 + 517 * i if i < 2 else 64 * i + 63 for i in range(rows)],
}


@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("dtype,d,B,Hkv,G", [(BF, 128, 2, 4, 4), (BF, 128, 3, 1, 7), (BF, 64, 4, 2, 1), (BF, 80, 1, 3, 8),
                                             (BF, 256, 2, 1, 12), (BF, 128, 1, 2, 33), (BF, 192, 1, 2, 3), (BF, 8, 2, 2, 2),
                                             (BF, 128, 2, 1, 16), (BF, 64, 1, 2, 9),
                                             (F32, 128, 2, 2, 4), (F32, 64, 1, 1, 16), (F32, 96, 2, 2, 5), (F32, 256, 1, 2, 3)])
def test_one_query_token(ckv, dtype, d, B, Hkv, G, lens):
    cache, g = random_cache(ckv, B, Hkv, d, LENS[lens](B * Hkv), seed=d + G)
    q = torch.randn(B, Hkv * G, d, generator=g, device=DEV).to(dtype)
    out = torch.full_like(q, float("nan"))
    ws = torch.zeros(ckv.chunkkv_q4_workspace_size(cache, G, 1, dtype), dtype=torch.uint8, device=DEV)
    for call in range(2):                             # the second call finds what the first left in the workspace
        out.fill_(float("nan"))
        ckv.chunkkv_q4_attention(cache, 0, q, out, ws)
        ckv.chunkkv_status_check(ws)
        check(ckv, cache, q, out, 1 / math.sqrt(d))
    assert torch.equal(ckv.q4_attention(cache, 0, q), out)                      # the same call gives the same bits
    assert torch.equal(ckv.q4_attention(cache, 0, q[:, None])[:, 0], out)       # one token of several is the same


@pytest.mark.parametrize("lens", ["short", "pages", "long"])
@pytest.mark.parametrize("dtype,d,B,Hkv,G,n_q", [(BF, 128, 2, 2, 4, 2), (BF, 128, 2, 1, 7, 5), (BF, 64, 3, 2, 1, 40), (BF, 80, 1, 3, 2, 130),
                                                 (BF, 128, 2, 2, 4, 100), (BF, 256, 2, 1, 2, 9), (BF, 128, 1, 2, 4, 301),
                                                 (BF, 8, 2, 2, 3, 70), (F32, 64, 2, 2, 2, 9), (F32, 128, 2, 1, 3, 70)])
def test_several_query_tokens(ckv, dtype, d, B, Hkv, G, n_q, lens):
    ls = LENS[lens](B * Hkv)                          # shorter than n_q among them: queries that see nothing
    cache, g = random_cache(ckv, B, Hkv, d, ls, seed=d + G + n_q)
    q = torch.randn(B, n_q, Hkv * G, d, generator=g, device=DEV).to(dtype)
    ws = torch.zeros(ckv.chunkkv_q4_workspace_size(cache, G, n_q, dtype), dtype=torch.uint8, device=DEV)
    for counts in (None, [n_q // 2 + 1, 0, 1][:B], [n_q + 3, n_q - 1, -2][:B]):
        q_lens = None if counts is None else torch.tensor(counts, dtype=torch.int32, device=DEV)
        out = torch.full_like(q, 7.0)
        ckv.chunkkv_q4_attention(cache, 0, q, out, ws, q_lens=q_lens)
        ckv.chunkkv_status_check(ws)
        check(ckv, cache, q, out, 1 / math.sqrt(d), q_lens=q_lens)
        for b in range(B):
            m = n_q if counts is None else min(max(counts[b], 0), n_q)
            assert bool((out[b, m:] == 7.0).all())    # rows behind the sequence's last query are left alone
        again = ckv.q4_attention(cache, 0, q, q_lens=q_lens)
        assert torch.equal(torch.where(out == 7.0, 0.0, out.float()), torch.where(out == 7.0, 0.0, again.float()))


@pytest.mark.parametrize("n_q,G,d,extra", [(1100, 4, 128, 0), (600, 7, 128, 3), (333, 1, 64, 129), (257, 128, 64, 0), (40, 300, 8, 2)])
def test_a_whole_prompt_over_its_own_cache(ckv, n_q, G, d, extra):
    # every token a query, each sees itself and those before it; many units, and heads that make several groups
    cache, g = random_cache(ckv, 1, 2, d, [n_q + extra, n_q], seed=n_q, offset=0.3)
    q = torch.randn(1, n_q, 2 * G, d, generator=g, device=DEV).to(BF)
    check(ckv, cache, q, ckv.q4_attention(cache, 0, q), 1 / math.sqrt(d))


@pytest.mark.parametrize("dtype,n_q", [(BF, 4), (BF, 33), (F32, 3)])
def test_axes_that_are_repeated(ckv, dtype, n_q):
    # one query for all heads, or for all sequences (strides of zero): no tensor map can address it
    cache, g = random_cache(ckv, 2, 2, 64, [200, 70, 64, 130], seed=23)
    for shape in ((2, n_q, 1, 64), (1, n_q, 8, 64), (2, 1, 8, 64)):
        q = torch.randn(*shape, generator=g, device=DEV).to(dtype).expand(2, n_q, 8, 64)
        out = torch.full((2, n_q, 8, 64), float("nan"), dtype=dtype, device=DEV)
        ckv.q4_attention(cache, 0, q, out=out)
        check(ckv, cache, q, out, 1 / 8)


def test_many_rows(ckv):
    lens = [int(x) for x in torch.randint(0, 200, (1200,), generator=torch.Generator().manual_seed(1))]
    cache, g = random_cache(ckv, 300, 4, 64, lens, seed=6)
    for shape in ((300, 8, 64), (300, 30, 8, 64)):
        q = torch.randn(*shape, generator=g, device=DEV).to(BF)
        check(ckv, cache, q, ckv.q4_attention(cache, 0, q), 1 / 8)


@pytest.mark.parametrize("dtype,n_q", [(BF, 1), (F32, 1), (BF, 3), (BF, 50)])
def test_long_rows_with_uneven_steps_and_sharp_logits(ckv, dtype, n_q):
    # value steps that differ by orders of magnitude between tokens, offsets, one dominant key, large and tiny queries
    cache, g = random_cache(ckv, 2, 2, 128, [20001, 0, 1, 9000], seed=77, spread=2.0, offset=0.5)
    q = torch.randn(2, n_q, 8, 128, generator=g, device=DEV)
    q[1] *= 30.0
    q = q.to(dtype)
    check(ckv, cache, q, ckv.q4_attention(cache, 0, q), 1 / math.sqrt(128))
    tiny = (q.float() * 1e-30).to(dtype)
    check(ckv, cache, tiny, ckv.q4_attention(cache, 0, tiny), 1 / math.sqrt(128))
    zero = torch.zeros_like(q)
    check(ckv, cache, zero, ckv.q4_attention(cache, 0, zero, scale=0.5), 0.5)


@pytest.mark.parametrize("dtype,G,n_q", [(BF, 4, 1), (BF, 12, 1), (F32, 4, 1), (BF, 4, 3), (BF, 4, 20)])
def test_value_steps_far_apart(ckv, dtype, G, n_q):
    # half of a row's tokens hold values 2^r times the others' under weights below 2^-150 of theirs, in either order;
    # the tolerance goes by the tokens that count
    d, n, powers = 64, 768, [0, 20, 40, 60, 80]
    rows = 2 * len(powers)
    g = torch.Generator(device=DEV).manual_seed(61)
    cache = ckv.q4_cache(rows, 1, d, n_pages=rows * 12, max_pages=12)
    k = 0.1 * torch.randn(rows, 1, n, d, generator=g, device=DEV)
    v = torch.randn(rows, 1, n, d, generator=g, device=DEV)
    far = (torch.arange(n, device=DEV)[None] < n // 2) ^ (torch.arange(rows, device=DEV) % 2 == 1)[:, None]
    k[:, 0, :, 0] = torch.where(far, -150.0, 1.0)
    k[:, 0, :, 1] = torch.where(far, 150.0, 1.0)
    v *= torch.where(far, 2.0 ** torch.tensor(powers, device=DEV).repeat_interleave(2)[:, None], 1.0)[:, None, :, None]
    fill(ckv, cache, [n] * rows, k, v)
    q = torch.zeros(rows, n_q, G, d, device=DEV)
    q[..., 0] = 1 + torch.arange(G, device=DEV) / 16
    q = q.to(dtype)
    out = ckv.q4_attention(cache, 0, q, scale=1.0)
    path = ckv.chunkkv_q4_path(cache, G, n_q, dtype)
    for r in range(rows):
        (ks, km), (vs, vm) = held(cache, r, 0), held(cache, r, 1)
        near = ~far[r]
        for i in range(n_q):
            qr, m = q[r, i].double(), n - n_q + 1 + i
            p = torch.softmax(qr @ (ks + km)[:m].T, -1)
            ref, A = p @ (vs + vm)[:m], p @ (vs + vm.abs())[:m]
            E = (qr.abs() @ (ks + km.abs())[near].T).amax(1, keepdim=True)
            tol = (2 * (d + 8) * 2.0 ** -22 * E + (n + 16) * 2.0 ** -22) * A
            if dtype == BF:
                tol = tol + 2.0 ** -8 * ref.abs() + (2.0 ** -11 + n * 2.0 ** -35) * A
            if path:
                tol = tol + many_rows_tol(qr, (ks + km.abs())[near], (vs + vm.abs())[near], E, A, n, 1.0)
            err = (out[r, i].double() - ref).abs()
            assert bool((err <= tol).all()), f"2^{powers[r // 2]}, row {r}, query {i}: {float((err / tol).max())} of the tolerance"


@pytest.mark.parametrize("dtype,n_q,d", [(BF, 3, 128), (BF, 60, 128), (F32, 5, 64), (BF, 2, 256), (BF, 90, 64)])
def test_hidden_tokens_may_hold_anything(ckv, dtype, n_q, d):
    # non-finite keys and values among the query tokens' own: each reaches the queries from its token on, its group's
    # columns alone where it is a value
    lens = [700, n_q, 130, n_q + 1]
    cache, g = random_cache(ckv, 2, 2, d, lens, seed=41)
    q = torch.randn(2, n_q, 8, d, generator=g, device=DEV).to(dtype)
    clean = ckv.q4_attention(cache, 0, q)
    at = n_q // 2                                     # the query token whose value is spoilt, for the second row
    for which in (0, 1):
        x = torch.zeros(2, 2, 1, d, device=DEV).to(dtype)
        x[0, 1, 0, 1] = float("nan")
        (token,) = [lens[1] - n_q + at]
        slots = torch.full((4, 1), -1, dtype=torch.int64, device=DEV)
        slots[1, 0] = int(cache.table[1, token // 64]) * 64 + token % 64
        ok = torch.zeros_like(x)
        pages = cache.pages[0].clone()
        ckv.chunkkv_q4_append(cache, 0, x if which == 0 else ok, x if which else ok,
                              torch.tensor([0, 1, 0, 0], dtype=torch.int32, device=DEV), slots)
        spoilt = ckv.q4_attention(cache, 0, q)
        cache.pages[0].copy_(pages)
        assert torch.equal(spoilt[1], clean[1]) and torch.equal(spoilt[0, :, :4], clean[0, :, :4])
        # queries before the token see neither it nor what it replaced
        assert torch.equal(spoilt[0, :at, 4:], clean[0, :at, 4:])
        if which == 0:
            assert bool(spoilt[0, at:, 4:].isnan().all())
        else:
            assert bool(spoilt[0, at:, 4:, :64].isnan().all()) and not bool(spoilt[0, at:, 4:, 64:].isnan().any())


@pytest.mark.parametrize("dtype,n_q", [(BF, 1), (BF, 3), (F32, 2), (BF, 40)])
def test_logits_of_minus_infinity(ckv, dtype, n_q):
    # all of a row's visible logits -inf: NaN, as the formula; some of them: the others decide
    d = 64
    cache = ckv.q4_cache(2, 1, d, n_pages=8, max_pages=3)
    k = torch.ones(2, 1, 150, d, device=DEV)
    k[0] = -1e20
    k[1, :, :140] = -1e20
    v = torch.randn(2, 1, 150, d, generator=torch.Generator(device=DEV).manual_seed(2), device=DEV)
    fill(ckv, cache, [150, 150], k, v)
    q = torch.full((2, n_q, 2, d), 1e30, device=DEV).to(dtype)
    out = ckv.q4_attention(cache, 0, q, scale=1.0)
    assert bool(out[0].isnan().all())
    small = torch.full_like(q, 1e-3)
    few = ckv.q4_attention(cache, 0, small)
    sc, m = held(cache, 1, 1)
    last = (sc + m)
    for i in range(n_q):
        n = 150 - n_q + 1 + i
        if n > 140:
            want = last[140:n].mean(0)
            assert bool(((few[1, i].double() - want).abs() <= 2.0 ** -7 * (sc + m.abs())[140:n].mean(0)).all()), i


@pytest.mark.parametrize("lens", [[6582] * 8, [800, 900], [577, 64, 4000, 1, 1300], [3001] * 40])
@pytest.mark.parametrize("dtype,n_q", [(F32, 1), (BF, 3), (BF, 30)])
def test_every_token_counts_once(ckv, lens, dtype, n_q):
    # zero keys, so equal weights; a code of 15 in column c of 128 tokens' run w for token w + c gives 15 / n there
    d, rows = 128, len(lens)
    lens = [max(n, n_q) for n in lens]
    cache, g = random_cache(ckv, rows, 1, d, lens, seed=71)
    one = 0x3F80 << 16
    parts = cache.pages[0].view(torch.int32)          # [n_pages, 2304]: keys 1024, (m, s) 128, values 1024, (m, s) 128
    parts[:, :1024] = 0
    for a in (1024, 2176):
        parts[:, a:a + 128] = one                     # m = 0, s = 1
    q = torch.randn(rows, n_q, 2, d, generator=g, device=DEV).to(dtype)
    ws = torch.zeros(ckv.chunkkv_q4_workspace_size(cache, 2, n_q, dtype), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(q)
    sees = torch.tensor(lens, device=DEV)[:, None] - n_q + 1 + torch.arange(n_q, device=DEV)
    t = torch.arange(64, device=DEV)
    values = cache.pages[0].view(-1, 9216)[:, 4608:8704]
    for w in range(0, max(lens), d):
        values.zero_()
        for half in (0, 64):
            has = [r for r in range(rows) if lens[r] > w + half]
            if has:
                page = cache.table[has, (w + half) // 64].long()
                col, i = t + half, t % 16
                nib = i % 8 // 2 + 4 * (i % 2)
                at = (((col // 16 * 8 + col % 8) * 4 + t // 16) * 2 + col % 16 // 8) * 8 + 4 * (i // 8) + nib // 2
                values[page[:, None], at] = (15 << (4 * (nib % 2))).to(torch.uint8)
        ckv.chunkkv_q4_attention(cache, 0, q, out, ws)
        want = (w + torch.arange(d, device=DEV) < sees[:, :, None]) * (15.0 / sees[:, :, None].double())
        tol = ((sees[:, :, None] + 16) * 2.0 ** -22 + (2.0 ** -8 if dtype == BF else 0)) * want
        assert bool(((out.double() - want[:, :, None]).abs() <= tol[:, :, None]).all()), w


@pytest.mark.parametrize("kind", ["large", "nan"])
@pytest.mark.parametrize("dtype,n_q", [(F32, 1), (BF, 1), (BF, 2), (BF, 40)])
def test_rows_keep_their_bits_whatever_others_ask(ckv, kind, dtype, n_q):
    cache, g = random_cache(ckv, 3, 2, 128, [3000, 70, 1, 900, 64, 2000], seed=97, spread=2.0)
    q = torch.randn(3, n_q, 12, 128, generator=g, device=DEV)
    want = ckv.q4_attention(cache, 0, q.to(dtype))
    other = q.clone()
    other[:, :, 2::6] = q[:, :, 2::6] * 60 if kind == "large" else float("nan")
    out = ckv.q4_attention(cache, 0, other.to(dtype))
    rest = [h for h in range(12) if h % 6 != 2]
    assert torch.equal(out[:, :, rest], want[:, :, rest])


@pytest.mark.parametrize("n_q", [1, 5, 60])
def test_strides_layers_and_streams(ckv, n_q):
    B, Hkv, G, d = 2, 2, 4, 128
    lens = [100, 260, 61, 64]
    cache = ckv.q4_cache(B, Hkv, d, n_pages=30, max_pages=5, n_layers=2)
    g = torch.Generator(device=DEV).manual_seed(12)
    k = torch.randn(B, Hkv, 260, d, generator=g, device=DEV).to(BF)
    counts = fill(ckv, cache, lens, k, k, layer=0)
    slots = torch.empty(4, 260, dtype=torch.int64, device=DEV)
    for r in range(4):                                # the second layer's rows go to the same slots
        pos = torch.arange(260, device=DEV)
        slots[r] = cache.table[r].long()[(pos // 64).clamp(max=4)] * 64 + pos % 64
    ckv.chunkkv_q4_append(cache, 1, 2 * k, -k, counts, slots)
    qkv = torch.randn(n_q, B, Hkv * G + 3, d, generator=g, device=DEV).to(BF)
    q = qkv[:, :, 1:1 + Hkv * G].transpose(0, 1)      # tokens before sequences
    for layer in range(2):
        wide = torch.full((B, n_q, Hkv * G, 2 * d), 3.0, dtype=BF, device=DEV)
        out = wide[..., d:]
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            ckv.q4_attention(cache, layer, q, out=out)
        side.synchronize()
        check(ckv, cache, q, out, 1 / math.sqrt(d), layer)
        assert bool((wide[..., :d] == 3.0).all())


@pytest.mark.parametrize("n_q", [1, 4, 50])
def test_a_graph_follows_the_lengths(ckv, n_q):
    # one captured step serves later lengths and counts: they are read on the device
    cache, g = random_cache(ckv, 2, 2, 128, [500, 60, 0, 64], seed=31)
    q = torch.randn(2, n_q, 8, 128, generator=g, device=DEV).to(BF)
    q_lens = torch.full((2,), n_q, dtype=torch.int32, device=DEV)
    ws = torch.zeros(ckv.chunkkv_q4_workspace_size(cache, 4, n_q), dtype=torch.uint8, device=DEV)
    out = torch.zeros_like(q)
    ckv.chunkkv_q4_attention(cache, 0, q, out, ws, q_lens=q_lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ckv.chunkkv_q4_attention(cache, 0, q, out, ws, q_lens=q_lens)
    for new, m in (([500, 60, 0, 64], [n_q, n_q]), ([77, 60, 0, 1], [1, n_q]), ([0, 0, 0, 0], [n_q, 0])):
        ckv.chunkkv_q4_resize(cache, torch.tensor(new, dtype=torch.int32, device=DEV))
        q_lens.copy_(torch.tensor(m, dtype=torch.int32))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check(ckv, cache, q, out, 1 / math.sqrt(128), q_lens=q_lens)


def test_one_workspace_serves_any_calls_in_turn(ckv):
    import test_gpu_serving as other
    small, g = random_cache(ckv, 2, 4, 128, [6000 + 100 * i for i in range(8)], seed=51)
    large, _ = random_cache(ckv, 64, 8, 128, [600 + (i * 97) % 700 for i in range(512)], seed=52)
    narrow, _ = random_cache(ckv, 3, 1, 64, [5000, 40, 2000], seed=53)
    eight, _ = other.random_cache(ckv, 2, 4, 128, [5000 + 90 * i for i in range(8)], seed=54)
    pq, pk, pv = other.make_qkv([20], [9000], 8, 2, 128, BF, seed=54)
    p, keep = ckv.prefill_params_for(pq, pk, [0, 20], [0, 9000])
    want = ckv.prefill_attention(pq, pk, pv, [0, 20], [0, 9000])
    shapes = [(small, 4, 1, BF), (large, 2, 1, F32), (narrow, 7, 30, BF), (small, 3, 5, BF), (narrow, 20, 1, F32), (large, 4, 3, BF)]
    ws = torch.zeros(max([ckv.chunkkv_q4_workspace_size(c, G, n, t) for c, G, n, t in shapes]
                         + [ckv.chunkkv_prefill_workspace_size(p), ckv.chunkkv_q8_workspace_size(eight, 12)]),
                     dtype=torch.uint8, device=DEV)
    for cache, G, n, dtype in shapes:
        q = torch.randn(cache.B, n, cache.Hkv * G, cache.d, generator=g, device=DEV).to(dtype)
        out = torch.full_like(q, float("nan"))
        ckv.chunkkv_q4_attention(cache, 0, q, out, ws)
        ckv.chunkkv_status_check(ws)
        check(ckv, cache, q, out, 1 / math.sqrt(cache.d))
        prompt = torch.full_like(pq, float("nan"))
        ckv.chunkkv_prefill_attention(p, pq, pk, pv, prompt, ws)
        assert torch.equal(prompt, want)
        q8 = torch.randn(2, 48, 128, generator=g, device=DEV).to(BF)
        out8 = torch.empty_like(q8)
        ckv.chunkkv_q8_attention(eight, 0, q8, out8, ws)
        other.check_decode(ckv, eight, q8, out8, 1 / math.sqrt(128))


def test_calls_refuse_tensors_outside_the_gpu(ckv):
    # one argument at a time in host memory: an error on the host, and nothing is launched
    cache, _ = random_cache(ckv, 1, 2, 64, [70, 5], seed=91)
    i32, i64 = torch.zeros(2, dtype=torch.int32, device=DEV), torch.zeros(2, 4, dtype=torch.int64, device=DEV)
    k = torch.zeros(1, 2, 4, 64, device=DEV)
    start, rows = torch.zeros(2, dtype=torch.int64, device=DEV), torch.zeros(100, 64, device=DEV)
    q, ws = torch.zeros(1, 4, 64, device=DEV), torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
    calls = [(lambda n, s: ckv.chunkkv_q4_resize(cache, n, s), (i32, i64)),
             (lambda k, v, n, s: ckv.chunkkv_q4_append(cache, 0, k, v, n, s), (k, k, i32, i64)),
             (lambda s, k, v: ckv.chunkkv_q4_load(cache, 0, s, 4, k, v), (start, rows, rows)),
             (lambda q, o, w, n: ckv.chunkkv_q4_attention(cache, 0, q, o, w, q_lens=n), (q, q.clone(), ws, i32[:1].contiguous()))]
    torch.cuda.synchronize()
    before = ckv.chunkkv_launch_count()
    for call, args in calls:
        for i in range(len(args)):
            with pytest.raises(ValueError):
                call(*args[:i], args[i].cpu(), *args[i + 1:])
    assert ckv.chunkkv_launch_count() == before


# ------------------------------------------------------------------ together

def test_the_example_serves_a_layer_in_4_bits(ckv):
    # a next turn, decoding and a second compression over the cache: each output within what the rounding of keys and
    # values to 4 bits does (half a step of 1/15 of a group's range, 5 for normal data: 0.1 relative to a value)
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import serve_layer
    result = serve_layer.serve(bits=4)
    assert len(result["errors"]) == 40 and max(result["errors"]) < 0.3 and result["turn_error"] < 0.3
    assert result["lengths"][2] != result["lengths"][1] and result["free_pages"] > 0
    again = serve_layer.serve(bits=4)
    assert again["errors"] == result["errors"]        # the same run gives the same bits
