"""What is timed of the operators of the 4-bit cache, and their plain forms.

Five kinds of case:
  store    rows written into the cache, quantised, and the rows read back (chunkkv_q4_append, chunkkv_q4_load)
  read     rows read back alone (chunkkv_q4_load)
  step     one token written to each row, then one query token per sequence over the cache
           (chunkkv_q4_append, chunkkv_q4_attention)
  decode   one query token per sequence over the cache (chunkkv_q4_attention)
  turn     several query tokens per sequence, the last of the cache's tokens being their own (chunkkv_q4_attention)

The 4-bit cache.  A cache row r = b * Hkv + h is one (sequence, KV head) with a length of its own (chunk compression
keeps another number of tokens for each head).  Every token's 64-column groups are quantised by themselves:
  m = lo rounded down to bf16, s = (hi - m) / 15 rounded up to bf16, code = round((x - m) / s) in 0 .. 15
(lo, hi: the group's smallest and largest value), and a code stands for s * code + m.  A page holds 64 tokens of one row,
with ND = ceil(d / 64) groups a token:
  keys     [64 tokens][4][ND][8 bytes]            bytes t, g of a token: columns 64 g + 16 t .. + 15
  their m, s   [ND][64 tokens][2] bf16
  values   [4 ND][8][4][2][8 bytes]               bytes p, c, t, h: tokens 16 t .. + 15 of column 16 p + 8 h + c
  their m, s   [ND][64 tokens][2] bf16
Of 16 codes in 8 bytes, code 8 w + 2 p + e is nibble p + 4 e of 32-bit word w.  table[r][j] is the page of tokens
64 j .. 64 j + 63 of row r; a slot is page * 64 + offset.
"""
import math
import random

import torch

own = False

PAGE = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SMALLEST = 2.0 ** -100                  # a group that spans less has step 0


def dev():
    return torch.device("cuda:0")


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the kept rows of a 32K prompt at a 20 % budget are written after compression, and read back for the next one
        dict(name="store_llama_kept", kind="store", B=1, Hkv=8, d=128, dtype="bf16", old=0, new=6582, lens=8),
        # tokens decoded since join small caches (budget 256), inside a page that is already open
        dict(name="store_tail", kind="store", B=16, Hkv=8, d=128, dtype="bf16", old=288, new=37, lens=9),
        # the kept rows of eight 128K prompts
        dict(name="store_qwen_8", kind="store", B=8, Hkv=4, d=128, dtype="bf16", old=0, new=13164, lens=21),
        # ragged caches of an odd head size read back in fp32
        dict(name="read_f32_80", kind="read", B=6, Hkv=2, d=80, dtype="f32", lmin=1, lmax=2001, lens=22),
        # a serving step of sixteen sequences: their new tokens are written and attended to
        dict(name="step_mistral_16", kind="step", B=16, Hq=32, Hkv=8, d=128, dtype="bf16", lmin=256, lmax=300, lens=23),
        # one sequence decodes over its compressed 32K prompt: latency
        dict(name="decode_llama_6582", kind="decode", B=1, Hq=32, Hkv=8, d=128, dtype="bf16", lmin=6500, lmax=6582,
             lens=10),
        # a large batch over compressed 128K prompts: bandwidth
        dict(name="decode_qwen_64", kind="decode", B=64, Hq=28, Hkv=4, d=128, dtype="bf16", lmin=12000, lmax=13164,
             lens=12),
        # the framework's small fp32 heads over ragged rows, empty ones among them
        dict(name="decode_f32_ragged", kind="decode", B=5, Hq=4, Hkv=2, d=64, dtype="f32", lmin=0, lmax=1500, lens=24),
        # eight sequences check drafts of five tokens over their compressed 32K prompts
        dict(name="draft_llama_8", kind="turn", B=8, Hq=32, Hkv=8, d=128, dtype="bf16", qmin=5, qmax=5, lmin=6500,
             lmax=6582, lens=25),
        # the next turns of two conversations against what the cache holds
        dict(name="turn_llama_2", kind="turn", B=2, Hq=32, Hkv=8, d=128, dtype="bf16", qmin=300, qmax=700, lmin=4501,
             lmax=9001, lens=26),
        # a long document follows a compressed 128K prompt
        dict(name="turn_qwen_4001", kind="turn", B=1, Hq=28, Hkv=4, d=128, dtype="bf16", qmin=4001, qmax=4001,
             lmin=12000, lmax=13164, lens=27),
        # a few tokens against small fp32 caches
        dict(name="turn_f32_small", kind="turn", B=3, Hq=4, Hkv=2, d=64, dtype="f32", qmin=1, qmax=9, lmin=0, lmax=700,
             lens=28),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["store", "read", "step", "decode", "decode", "turn", "turn"])
    Hq, Hkv, d, dtype = rng.choice([(32, 8, 128, "bf16"), (28, 4, 128, "bf16"), (8, 8, 64, "bf16"), (4, 2, 64, "f32"),
                                    (12, 2, 80, "bf16"), (16, 1, 128, "bf16"), (6, 2, 128, "f32"), (4, 1, 256, "bf16")])
    case = dict(kind=kind, B=1, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, lens=rng.randrange(1 << 20))
    if kind in ("store", "read"):
        del case["Hq"]
        case["B"] = _log(rng, 1, 32)
        most = max(2, 200000 // (case["B"] * Hkv))
        if kind == "store":
            case.update(old=rng.choice([0, _log(rng, 1, 700)]), new=_log(rng, 1, most))
        else:
            case.update(lmin=rng.choice([0, most // 3]), lmax=most)
        return case
    if kind in ("step", "decode"):
        case["B"] = _log(rng, 1, 64)
        top = _log(rng, 16, min(40000, 3000000 // (case["B"] * Hkv)))
        case.update(lmin=rng.choice([0, top // 2, top]), lmax=top)
        return case
    case["B"] = rng.choice([1, 1, 2, 4, 8, 16])
    n = _log(rng, 2, (3000 if dtype == "bf16" and d <= 128 else 200) // (1 if case["B"] == 1 else case["B"]))
    top = _log(rng, 100, min(16000, 150000 // (case["B"] * Hkv)))
    case.update(qmin=rng.choice([n, max(1, n // 4), 1]), qmax=n, lmin=rng.choice([0, top // 2, top]), lmax=top)
    return case


def _lens(case):
    """Lengths by cache row before the call, what each row gains, and the query tokens of each sequence."""
    r = random.Random(case["lens"])
    B, Hkv = case["B"], case["Hkv"]
    rows = B * Hkv
    if case["kind"] == "store":
        old = [r.randint(case["old"] // 2, case["old"]) if case["old"] else 0 for _ in range(rows)]
        return old, [r.randint((case["new"] * 9) // 10, case["new"]) for _ in range(rows)], [0] * B
    have = [r.randint(case["lmin"], case["lmax"]) for _ in range(rows)]
    if case["kind"] == "turn":          # the queries' own tokens are in the cache already
        q = [r.randint(case["qmin"], case["qmax"]) for _ in range(B)]
        return [n + q[i // Hkv] for i, n in enumerate(have)], [0] * rows, q
    return have, [1 if case["kind"] == "step" else 0] * rows, [0 if case["kind"] == "read" else 1] * B


def _groups(d):
    return (d + 63) // 64


def work(case):
    old, new, q = _lens(case)
    d, elt = case["d"], 2 if case["dtype"] == "bf16" else 4
    token = 2 * (d / 2 + 4 * _groups(d))                # a token's keys and values as they are held
    n = sum(old) + sum(new)
    if case["kind"] in ("store", "read"):
        return {"bytes": int(sum(new) * (2 * d * elt + token) + n * (2 * d * elt + token)), "flops": 0}
    G = case["Hq"] // case["Hkv"]
    pairs = 0                                           # (query, key) pairs of a head of each row
    for r, (a, b) in enumerate(zip(old, new)):
        m = q[r // case["Hkv"]]
        pairs += m * (a + b - m) + m * (m + 1) // 2
    return {"bytes": int(n * token + sum(new) * 2 * d * elt + 2 * sum(q) * case["Hq"] * d * elt),
            "flops": 4 * d * G * pairs}


# ------------------------------------------------------------------ the layout

def _unpack(b):
    """8 bytes of codes (last axis) as 16 codes."""
    b = b.to(torch.uint8)
    n = torch.stack([b & 15, b >> 4], -1)                               # byte 4 w + 2 e + ph, nibble pl
    n = n.view(*b.shape[:-1], 2, 2, 2, 2)                               # [w][e][ph][pl]
    k = n.dim()
    return n.permute(*range(k - 4), k - 4, k - 2, k - 1, k - 3).reshape(*b.shape[:-1], 16)


def _pack(c):
    """16 codes (last axis) as 8 bytes."""
    n = c.to(torch.uint8).view(*c.shape[:-1], 2, 2, 2, 2)               # [w][ph][pl][e]
    k = n.dim()
    n = n.permute(*range(k - 4), k - 4, k - 1, k - 3, k - 2)            # [w][e][ph][pl]
    return (n[..., 0] | (n[..., 1] << 4)).reshape(*c.shape[:-1], 8)


def _split(pages, nd):
    """A pool's parts: keys, their (m, s), values, their (m, s); views."""
    n = pages.shape[0]
    a, b = 2048 * nd, 256 * nd
    return (pages[:, :a].view(n, 64, 4, nd, 8), pages[:, a:a + b].view(torch.bfloat16).view(n, nd, 64, 2),
            pages[:, a + b:2 * a + b].view(n, 4 * nd, 8, 4, 2, 8),
            pages[:, 2 * a + b:].view(torch.bfloat16).view(n, nd, 64, 2))


def _codes(part, which):
    """Codes of some pages as [pages, 64 tokens, 64 nd]."""
    c = _unpack(part)
    if which == 0:                                                      # [n, token, t, g, 16]
        return c.permute(0, 1, 3, 2, 4).reshape(c.shape[0], 64, -1)
    return c.permute(0, 3, 5, 1, 4, 2).reshape(c.shape[0], 64, -1)      # [n, p, c, t, h, 16]


def _bytes_of(codes, which):
    """The same the other way: [pages, 64 tokens, 64 nd] to a part's bytes."""
    n, nd = codes.shape[0], codes.shape[2] // 64
    if which == 0:
        return _pack(codes.view(n, 64, nd, 4, 16).permute(0, 1, 3, 2, 4).contiguous())
    return _pack(codes.view(n, 4, 16, 4 * nd, 2, 8).permute(0, 3, 5, 1, 4, 2).contiguous())


def _quantise(x):
    """Codes, m and s of tokens x [..., d] in fp32: [..., 64 nd], [..., nd], [..., nd]."""
    d = x.shape[-1]
    nd = _groups(d)
    wide = torch.nn.functional.pad(x, (0, 64 * nd - d))
    inside = (torch.arange(64 * nd, device=x.device) < d).view(nd, 64)
    g = wide.view(*x.shape[:-1], nd, 64)
    lo = g.masked_fill(~inside, math.inf).amin(-1)
    hi = g.masked_fill(~inside, -math.inf).amax(-1)
    bits = lo.contiguous().view(torch.int32)
    m = ((bits + ((bits >> 31) & 0xFFFF)) & -65536).view(torch.float32)        # rounded down
    span = hi - m
    s = (((span * (1.0 / 15.0)).view(torch.int32) + 0xFFFF) & -65536).view(torch.float32)   # rounded up
    s = torch.where(span >= SMALLEST, s, 0.0)
    inv = torch.where(s > 0, torch.reciprocal(s), 0.0)
    c = torch.round((g - m[..., None]) * inv[..., None]).clamp(0, 15)
    c = torch.where(inside, c, 0.0)
    return c.reshape(*x.shape[:-1], 64 * nd).to(torch.uint8), m, s


def _values(pages, which, nd, d, dtype=torch.float32):
    """What some pages stand for, [pages, 64 tokens, d]."""
    parts = _split(pages, nd)
    ms = parts[2 * which + 1].to(dtype)
    c = _codes(parts[2 * which], which).view(-1, 64, nd, 64).to(dtype)
    x = c * ms[..., 1].transpose(1, 2)[..., None] + ms[..., 0].transpose(1, 2)[..., None]
    return x.reshape(-1, 64, 64 * nd)[:, :, :d]


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=dev()).manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=dev())


def _chan(g, *shape):
    """Per-channel scales of keys: a few channels are much larger than the rest, as in trained models."""
    c = torch.rand(*shape, generator=g, device=dev()) * 1.5 + 0.5
    return torch.where(torch.rand(*shape, generator=g, device=dev()) < 0.04, 4 * c, c)


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _layout(rows_pages, max_pages, n_pages, g):
    """Tables of rows that hold rows_pages pages each, scattered over the pool; the ring of the free ones."""
    perm = torch.randperm(n_pages, generator=g, device=dev()).to(torch.int32)
    have = torch.tensor(rows_pages, device=dev(), dtype=torch.int64)
    first = have.cumsum(0) - have
    j = torch.arange(max_pages, device=dev())
    at = first[:, None] + j
    table = torch.where(j < have[:, None], perm[at.clamp(max=n_pages - 1)], -1).to(torch.int32)
    used = int(have.sum())
    ring = perm.roll(-used).contiguous()
    return table, ring, torch.tensor([0, n_pages - used, 0, 0], dtype=torch.int32, device=dev())


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device=dev())


def prepare(case, seed):
    g = _gen(seed)
    old, new, q = _lens(case)
    dt, d = DTYPES[case["dtype"]], case["d"]
    nd, lens = _groups(d), [a + b for a, b in zip(old, new)]
    rows = len(lens)
    s = {"case": case, "nd": nd}
    s["max_pages"] = max(1, max(_pages(n) for n in lens))
    s["n_pages"] = sum(_pages(n) for n in lens) + 3
    s["table"], s["ring"], s["state"] = _layout([_pages(n) for n in lens], s["max_pages"], s["n_pages"], g)
    s["lens"] = _int32(lens)
    # what earlier steps wrote (older tokens past the rows' ends included)
    chan = _chan(g, d)
    s["pages"] = torch.zeros(s["n_pages"], 4608 * nd, dtype=torch.uint8, device=dev())
    for at in range(0, s["n_pages"], 8192):
        part = _split(s["pages"][at:at + 8192], nd)
        for i in range(2):
            c, m, step = _quantise((_normal(g, part[0].shape[0], PAGE, d) * (chan if i == 0 else 1.0)).to(dt).float())
            part[2 * i].copy_(_bytes_of(c, i))
            part[2 * i + 1].copy_(torch.stack([m, step], -1).transpose(1, 2))
    if case["kind"] in ("store", "step"):
        cap = max(max(new), 1)
        s["k"] = (_normal(g, case["B"], case["Hkv"], cap, d) * chan).to(dt)
        s["v"] = _normal(g, case["B"], case["Hkv"], cap, d).to(dt)
        s["counts"] = _int32(new).view(case["B"], case["Hkv"])
        pos = _int32(old).long()[:, None] + torch.arange(cap, device=dev())
        page = s["table"].long().gather(1, (pos // PAGE).clamp(max=s["max_pages"] - 1))
        fill = torch.arange(cap, device=dev()) < _int32(new)[:, None]
        s["slots"] = torch.where(fill, page * PAGE + pos % PAGE, -1)
    if case["kind"] in ("store", "read"):
        s["cap"] = max(max(lens), 1)
        s["start"] = torch.arange(rows, device=dev()) * s["cap"]
        s["k_out"] = torch.zeros(rows * s["cap"], d, dtype=dt, device=dev())
        s["v_out"] = torch.zeros(rows * s["cap"], d, dtype=dt, device=dev())
        return s
    if case["kind"] == "turn":          # a padded batch of query tokens, with how many of them are real
        s["q"] = _normal(g, case["B"], max(q), case["Hq"], d).to(dt)
        s["q_lens"] = _int32(q)
    else:
        s["q"] = _normal(g, case["B"], case["Hq"], d).to(dt)
        s["q_lens"] = None
    s["out"] = torch.zeros_like(s["q"])
    return s


# ------------------------------------------------------------------ the framework's operators

def _run_own(s):
    import chunk_level_kv_gb300 as ckv
    c = s["case"]
    if "cache" not in s:                # the handle and the workspace that a program keeps beside its pools
        s["cache"] = ckv.Q4Cache(B=c["B"], Hkv=c["Hkv"], d=c["d"], pages=[s["pages"]], table=s["table"], lens=s["lens"],
                                 ring=s["ring"], state=s["state"])
        if "q" in s:
            n_q = s["q"].shape[1] if s["q"].dim() == 4 else 1
            n = ckv.chunkkv_q4_workspace_size(s["cache"], c["Hq"] // c["Hkv"], n_q, s["q"].dtype)
            s["ws"] = torch.zeros(n, dtype=torch.uint8, device=dev())
    cache = s["cache"]
    if c["kind"] in ("store", "step"):
        ckv.chunkkv_q4_append(cache, 0, s["k"], s["v"], s["counts"], s["slots"])
    if c["kind"] in ("store", "read"):
        ckv.chunkkv_q4_load(cache, 0, s["start"], s["cap"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    ckv.chunkkv_q4_attention(cache, 0, s["q"], s["out"], s["ws"], q_lens=s["q_lens"])
    return s["out"]


# ------------------------------------------------------------------ the plain forms

def _plain_append(s):
    nd = s["nd"]
    slots = s["slots"].view(-1)
    live = slots >= 0
    slot = slots[live]
    page, off = slot // PAGE, slot % PAGE
    touched, where = torch.unique(page, return_inverse=True)
    parts = _split(s["pages"], nd)
    for i, name in ((0, "k"), (1, "v")):
        c, m, step = _quantise(s[name].view(-1, s["case"]["d"])[live].float())
        codes = _codes(parts[2 * i][touched], i)
        codes[where, off] = c
        parts[2 * i][touched] = _bytes_of(codes, i)
        parts[2 * i + 1][page, :, off] = torch.stack([m, step], -1).to(torch.bfloat16)


def _plain_load(s):
    c = s["case"]
    tokens = torch.arange(s["cap"], device=dev())
    held = tokens < s["lens"][:, None]
    rows = s["table"].long()
    slot = (rows.gather(1, (tokens // PAGE).expand(rows.shape[0], -1)) * PAGE + tokens % PAGE)[held]
    at = (s["start"][:, None] + tokens)[held]
    for i, name in ((0, "k_out"), (1, "v_out")):
        s[name][at] = _values(s["pages"], i, s["nd"], c["d"]).reshape(-1, c["d"])[slot].to(s[name].dtype)


def _plain_attention(s):
    """softmax(q k^T / sqrt(d) + mask) v over the rows padded to one length."""
    c = s["case"]
    G, rows, d = c["Hq"] // c["Hkv"], s["table"].shape[0], c["d"]
    q = s["q"] if s["q"].dim() == 4 else s["q"][:, None]
    nq = q.shape[1]
    count = s["q_lens"] if s["q_lens"] is not None else torch.ones(c["B"], dtype=torch.int32, device=dev())
    i = torch.arange(nq, device=dev())
    live = i < count[:, None]
    sees = (s["lens"].view(c["B"], c["Hkv"], 1) - count[:, None, None] + 1 + i).view(rows, nq)    # keys that a query sees
    page = s["table"].long().clamp(min=0)
    n = page.shape[1] * PAGE
    qr = q.float().view(c["B"], nq, c["Hkv"], G, d).permute(0, 2, 3, 1, 4).reshape(rows, G * nq, d)
    k = _values(s["pages"], 0, s["nd"], d)[page].view(rows, n, d)
    p = torch.matmul(qr, k.transpose(1, 2)).mul_(1.0 / math.sqrt(d)).view(rows, G, nq, n)
    del k
    p.masked_fill_((torch.arange(n, device=dev()) >= sees[:, :, None])[:, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    v = _values(s["pages"], 1, s["nd"], d)[page].view(rows, n, d)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(rows, G * nq, n), v).view(rows, G, nq, d) / torch.where(total > 0, total, 1.0)
    o = o.view(c["B"], c["Hkv"], G, nq, d).permute(0, 3, 1, 2, 4).reshape(c["B"], nq, c["Hq"], d)
    out = s["out"].view(q.shape)
    out.copy_(torch.where(live[:, :, None, None], o, out.float()))


def run(state):
    if own:
        return _run_own(state)
    kind = state["case"]["kind"]
    if kind in ("store", "step"):
        _plain_append(state)
    if kind in ("store", "read"):
        _plain_load(state)
        return {"k": state["k_out"], "v": state["v_out"]}
    _plain_attention(state)
    return state["out"]


# ------------------------------------------------------------------ from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    d, nd = case["d"], s["nd"]
    lens = s["lens"].tolist()
    def of_row(r, which):
        """Row r's keys or values, code by code from the bytes: item i of 8 bytes is nibble p + 4 e of word w."""
        used = s["table"][r, :_pages(lens[r])].long()
        raw = s["pages"][used].long()
        item = torch.arange(16, device=dev())
        w, p, e = item // 8, item % 8 // 2, item % 2
        nib = p + 4 * e
        byte, up = 4 * w + nib // 2, 4 * (nib % 2)
        token, col = torch.arange(PAGE, device=dev())[:, None], torch.arange(d, device=dev())[None]
        if which == 0:
            at = ((token * 4 + col % 64 // 16) * nd + col // 64) * 8 + byte[col % 16]
            code = raw[:, at] >> up[col % 16] & 15
            base = 2048 * nd
        else:
            at = 2304 * nd + (((col // 16 * 8 + col % 8) * 4 + token // 16) * 2 + col % 16 // 8) * 8 + byte[token % 16]
            code = raw[:, at] >> up[token % 16] & 15
            base = 4352 * nd
        ms = base + ((col // 64) * PAGE + token) * 4

        def bf16(at):                   # two bytes as a number
            return ((raw[:, at] | raw[:, at + 1] << 8) << 16).to(torch.int32).view(torch.float32).double()
        return (code.double() * bf16(ms + 2) + bf16(ms)).reshape(-1, d)[:lens[r]]

    def rounded(x, up):
        """x in fp32 to bf16, upwards or downwards."""
        y = x.to(torch.bfloat16)
        to = torch.full_like(y, math.inf if up else -math.inf)
        short = y.float() < x if up else y.float() > x
        return torch.where(short, torch.nextafter(y, to), y).float()

    def held(x):
        """What tokens x [n, d] are held as, from the definition in the arithmetic that it names."""
        out = torch.zeros(x.shape, dtype=torch.float64, device=dev())
        for g in range(0, d, 64):
            y = x[:, g:g + 64].float()
            m = rounded(y.amin(1, keepdim=True), False)
            step = rounded((y.amax(1, keepdim=True) - m) * (1.0 / 15.0), True)
            c = torch.round((y - m) * (1.0 / step.clamp(min=SMALLEST / 64))).clamp(0, 15).double()
            out[:, g:g + 64] = torch.where(step >= SMALLEST / 16, c * step.double(), 0.0) + m.double()
        return out

    if case["kind"] in ("store", "read"):
        out = [torch.zeros(s["k_out"].shape, dtype=torch.float64, device=dev()) for _ in range(2)]
        new = s["counts"].view(-1).tolist() if case["kind"] == "store" else [0] * len(lens)
        for r, n in enumerate(lens):
            b, h = divmod(r, case["Hkv"])
            for i, name in ((0, "k"), (1, "v")):
                if n:
                    x = of_row(r, i)
                    if new[r]:
                        x[n - new[r]:] = held(s[name][b, h, :new[r]])
                    out[i][r * s["cap"]:r * s["cap"] + n] = x
        return {"k": out[0], "v": out[1]}
    if work(case)["flops"] > 6e12:
        return None
    q = s["q"].double().view(case["B"], -1, case["Hq"], d)
    out = torch.zeros_like(q)
    G = case["Hq"] // case["Hkv"]
    for r, n in enumerate(lens):
        b, h = divmod(r, case["Hkv"])
        if n == 0:
            continue
        k, v = of_row(r, 0), of_row(r, 1)
        if case["kind"] == "step":
            k[n - 1], v[n - 1] = held(s["k"][b, h, :1])[0], held(s["v"][b, h, :1])[0]     # the token just written
        m = int(s["q_lens"][b]) if s["q_lens"] is not None else 1
        for g in range(G):
            for a in range(0, m, 2048):
                z = min(a + 2048, m)
                x = q[b, a:z, h * G + g] @ k.T / math.sqrt(d)
                sees = n - m + 1 + torch.arange(a, z, device=dev())
                x = x.masked_fill(torch.arange(n, device=dev())[None] >= sees[:, None], -math.inf)
                p = torch.softmax(x, -1).masked_fill((sees <= 0)[:, None], 0.0)
                out[b, a:z, h * G + g] = p @ v
    return out.view(s["q"].shape)
