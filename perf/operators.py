"""What is timed of the serving operators around the compression, and their plain forms.

Four kinds of case, in the order in which a serving program meets them:
  prefill  causal attention over packed prompts with grouped heads (chunkkv_prefill_attention)
  tables   block tables and slot maps of the 8-bit cache from lengths (chunkkv_q8_resize)
  store    rows written into the 8-bit cache and read back (chunkkv_q8_append, chunkkv_q8_load)
  decode   one query token per sequence over the 8-bit cache (chunkkv_q8_attention)

The 8-bit cache.  A cache row r = b * Hkv + h is one (sequence, KV head) with a length of its own (chunk
compression keeps another number of tokens for each head).  A page holds 64 tokens of one row: keys as
int8 [ceil(d / 64), 64 tokens, 64], values transposed as int8 [64 ceil(d / 64), 64 tokens], and one fp32 scale each
for the page's keys and values; columns at or beyond d are zero.  table[r][j] is the page of tokens 64 j ..
64 j + 63 of row r.  Free pages wait in a ring (first in, first out): state = (head, number free, status, 0).
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev():
    return torch.device("cuda:0")


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one LLaMA-3-8B-shaped prefill layer, the length of the framework's single-layer workload
        dict(name="prefill_llama_8192", kind="prefill", B=1, qmin=8192, qmax=8192, prefix=0, Hq=32, Hkv=8, d=128,
             dtype="bf16", lens=1),
        # a long prompt of the Qwen2-7B shape (groups of 7 query heads)
        dict(name="prefill_qwen_16384", kind="prefill", B=1, qmin=16384, qmax=16384, prefix=0, Hq=28, Hkv=4, d=128,
             dtype="bf16", lens=2),
        # a batch of ordinary ragged prompts packed together, Mistral-7B-shaped
        dict(name="prefill_ragged_16", kind="prefill", B=16, qmin=100, qmax=2000, prefix=0, Hq=32, Hkv=8, d=128,
             dtype="bf16", lens=3),
        # the next turns of two conversations: new tokens against a prefix that the cache already holds
        dict(name="prefill_next_turn", kind="prefill", B=2, qmin=300, qmax=700, prefix=9001, Hq=32, Hkv=8, d=128,
             dtype="bf16", lens=4),
        # the framework's small fp32 layer
        dict(name="prefill_tiny_f32", kind="prefill", B=1, qmin=512, qmax=512, prefix=0, Hq=4, Hkv=2, d=64,
             dtype="f32", lens=5),
        # a serving step: each row of 256 sequences grows by a token; some are cut (compressed again) or end
        dict(name="tables_step", kind="tables", rows=2048, now=288, new=1, churn=0.03, n_cap=288, lens=6),
        # sixteen compressed prompts are admitted at once
        dict(name="tables_admit", kind="tables", rows=128, now=0, new=6582, churn=0.0, n_cap=6582, lens=7),
        # the kept rows of a 32K prompt at a 20 % budget are written after compression
        dict(name="store_llama_kept", kind="store", B=1, Hkv=8, d=128, dtype="bf16", old=0, new=6582, lens=8),
        # tokens decoded since join small caches (budget 256), inside a page that is already open
        dict(name="store_tail", kind="store", B=16, Hkv=8, d=128, dtype="bf16", old=288, new=37, lens=9),
        # one sequence decodes over its compressed 32K prompt: latency
        dict(name="decode_llama_6582", kind="decode", B=1, Hq=32, Hkv=8, d=128, dtype="bf16", lmin=6500, lmax=6582,
             lens=10),
        # sixteen sequences with a budget of 256: the smallest call
        dict(name="decode_mistral_16", kind="decode", B=16, Hq=32, Hkv=8, d=128, dtype="bf16", lmin=256, lmax=300,
             lens=11),
        # a large batch over compressed 128K prompts
        dict(name="decode_qwen_64", kind="decode", B=64, Hq=28, Hkv=4, d=128, dtype="bf16", lmin=12000, lmax=13164,
             lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["prefill", "tables", "store", "decode"])
    Hq, Hkv, d, dtype = rng.choice([(32, 8, 128, "bf16"), (28, 4, 128, "bf16"), (8, 8, 64, "bf16"), (4, 2, 64, "f32"),
                                    (12, 2, 80, "bf16"), (16, 1, 128, "bf16"), (6, 2, 128, "f32")])
    lens = rng.randrange(1 << 20)
    if kind == "prefill":
        B = rng.choice([1, 1, 2, 5, 16])
        top = _log(rng, 40, (12000 if dtype == "bf16" else 2000) // (1 if B == 1 else B // 2 + 1))
        return dict(kind=kind, B=B, qmin=max(1, top // rng.choice([1, 3, 20])), qmax=top,
                    prefix=rng.choice([0, 0, _log(rng, 1, 5000)]), Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, lens=lens)
    if kind == "tables":
        rows = _log(rng, 8, 4096)
        new = rng.choice([1, _log(rng, 1, max(2, 800000 // rows))])
        return dict(kind=kind, rows=rows, now=_log(rng, 1, 3000), new=min(new, 8000), churn=rng.choice([0.0, 0.1]),
                    n_cap=max(min(new, 8000), 64), lens=lens)
    if kind == "store":
        B = _log(rng, 1, 32)
        return dict(kind=kind, B=B, Hkv=Hkv, d=d, dtype=dtype, old=rng.choice([0, _log(rng, 1, 700)]),
                    new=_log(rng, 1, max(2, 50000 // (B * Hkv))), lens=lens)
    B = _log(rng, 1, 64)
    top = _log(rng, 16, min(40000, 3000000 // (B * Hkv)))
    return dict(kind=kind, B=B, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, lmin=rng.choice([0, top // 2, top]), lmax=top, lens=lens)


def _lens(case):
    """The case's lengths, one per prompt or cache row, the same for every seed."""
    r = random.Random(case["lens"])
    if case["kind"] == "prefill":
        q = [r.randint(case["qmin"], case["qmax"]) for _ in range(case["B"])]
        return q, [n + (r.randint(case["prefix"] // 2, case["prefix"]) if case["prefix"] else 0) for n in q]
    if case["kind"] == "tables":
        low = max(1, (case["now"] * 9) // 10)
        a = [r.randint(low, case["now"]) if case["now"] else 0 for _ in range(case["rows"])]
        b = []
        for n in a:
            gone = r.random() < case["churn"]
            b.append(r.randint(0, 1) * r.randint(1, case["n_cap"]) if gone else n + (1 if case["new"] == 1 else r.randint(
                max(1, (case["new"] * 9) // 10), case["new"])))
        # one call maps at most n_cap new tokens a row
        return a, [min(n, m + case["n_cap"]) for n, m in zip(b, a)]
    rows = case["B"] * case["Hkv"]
    if case["kind"] == "store":
        old = [r.randint(case["old"] // 2, case["old"]) if case["old"] else 0 for _ in range(rows)]
        return old, [r.randint((case["new"] * 9) // 10, case["new"]) for _ in range(rows)]
    return [r.randint(case["lmin"], case["lmax"]) for _ in range(rows)]


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _d64(d):
    return (d + 63) // 64 * 64


def work(case):
    if case["kind"] == "prefill":
        q, k = _lens(case)
        elt = 2 if case["dtype"] == "bf16" else 4
        pairs = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(q, k))
        return {"bytes": elt * case["d"] * (2 * sum(q) * case["Hq"] + 2 * sum(k) * case["Hkv"]),
                "flops": 4 * case["d"] * case["Hq"] * pairs}
    if case["kind"] == "tables":        # there and back: lengths, the slot maps, pages that change hands
        a, b = _lens(case)
        moved = sum(abs(_pages(n) - _pages(m)) for n, m in zip(a, b))
        return {"bytes": 2 * (12 * len(a) + 8 * len(a) * case["n_cap"] + 8 * moved), "flops": 0}
    elt = 2 if case["dtype"] == "bf16" else 4
    if case["kind"] == "store":         # new rows in, their codes out; every row's codes in, the rows out
        old, new = _lens(case)
        n, m = sum(new), sum(old) + sum(new)
        return {"bytes": 2 * case["d"] * (n * (elt + 1) + m * (elt + 1)), "flops": 0}
    n = sum(_lens(case))
    qo = 2 * case["B"] * case["Hq"] * case["d"] * elt
    return {"bytes": 2 * case["d"] * n + qo, "flops": 4 * case["d"] * n * (case["Hq"] // case["Hkv"])}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=dev()).manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=dev())


def _chan(g, *shape):
    """Per-channel scales of keys: a few channels are much larger than the rest, as in trained models."""
    return torch.rand(*shape, generator=g, device=dev()) * 1.5 + 0.5


def _cumulative(ns):
    out = [0]
    for n in ns:
        out.append(out[-1] + n)
    return out


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
    s = {"case": case}
    if case["kind"] == "prefill":
        ql, kl = _lens(case)
        dt = DTYPES[case["dtype"]]
        s["cu_q"], s["cu_k"] = _cumulative(ql), _cumulative(kl)
        s["q"] = _normal(g, sum(ql), case["Hq"], case["d"]).to(dt)
        s["k"] = (_normal(g, sum(kl), case["Hkv"], case["d"]) * _chan(g, case["Hkv"], case["d"])).to(dt)
        s["v"] = _normal(g, sum(kl), case["Hkv"], case["d"]).to(dt)
        s["out"] = torch.zeros_like(s["q"])
        return s
    if case["kind"] == "tables":
        a, b = _lens(case)
        need = sum(max(_pages(n), _pages(m)) for n, m in zip(a, b))
        s["max_pages"] = max(_pages(max(n, m)) for n, m in zip(a, b))
        s["n_pages"] = need + 64
        s["table"], s["ring"], s["state"] = _layout([_pages(n) for n in a], s["max_pages"], s["n_pages"], g)
        s["lens"], s["there"], s["back"] = _int32(a), _int32(b), _int32(a)
        s["slots"] = [torch.full((len(a), case["n_cap"]), -1, dtype=torch.int64, device=dev()) for _ in range(2)]
        return s
    dt = DTYPES[case["dtype"]]
    d, d64 = case["d"], _d64(case["d"])
    if case["kind"] == "store":
        old, new = _lens(case)
        lens = [n + m for n, m in zip(old, new)]
    else:
        lens = _lens(case)
        old = lens
    rows = len(lens)
    s["max_pages"] = max(1, max(_pages(n) for n in lens))
    s["n_pages"] = sum(_pages(n) for n in lens) + 3
    s["table"], s["ring"], s["state"] = _layout([_pages(n) for n in lens], s["max_pages"], s["n_pages"], g)
    s["lens"] = _int32(lens)
    # what earlier steps wrote, quantised page by page (stale codes past the rows' ends included)
    chan = _chan(g, d)
    s["k_pages"] = torch.zeros(s["n_pages"], d64 // 64, PAGE, 64, dtype=torch.int8, device=dev())
    s["v_pages"] = torch.zeros(s["n_pages"], d64, PAGE, dtype=torch.int8, device=dev())
    s["scales"] = torch.zeros(s["n_pages"], 2, device=dev())
    for at in range(0, s["n_pages"], 8192):
        n = min(8192, s["n_pages"] - at)
        for i in range(2):
            x = _normal(g, n, PAGE, d) * (chan if i == 0 else 1.0)
            top = x.abs().amax((1, 2))
            code = torch.zeros(n, PAGE, d64, dtype=torch.int8, device=dev())
            code[:, :, :d] = torch.round(x * (127.0 / top)[:, None, None]).to(torch.int8)
            s["scales"][at:at + n, i] = top / 127.0
            if i == 0:
                s["k_pages"][at:at + n] = code.view(n, PAGE, d64 // 64, 64).transpose(1, 2)
            else:
                s["v_pages"][at:at + n] = code.transpose(1, 2)
    if case["kind"] == "store":
        cap = max(max(new), 1)
        s["k"] = (_normal(g, case["B"], case["Hkv"], cap, d) * chan).to(dt)
        s["v"] = _normal(g, case["B"], case["Hkv"], cap, d).to(dt)
        s["counts"] = _int32(new).view(case["B"], case["Hkv"])
        pos = _int32(old).long()[:, None] + torch.arange(cap, device=dev())
        page = s["table"].long().gather(1, (pos // PAGE).clamp(max=s["max_pages"] - 1))
        fill = torch.arange(cap, device=dev()) < _int32(new)[:, None]
        s["slots"] = torch.where(fill, page * PAGE + pos % PAGE, -1)
        s["cap"] = max(lens)
        s["start"] = torch.arange(rows, device=dev()) * s["cap"]
        s["k_out"] = torch.zeros(rows * s["cap"], d, dtype=dt, device=dev())
        s["v_out"] = torch.zeros(rows * s["cap"], d, dtype=dt, device=dev())
        return s
    s["q"] = _normal(g, case["B"], case["Hq"], d).to(dt)
    s["out"] = torch.zeros_like(s["q"])
    return s


# ------------------------------------------------------------------ the framework's operators

def _cache(s):
    if "cache" not in s:                # the handle that a program keeps beside its pools
        import chunk_level_kv_gb300 as ckv
        c = s["case"]
        s["cache"] = ckv.Q8Cache(B=c.get("B", c.get("rows")), Hkv=c.get("Hkv", 1), d=c.get("d", 64),
                                 k_pages=[s["k_pages"]] if "k_pages" in s else [],
                                 v_pages=[s["v_pages"]] if "v_pages" in s else [],
                                 scales=[s["scales"]] if "scales" in s else [],
                                 table=s["table"], lens=s["lens"], ring=s["ring"], state=s["state"])
    return s["cache"]


def _run_own(s):
    import chunk_level_kv_gb300 as ckv
    kind = s["case"]["kind"]
    if kind == "prefill":
        if "plan" not in s:
            s["plan"] = ckv.prefill_params_for(s["q"], s["k"], s["cu_q"], s["cu_k"])
            s["ws"] = torch.zeros(ckv.chunkkv_prefill_workspace_size(s["plan"][0]), dtype=torch.uint8, device=dev())
        ckv.chunkkv_prefill_attention(s["plan"][0], s["q"], s["k"], s["v"], s["out"], s["ws"])
        return s["out"]
    cache = _cache(s)
    if kind == "tables":
        ckv.chunkkv_q8_resize(cache, s["there"], s["slots"][0])
        ckv.chunkkv_q8_resize(cache, s["back"], s["slots"][1])
        return {"slots": s["slots"], "table": s["table"], "lens": s["lens"], "ring": s["ring"], "state": s["state"]}
    if kind == "store":
        ckv.chunkkv_q8_append(cache, 0, s["k"], s["v"], s["counts"], s["slots"])
        ckv.chunkkv_q8_load(cache, 0, s["start"], s["cap"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"], "scales": s["scales"]}
    if "ws" not in s:
        s["ws"] = torch.zeros(ckv.chunkkv_q8_workspace_size(cache, s["case"]["Hq"] // s["case"]["Hkv"]), dtype=torch.uint8,
                              device=dev())
    ckv.chunkkv_q8_attention(cache, 0, s["q"], s["out"], s["ws"])
    return s["out"]


# ------------------------------------------------------------------ the plain forms

def _pad_index(cu, top):
    start = torch.tensor(cu[:-1], device=dev())
    n = torch.tensor(cu[1:], device=dev()) - start
    i = torch.arange(top, device=dev())
    return (start[:, None] + i).clamp(max=max(cu[-1] - 1, 0)), i < n[:, None], n


def _plain_prefill(s):
    """softmax(q k^T / sqrt(d) + mask) v over the prompts padded to one length."""
    c = s["case"]
    G = c["Hq"] // c["Hkv"]
    qi, q_in, qn = _pad_index(s["cu_q"], max(b - a for a, b in zip(s["cu_q"], s["cu_q"][1:])))
    ki, _, kn = _pad_index(s["cu_k"], max(b - a for a, b in zip(s["cu_k"], s["cu_k"][1:])))
    B, Tq, Tk = c["B"], qi.shape[1], ki.shape[1]
    q = s["q"].float()[qi].view(B, Tq, c["Hkv"], G, c["d"]).permute(0, 2, 3, 1, 4).reshape(B, c["Hkv"], G * Tq, c["d"])
    k = s["k"].float()[ki].permute(0, 2, 3, 1)
    v = s["v"].float()[ki].permute(0, 2, 1, 3)
    last = (kn - qn)[:, None] + torch.arange(Tq, device=dev())           # the last key that a query sees
    hidden = torch.arange(Tk, device=dev()) > last[:, :, None]
    p = torch.matmul(q, k).mul_(1.0 / math.sqrt(c["d"])).view(B, c["Hkv"], G, Tq, Tk)
    p.masked_fill_(hidden[:, None, None], -math.inf)
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(p.view(B, c["Hkv"], G * Tq, Tk), v) / p.sum(-1).view(B, c["Hkv"], G * Tq, 1)
    o = o.view(B, c["Hkv"], G, Tq, c["d"]).permute(0, 3, 1, 2, 4).reshape(B, Tq, c["Hq"], c["d"])
    s["out"].copy_(o[q_in])
    return s["out"]


def _plain_resize(s, new, slots):
    table, ring, state, lens = s["table"], s["ring"], s["state"], s["lens"]
    n_pages, width, cap = s["n_pages"], s["max_pages"], slots.shape[1]
    have, need = (lens + PAGE - 1) // PAGE, (new + PAGE - 1) // PAGE
    grow, give = (need - have).clamp(min=0), (have - need).clamp(min=0)
    g_total, s_total = grow.sum(), give.sum()
    bad = ((new < 0) | (need > width) | (new - lens > cap)).any()
    short = g_total > state[1]
    fine = ~bad & ~short
    j = torch.arange(width, device=dev())
    takes = (j >= have[:, None]) & (j < need[:, None]) & fine
    gives = (j >= need[:, None]) & (j < have[:, None]) & fine
    taken = (state[0] + (grow.cumsum(0) - grow - have)[:, None] + j) % n_pages
    after = torch.where(takes, ring[taken.clamp(min=0)], table)
    # pages given back join the ring behind those that are free
    to = (state[0] + state[1] + (give.cumsum(0) - give - need)[:, None] + j) % n_pages
    wide = torch.cat([ring, ring.new_zeros(1)])
    wide.scatter_(0, torch.where(gives, to, n_pages).view(-1), table.view(-1))
    ring.copy_(wide[:n_pages])
    table.copy_(torch.where(gives, -1, after))
    i = torch.arange(cap, device=dev())
    pos = lens[:, None].long() + i
    page = table.long().gather(1, (pos // PAGE).clamp(max=width - 1))
    slots.copy_(torch.where((i < (new - lens)[:, None]) & fine, page * PAGE + pos % PAGE, -1))
    moved = torch.stack([(state[0] + g_total) % n_pages, state[1] - g_total + s_total, state[2] * 0, state[3]])
    kept = torch.stack([state[0].long(), state[1].long(), torch.where(bad, 2, 1), state[3].long()])
    state.copy_(torch.where(fine, moved, kept))
    lens.copy_(torch.where(fine, new, lens))


def _codes(s, name):
    """A pool's codes as [n_pages, 64 tokens, d]."""
    c = s["case"]
    if name == "k_pages":
        return s[name].transpose(1, 2).reshape(s["n_pages"], PAGE, _d64(c["d"]))[:, :, :c["d"]]
    return s[name].transpose(1, 2)[:, :, :c["d"]]


def _plain_store(s):
    c = s["case"]
    d, n_pages = c["d"], s["n_pages"]
    slots = s["slots"].view(-1)
    live = slots >= 0
    slot = slots[live]
    page = slot // PAGE
    fresh = torch.zeros(n_pages, dtype=torch.bool, device=dev())
    fresh[page[slot % PAGE == 0]] = True
    rows = s["table"].long()
    tokens = torch.arange(s["cap"], device=dev())
    held = tokens < s["lens"][:, None]
    where = rows.gather(1, (tokens // PAGE).expand(rows.shape[0], -1))[held] * PAGE + (tokens % PAGE).expand_as(held)[held]
    at = (s["start"][:, None] + tokens)[held]
    for i, name in ((0, "k"), (1, "v")):
        x = s[name].float().view(-1, d)[live]
        top = torch.zeros(n_pages, device=dev()).scatter_reduce_(0, page, x.abs().amax(1), "amax")
        grown = torch.where(top >= 2.0 ** -100, top * float(np.float32(1) / np.float32(127)), 0.0)
        before = torch.where(fresh, 0.0, s["scales"][:, i])
        scale = torch.maximum(before, grown)
        ratio = torch.where(scale > before, before / scale, 1.0)
        codes = torch.round(_codes(s, name + "_pages").float() * ratio[:, None, None]).reshape(n_pages * PAGE, d)
        inv = torch.where(scale > 0, torch.reciprocal(scale), 0.0)
        codes[slot] = torch.round(x * inv[page][:, None]).clamp(-127, 127)
        codes = codes.view(n_pages, PAGE, d)
        if name == "k":
            full = s["k_pages"].transpose(1, 2).reshape(n_pages, PAGE, _d64(d)).clone()
            full[:, :, :d] = codes.to(torch.int8)
            s["k_pages"].copy_(full.view(n_pages, PAGE, -1, 64).transpose(1, 2))
        else:
            s["v_pages"][:, :d] = codes.transpose(1, 2).to(torch.int8)
        s["scales"][:, i] = scale
        values = codes * scale[:, None, None]
        s[name + "_out"][at] = values.reshape(-1, d)[where].to(s[name].dtype)
    return {"k": s["k_out"], "v": s["v_out"], "scales": s["scales"]}


def _plain_decode(s):
    c = s["case"]
    G, rows = c["Hq"] // c["Hkv"], s["table"].shape[0]
    page = s["table"].long().clamp(min=0)
    n = page.shape[1] * PAGE
    k = (_codes(s, "k_pages")[page].float() * s["scales"][:, 0][page][:, :, None, None]).reshape(rows, n, c["d"])
    q = s["q"].float().view(rows, G, c["d"])
    p = torch.matmul(q, k.transpose(1, 2)) * (1.0 / math.sqrt(c["d"]))
    del k
    p.masked_fill_((torch.arange(n, device=dev()) >= s["lens"][:, None])[:, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p = torch.exp(p - torch.where(top > -math.inf, top, 0.0))
    v = (_codes(s, "v_pages")[page].float() * s["scales"][:, 1][page][:, :, None, None]).reshape(rows, n, c["d"])
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    s["out"].copy_(o.view(c["B"], c["Hq"], c["d"]))
    return s["out"]


def run(state):
    if own:
        return _run_own(state)
    kind = state["case"]["kind"]
    if kind == "prefill":
        return _plain_prefill(state)
    if kind == "tables":
        _plain_resize(state, state["there"], state["slots"][0])
        _plain_resize(state, state["back"], state["slots"][1])
        return {"slots": state["slots"], "table": state["table"], "lens": state["lens"], "ring": state["ring"],
                "state": state["state"]}
    return _plain_store(state) if kind == "store" else _plain_decode(state)


# ------------------------------------------------------------------ from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "prefill":
        if work(case)["flops"] > 6e12:
            return None
        out = torch.zeros(s["cu_q"][-1], case["Hq"], case["d"], dtype=torch.float64, device=dev())
        G = case["Hq"] // case["Hkv"]
        for b in range(case["B"]):
            q0, q1, k0, k1 = s["cu_q"][b], s["cu_q"][b + 1], s["cu_k"][b], s["cu_k"][b + 1]
            for h in range(case["Hq"]):
                for a in range(q0, q1, 4096):
                    z = min(a + 4096, q1)
                    sees = k1 - k0 - (q1 - z)                            # keys that the last of these rows sees
                    k, v = s["k"][k0:k0 + sees, h // G].double(), s["v"][k0:k0 + sees, h // G].double()
                    x = s["q"][a:z, h].double() @ k.T / math.sqrt(case["d"])
                    x.masked_fill_(torch.ones_like(x, dtype=torch.bool).triu(sees - (z - a) + 1), -math.inf)
                    out[a:z, h] = torch.softmax(x, -1) @ v
        return out
    if case["kind"] == "tables":
        return None                     # whole numbers alone
    d = case["d"]

    def row_values(pages, i):
        x = s["k_pages"][pages].permute(0, 2, 1, 3) if i == 0 else s["v_pages"][pages].transpose(1, 2)
        x = x.reshape(len(pages), PAGE, -1)[:, :, :d].double() * s["scales"][pages, i].double()[:, None, None]
        return x.reshape(-1, d)

    if case["kind"] == "store":
        # each page's scale and codes from the definition; a code whose rounding hangs on the arithmetic's last bit may
        # differ by one, so the rows' values are not given here: the scales are
        scales = s["scales"].double().clone()
        rows, cap = s["slots"].shape
        for i, x in ((0, s["k"]), (1, s["v"])):
            top = x.double().abs().amax(-1).view(rows, cap)
            slots = s["slots"]
            for off in range(PAGE):     # the token at each place of a page
                m = (slots >= 0) & (slots % PAGE == off)
                if off == 0:
                    scales[slots[m] // PAGE, i] = top[m] / 127
                else:
                    p = slots[m] // PAGE
                    scales[p, i] = torch.maximum(scales[p, i], top[m] / 127)
        return {"k": None, "v": None, "scales": scales}
    out = torch.zeros(case["B"], case["Hq"], d, dtype=torch.float64, device=dev())
    G = case["Hq"] // case["Hkv"]
    lens = s["lens"].tolist()
    for r, n in enumerate(lens):
        if n == 0:
            continue
        used = s["table"][r, :_pages(n)].long()
        k, v = row_values(used, 0)[:n], row_values(used, 1)[:n]
        b, h = divmod(r, case["Hkv"])
        q = s["q"][b, h * G:(h + 1) * G].double()
        out[b, h * G:(h + 1) * G] = torch.softmax(q @ k.T / math.sqrt(d), -1) @ v
    return out
