"""One attention layer served with a compressed cache in 8 or 4 bits, from the prompt to decoding.

    python examples/serve_layer.py [--bits 4]

Ragged prompts go through causal attention (prefill_attention); ChunkKV keeps the best chunks of every KV head
(compress_layers); the kept rows go into the 8-bit paged cache (chunkkv_q8_resize, chunkkv_q8_append); every decoded
token is appended to it and attends to it (q8_attention); and when the caches have grown, they are read back,
compressed again and written anew (chunkkv_q8_load, compress_layers).  With --bits 4 the cache is the 4-bit one (the
chunkkv_q4 calls), and before decoding the conversation has a next turn: tokens of a second prompt, as many as each
sequence has, are appended together and attend to the cache and among themselves (q4_attention with q_lens).  The data
is synthetic; every output is compared with attention in 64 bits over the same tokens before their rounding.
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import chunk_level_kv_gb300 as ckv  # noqa: E402


class Layer:
    """The cache of one layer, with a copy of its rows in full precision for the comparison."""

    def __init__(self, B: int, Hkv: int, G: int, d: int, most_tokens: int, device, bits: int = 8, most_queries: int = 1):
        self.B, self.Hkv, self.G, self.d, self.dev, self.bits = B, Hkv, G, d, device, bits
        pages = -(-most_tokens // ckv.Q8_PAGE)
        make, self.resize, self.write, self.load = {
            8: (ckv.q8_cache, ckv.chunkkv_q8_resize, ckv.chunkkv_q8_append, ckv.chunkkv_q8_load),
            4: (ckv.q4_cache, ckv.chunkkv_q4_resize, ckv.chunkkv_q4_append, ckv.chunkkv_q4_load)}[bits]
        self.cache = make(B, Hkv, d, n_pages=B * Hkv * pages, max_pages=pages, device=device)
        if bits == 8:
            size = ckv.chunkkv_q8_workspace_size(self.cache, G)
        else:
            size = max(ckv.chunkkv_q4_workspace_size(self.cache, G, n) for n in (1, most_queries))
        self.ws = torch.zeros(size, dtype=torch.uint8, device=device)
        self.k = [torch.empty(0, d, device=device) for _ in range(B * Hkv)]
        self.v = [torch.empty(0, d, device=device) for _ in range(B * Hkv)]

    def append(self, k, v, counts):
        """Writes the first counts[b][h] tokens of k, v [B, Hkv, n, d] behind each row; all or nothing."""
        counts = counts.reshape(-1).to(torch.int32).contiguous()
        slots = torch.empty(self.cache.rows, k.shape[2], dtype=torch.int64, device=self.dev)
        self.resize(self.cache, self.cache.lens + counts, slots)
        if self.cache.state[2].item() != 0:
            raise RuntimeError("the cache has too few pages")
        self.write(self.cache, 0, k, v, counts, slots)
        for r, n in enumerate(counts.tolist()):
            b, h = divmod(r, self.Hkv)
            self.k[r] = torch.cat([self.k[r], k[b, h, :n].float()])
            self.v[r] = torch.cat([self.v[r], v[b, h, :n].float()])

    def clear(self):
        self.resize(self.cache, torch.zeros_like(self.cache.lens))
        self.k = [x[:0] for x in self.k]
        self.v = [x[:0] for x in self.v]

    def read(self):
        """The rows as they are held, packed: (k, v) [tokens, d] and the rows' offsets."""
        lens = self.cache.lens.tolist()
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        k = torch.empty(cu[-1], self.d, dtype=torch.bfloat16, device=self.dev)
        v = torch.empty_like(k)
        start = torch.tensor(cu[:-1], dtype=torch.int64, device=self.dev)
        self.load(self.cache, 0, start, max(lens), k, v)
        return k, v, cu

    def attend(self, q, q_lens=None):
        """One query token a sequence, or (4 bits) several: the last q_lens[b] tokens of every row are theirs."""
        if self.bits == 8:
            return ckv.q8_attention(self.cache, 0, q, workspace=self.ws)
        return ckv.q4_attention(self.cache, 0, q, q_lens=q_lens, workspace=self.ws)

    def error(self, q, out, q_lens=None) -> float:
        """Relative error of an output against 64 bits over the rows before their rounding."""
        if q.dim() == 3:
            q, out = q[:, None], out[:, None]
        want = torch.zeros_like(out, dtype=torch.float64)
        for r in range(self.cache.rows):
            b, h = divmod(r, self.Hkv)
            m = q.shape[1] if q_lens is None else int(q_lens[b])
            n = len(self.k[r])
            qr = q[b, :m, h * self.G:(h + 1) * self.G].double()
            logits = torch.einsum("mgd,nd->mgn", qr, self.k[r].double()) / math.sqrt(self.d)
            hidden = torch.arange(n, device=self.dev) > n - m + torch.arange(m, device=self.dev)[:, None]
            p = torch.softmax(logits.masked_fill(hidden[:, None], -math.inf), -1)
            want[b, :m, h * self.G:(h + 1) * self.G] = p @ self.v[r].double()
        return float((out.double() - want).norm() / want.norm())


def serve(seqlens=(700, 1500, 333), Hkv=2, G=4, d=128, w=16, c=10, budget=200, steps=40, again_at=24, seed=0, bits=8,
          turn=(120, 37, 200)) -> dict:
    assert again_at >= w, "the second compression scores with the last w decoded queries"
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev).to(torch.bfloat16)
    B, Hq = len(seqlens), Hkv * G
    cu = [0]
    for n in seqlens:
        cu.append(cu[-1] + n)

    # the prompts
    q, k, v = normal(cu[-1], Hq, d), normal(cu[-1], Hkv, d), normal(cu[-1], Hkv, d)
    hidden = ckv.prefill_attention(q, k, v, cu)

    # the kept chunks of every head, into the cache
    window = torch.stack([q[e - w:e] for e in cu[1:]])
    kept = ckv.compress_layers([window], [k], [v], cu, Hq=Hq, Hkv=Hkv, w=w, c=c, L_max=budget)
    next_turn = list(turn[:B]) if bits == 4 else [0] * B
    layer = Layer(B, Hkv, G, d, budget + w + steps + c + max(next_turn), dev, bits, max(1, *next_turn))
    layer.append(kept.k_out[0], kept.v_out[0], kept.counts[0])
    lengths = [layer.cache.lens.tolist()]

    # the next turn's tokens, a padded batch: into the cache, and then over it
    turn_error = None
    if bits == 4:
        q_lens = torch.tensor(next_turn, dtype=torch.int32, device=dev)
        n = max(next_turn)
        qt, kt, vt = normal(B, n, Hq, d), normal(B, Hkv, n, d), normal(B, Hkv, n, d)
        layer.append(kt, vt, q_lens[:, None].expand(B, Hkv))
        turn_error = layer.error(qt, layer.attend(qt, q_lens), next_turn)

    # decoding
    errors, queries = [], []
    for step in range(steps):
        q1, k1, v1 = normal(B, Hq, d), normal(B, Hkv, d), normal(B, Hkv, d)
        layer.append(k1[:, :, None], v1[:, :, None], torch.ones(B, Hkv, device=dev))
        out = layer.attend(q1)
        errors.append(layer.error(q1, out))
        queries.append(q1)
        if step + 1 == again_at:
            # the caches have grown: every head's cache is a sequence of its own now, with its group's queries
            lengths.append(layer.cache.lens.tolist())
            kr, vr, rows = layer.read()
            window = torch.stack(queries[-w:], 1).view(B, w, Hkv, G, d).transpose(1, 2).reshape(B * Hkv, w, G, d)
            kept = ckv.compress_layers([window.contiguous()], [kr[:, None]], [vr[:, None]], rows, Hq=G, Hkv=1, w=w, c=c,
                                       L_max=budget)
            layer.clear()
            layer.append(kept.k_out[0].view(B, Hkv, -1, d), kept.v_out[0].view(B, Hkv, -1, d), kept.counts[0])
            lengths.append(layer.cache.lens.tolist())
    lengths.append(layer.cache.lens.tolist())
    ckv.chunkkv_status_check(layer.ws)
    return {"hidden": hidden, "errors": errors, "lengths": lengths, "free_pages": int(layer.cache.state[1]),
            "turn_error": turn_error}


if __name__ == "__main__":
    import argparse
    parser = argparse.ArgumentParser()
    parser.add_argument("--bits", type=int, choices=(8, 4), default=8)
    result = serve(bits=parser.parse_args().bits)
    print("tokens per cache row after the prompt, before and after the second compression, at the end:")
    for row in result["lengths"]:
        print("   ", row)
    if result["turn_error"] is not None:
        print(f"relative error of the next turn's tokens against 64 bits before rounding: {result['turn_error']:.4f}")
    print(f"relative error of the decoded tokens against 64 bits before rounding: largest {max(result['errors']):.4f}")
