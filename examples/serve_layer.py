"""One attention layer served with a compressed 8-bit cache, from the prompt to decoding.

    python examples/serve_layer.py

Ragged prompts go through causal attention (prefill_attention); ChunkKV keeps the best chunks of every KV head
(compress_layers); the kept rows go into the 8-bit paged cache (chunkkv_q8_resize, chunkkv_q8_append); every decoded
token is appended to it and attends to it (q8_attention); and when the caches have grown, they are read back,
compressed again and written anew (chunkkv_q8_load, compress_layers).  The data is synthetic; every decoded
token's output is compared with attention in 64 bits over the same tokens before their rounding to 8 bits.
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

    def __init__(self, B: int, Hkv: int, G: int, d: int, most_tokens: int, device):
        self.B, self.Hkv, self.G, self.d, self.dev = B, Hkv, G, d, device
        pages = -(-most_tokens // ckv.Q8_PAGE)
        self.cache = ckv.q8_cache(B, Hkv, d, n_pages=B * Hkv * pages, max_pages=pages, device=device)
        self.ws = torch.zeros(ckv.chunkkv_q8_workspace_size(self.cache, G), dtype=torch.uint8, device=device)
        self.k = [torch.empty(0, d, device=device) for _ in range(B * Hkv)]
        self.v = [torch.empty(0, d, device=device) for _ in range(B * Hkv)]

    def append(self, k, v, counts):
        """Writes the first counts[b][h] tokens of k, v [B, Hkv, n, d] behind each row; all or nothing."""
        counts = counts.reshape(-1).to(torch.int32).contiguous()
        slots = torch.empty(self.cache.rows, k.shape[2], dtype=torch.int64, device=self.dev)
        ckv.chunkkv_q8_resize(self.cache, self.cache.lens + counts, slots)
        if self.cache.state[2].item() != 0:
            raise RuntimeError("the cache has too few pages")
        ckv.chunkkv_q8_append(self.cache, 0, k, v, counts, slots)
        for r, n in enumerate(counts.tolist()):
            b, h = divmod(r, self.Hkv)
            self.k[r] = torch.cat([self.k[r], k[b, h, :n].float()])
            self.v[r] = torch.cat([self.v[r], v[b, h, :n].float()])

    def clear(self):
        ckv.chunkkv_q8_resize(self.cache, torch.zeros_like(self.cache.lens))
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
        ckv.chunkkv_q8_load(self.cache, 0, start, max(lens), k, v)
        return k, v, cu

    def attend(self, q):
        return ckv.q8_attention(self.cache, 0, q, workspace=self.ws)

    def error(self, q, out) -> float:
        """Relative error of an output against 64 bits over the rows before their rounding to 8 bits."""
        want = torch.zeros_like(out, dtype=torch.float64)
        for r in range(self.cache.rows):
            b, h = divmod(r, self.Hkv)
            qr = q[b, h * self.G:(h + 1) * self.G].double()
            p = torch.softmax(qr @ self.k[r].double().T / math.sqrt(self.d), -1)
            want[b, h * self.G:(h + 1) * self.G] = p @ self.v[r].double()
        return float((out.double() - want).norm() / want.norm())


def serve(seqlens=(700, 1500, 333), Hkv=2, G=4, d=128, w=16, c=10, budget=200, steps=40, again_at=24, seed=0) -> dict:
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
    layer = Layer(B, Hkv, G, d, budget + w + steps + c, dev)
    layer.append(kept.k_out[0], kept.v_out[0], kept.counts[0])
    lengths = [layer.cache.lens.tolist()]

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
    return {"hidden": hidden, "errors": errors, "lengths": lengths, "free_pages": int(layer.cache.state[1])}


if __name__ == "__main__":
    result = serve()
    print("tokens per cache row after the prompt, before and after the second compression, at the end:")
    for row in result["lengths"]:
        print("   ", row)
    print(f"relative error of the decoded tokens against 64 bits before rounding: largest {max(result['errors']):.4f}")
