"""Python binding of the serving operators: attention over packed prompts, the 8-bit and the 4-bit paged cache.

Like api.py, this module marshals arguments only: every step runs in the library's CUDA kernels, on the
current torch stream of the tensors' device.
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass, field

import torch

from ._lib import LIB, Q8_PAGE, PrefillParams, Q4CacheStruct, Q8CacheStruct, q4_page_bytes
from .api import _check, _DT


def _host_i32(xs):
    xs = [int(x) for x in xs]
    if xs and not -(1 << 31) <= min(xs) <= max(xs) < 1 << 31:
        raise ValueError("offsets beyond 32 bits")           # ctypes would drop their upper bits
    return (ctypes.c_int32 * len(xs))(*xs)


def _bytes(t):
    return t.numel() * t.element_size()


def _stream(t, *others) -> int:
    """The current stream of the tensors' device, as the integer that ctypes passes on.  They lie on one GPU, and it
    is the current one: the library asks the current device for its size and launches there."""
    return _stream_of(t.get_device(), *others)


def _stream_of(dev: int, *others) -> int:
    if dev < 0:
        raise ValueError("the tensors live in GPU memory")
    for o in others:
        if o.get_device() != dev:
            raise ValueError("the tensors of a call lie on one GPU")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"the tensors lie on cuda:{dev}, which is not the current device (torch.cuda.device makes it so)")
    return torch._C._cuda_getCurrentRawStream(dev)


# ------------------------------------------------------------------ prefill attention

def prefill_params_for(q, k, cu_q, cu_k=None, *, scale: float | None = None, o_strides=None):
    """chunkkv_prefill_params describing q [Tq_total, Hq, d] and k, v [Tk_total, Hkv, d] as laid out in memory
    (v like k).  cu_q and cu_k are host offsets (cu_k None: as cu_q); o_strides = (token, head) of the output
    in elements (default: contiguous).  Returns (params, keepalive): keepalive owns the host offset arrays.
    """
    if cu_k is None:
        cu_k = cu_q
    if len(cu_q) != len(cu_k) or len(cu_q) < 1:
        raise ValueError("cu_q and cu_k need B + 1 offsets each")
    if q.dim() != 3 or k.dim() != 3 or q.shape[2] != k.shape[2] or q.dtype != k.dtype or q.dtype not in _DT:
        raise ValueError("q [Tq, Hq, d] and k [Tk, Hkv, d] of one type, float32 or bfloat16")
    if q.stride(2) != 1 or k.stride(2) != 1:
        raise ValueError("the head dimension must be contiguous")
    if cu_q[-1] > q.shape[0] or cu_k[-1] > k.shape[0]:
        raise ValueError("offsets beyond the packed rows")
    Hq, d = q.shape[1], q.shape[2]
    cq, ck = _host_i32(cu_q), _host_i32(cu_k)
    p32 = ctypes.POINTER(ctypes.c_int32)
    if o_strides is None:
        o_strides = (Hq * d, d)
    p = PrefillParams(B=len(cu_q) - 1, Hq=Hq, Hkv=k.shape[1], d=d, dtype=_DT[q.dtype],
                      scale=1.0 / math.sqrt(d) if scale is None else scale,
                      cu_q=ctypes.cast(cq, p32), cu_k=ctypes.cast(ck, p32), q_stride_t=q.stride(0),
                      q_stride_h=q.stride(1), kv_stride_t=k.stride(0), kv_stride_h=k.stride(1),
                      o_stride_t=o_strides[0], o_stride_h=o_strides[1])
    return p, (cq, ck)


def chunkkv_prefill_workspace_size(p: PrefillParams) -> int:
    n = ctypes.c_size_t()
    _check("chunkkv_prefill_workspace_size", LIB.chunkkv_prefill_workspace_size(ctypes.byref(p), ctypes.byref(n)))
    return n.value


def chunkkv_prefill_path(p: PrefillParams) -> int:
    return int(LIB.chunkkv_prefill_path(ctypes.byref(p)))


def chunkkv_prefill_attention(p: PrefillParams, q, k, v, out, ws) -> None:
    _check("chunkkv_prefill_attention",
           LIB.chunkkv_prefill_attention(ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), ws.data_ptr(), _bytes(ws),
                                         _stream(q, k, v, out, ws)))


def prefill_attention(q, k, v, cu_q, cu_k=None, *, scale: float | None = None, out=None, workspace=None):
    """Causal attention over packed prompts on the current stream; allocates the output with torch unless given.
    Rows of q behind cu_q's last offset belong to no sequence: zeros in an output allocated here, else left alone."""
    if v.shape != k.shape or v.dtype != k.dtype or v.stride() != k.stride():
        raise ValueError("v must have k's shape, type and strides")
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if len(cu_q) > 0 and 0 <= cu_q[-1] < q.shape[0]:
            out[cu_q[-1]:].zero_()
    if out.shape != q.shape or out.dtype != q.dtype or out.stride(2) != 1:
        raise ValueError("out must have q's shape and type, its head dimension contiguous")
    p, keep = prefill_params_for(q, k, cu_q, cu_k, scale=scale, o_strides=(out.stride(0), out.stride(1)))
    if workspace is None:
        workspace = torch.zeros(chunkkv_prefill_workspace_size(p), dtype=torch.uint8, device=q.device)
    chunkkv_prefill_attention(p, q, k, v, out, workspace)
    del keep
    return out


# ------------------------------------------------------------------ 8-bit cache

@dataclass
class Q8Cache:
    """The 8-bit cache of the layers that share one set of lengths (layouts as in chunkkv.h)."""
    B: int
    Hkv: int
    d: int
    k_pages: list            # per layer [n_pages, d64 / 64, 64, 64] int8
    v_pages: list            # per layer [n_pages, d64, 64] int8
    scales: list             # per layer [n_pages, 2] fp32
    table: torch.Tensor      # [B * Hkv, max_pages] int32
    lens: torch.Tensor       # [B * Hkv] int32
    ring: torch.Tensor       # [n_pages] int32
    state: torch.Tensor      # [4] int32: head, free pages, status of the last resize, 0
    rows: int = field(init=False, repr=False)
    _c: list = field(default_factory=list, repr=False)
    _refs: list = field(init=False, repr=False)     # _c by reference, the tensors' device and the usual scale: made
    _dev: int = field(init=False, repr=False)       # once, since a call's host time counts
    _scale: float = field(init=False, repr=False)

    def __post_init__(self):
        self.rows = self.B * self.Hkv
        rows, n_pages, d64 = self.rows, self.ring.numel(), -(-self.d // 64) * 64
        ints = (self.table, self.lens, self.ring, self.state)
        if any(t.dtype != torch.int32 or not t.is_contiguous() for t in ints):
            raise ValueError("table, lens, ring and state are contiguous int32")
        if self.table.dim() != 2 or self.table.shape[0] != rows or self.lens.numel() != rows or self.state.numel() != 4:
            raise ValueError("table [B * Hkv, max_pages], lens [B * Hkv], state [4]")
        if not len(self.k_pages) == len(self.v_pages) == len(self.scales):
            raise ValueError("k_pages, v_pages and scales of every layer")
        if len({t.device for t in (*ints, *self.k_pages, *self.v_pages, *self.scales)}) != 1:
            raise ValueError("the tensors of a cache lie on one device")
        for k, v, s in zip(self.k_pages, self.v_pages, self.scales):
            if (k.shape != (n_pages, d64 // 64, Q8_PAGE, 64) or v.shape != (n_pages, d64, Q8_PAGE)
                    or s.shape != (n_pages, 2) or k.dtype != torch.int8 or v.dtype != torch.int8
                    or s.dtype != torch.float32 or not (k.is_contiguous() and v.is_contiguous() and s.is_contiguous())):
                raise ValueError("k_pages [n_pages, d64 / 64, 64, 64], v_pages [n_pages, d64, 64] int8, "
                                 "scales [n_pages, 2] float32, contiguous")
        for i in range(max(1, len(self.k_pages))):
            pages = [x[i].data_ptr() if x else None for x in (self.k_pages, self.v_pages, self.scales)]
            self._c.append(Q8CacheStruct(self.B, self.Hkv, self.d, n_pages, self.table.shape[1], *pages,
                                         *[t.data_ptr() for t in ints]))
        self._refs = [ctypes.byref(c) for c in self._c]
        self._dev, self._scale = self.lens.get_device(), 1.0 / math.sqrt(self.d)

    @property
    def device(self):
        return self.lens.device

    def layer(self, i: int):
        """The chunkkv_q8_cache of layer i, by reference (the tensors' addresses as they were at construction)."""
        return self._refs[i]


def q8_cache(B: int, Hkv: int, d: int, *, n_pages: int, max_pages: int, n_layers: int = 1, device="cuda") -> Q8Cache:
    """An empty cache: pools for n_pages pages a layer, rows of up to max_pages pages, every page free."""
    d64 = -(-d // 64) * 64
    dev = torch.device(device)

    def zeros(*shape, dtype):
        return torch.zeros(*shape, dtype=dtype, device=dev)
    return Q8Cache(B=B, Hkv=Hkv, d=d,
                   k_pages=[zeros(n_pages, d64 // 64, Q8_PAGE, 64, dtype=torch.int8) for _ in range(n_layers)],
                   v_pages=[zeros(n_pages, d64, Q8_PAGE, dtype=torch.int8) for _ in range(n_layers)],
                   scales=[zeros(n_pages, 2, dtype=torch.float32) for _ in range(n_layers)],
                   table=torch.full((B * Hkv, max_pages), -1, dtype=torch.int32, device=dev),
                   lens=zeros(B * Hkv, dtype=torch.int32),
                   ring=torch.arange(n_pages, dtype=torch.int32, device=dev),
                   state=torch.tensor([0, n_pages, 0, 0], dtype=torch.int32, device=dev))


def _rows_i32(cache: Q8Cache, t, what: str):
    if t.dtype != torch.int32 or t.numel() != cache.rows or not t.is_contiguous():
        raise ValueError(f"{what}: one contiguous int32 per (sequence, KV head)")


def chunkkv_q8_resize(cache: Q8Cache, new_lens, slots=None) -> None:
    """Sets every row's length (device int32, one per row); slots: None or int64 [rows, n_cap] for the slot map."""
    _rows_i32(cache, new_lens, "new_lens")
    if slots is None:
        at, n_cap, stream = None, 0, _stream_of(cache._dev, new_lens)
    else:
        shape = slots.shape
        if slots.dtype != torch.int64 or len(shape) != 2 or shape[0] != cache.rows or not slots.is_contiguous():
            raise ValueError("slots: contiguous int64 [B * Hkv, n_cap]")
        at, n_cap, stream = slots.data_ptr(), shape[1], _stream_of(cache._dev, new_lens, slots)
    code = LIB.chunkkv_q8_resize(cache._refs[0], new_lens.data_ptr(), at, n_cap, stream)
    if code:
        _check("chunkkv_q8_resize", code)


def chunkkv_q8_append(cache: Q8Cache, layer: int, k, v, counts, slots) -> None:
    """Writes the first counts[b][h] of k, v [B, Hkv, n_cap, d] (any strides, d contiguous) to their slots."""
    shape, st, dt = k.shape, k.stride(), _DT.get(k.dtype)
    if dt is None or v.shape != shape or v.stride() != st or v.dtype != k.dtype:
        raise ValueError("k and v of one shape, type (float32 or bfloat16) and strides")
    n_cap = shape[2] if len(shape) == 4 else -1
    if shape != (cache.B, cache.Hkv, n_cap, cache.d) or st[3] != 1:
        raise ValueError("k, v [B, Hkv, n_cap, d], the head dimension contiguous")
    _rows_i32(cache, counts, "counts")
    if slots.dtype != torch.int64 or slots.shape != (cache.rows, n_cap) or not slots.is_contiguous():
        raise ValueError("slots: contiguous int64 [B * Hkv, n_cap]")
    code = LIB.chunkkv_q8_append(cache._refs[layer], dt, k.data_ptr(), v.data_ptr(), st[0], st[1], st[2],
                                 counts.data_ptr(), slots.data_ptr(), n_cap,
                                 _stream_of(cache._dev, k, v, counts, slots))
    if code:
        _check("chunkkv_q8_append", code)


def chunkkv_q8_load(cache: Q8Cache, layer: int, start, n_cap: int, k_out, v_out) -> None:
    """Reads rows back into k_out, v_out [tokens, d]: token i of row r to start[r] + i (int64), i < min(lens, n_cap).
    Tokens past the end of k_out are not written."""
    if start.dtype != torch.int64 or start.numel() != cache.rows or not start.is_contiguous():
        raise ValueError("start: one contiguous int64 per (sequence, KV head)")
    shape, st, dt = k_out.shape, k_out.stride(), _DT.get(k_out.dtype)
    if (dt is None or v_out.shape != shape or v_out.stride() != st or v_out.dtype != k_out.dtype
            or len(shape) != 2 or shape[1] != cache.d or st[1] != 1):
        raise ValueError("k_out, v_out [tokens, d] of one type and layout, the head dimension contiguous")
    code = LIB.chunkkv_q8_load_bounded(cache._refs[layer], dt, start.data_ptr(), n_cap, shape[0], k_out.data_ptr(),
                                       v_out.data_ptr(), st[0], _stream_of(cache._dev, start, k_out, v_out))
    if code:
        _check("chunkkv_q8_load", code)


def chunkkv_q8_workspace_size(cache: Q8Cache, G: int) -> int:
    n = ctypes.c_size_t()
    _check("chunkkv_q8_workspace_size", LIB.chunkkv_q8_workspace_size(cache.layer(0), G, ctypes.byref(n)))
    return n.value


def chunkkv_q8_attention(cache: Q8Cache, layer: int, q, out, ws, scale: float | None = None) -> None:
    """out [B, Hkv * G, d] = attention of q over the rows of one layer's cache."""
    shape, qs, os_, dt = q.shape, q.stride(), out.stride(), _DT.get(q.dtype)
    if dt is None or len(shape) != 3 or out.shape != shape or out.dtype != q.dtype:
        raise ValueError("q and out [B, Hq, d] of one type, float32 or bfloat16")
    if shape[0] != cache.B or shape[2] != cache.d or shape[1] % cache.Hkv or qs[2] != 1 or os_[2] != 1:
        raise ValueError("q and out [B, Hkv * G, d], the head dimension contiguous")
    code = LIB.chunkkv_q8_attention(cache._refs[layer], dt, shape[1] // cache.Hkv, cache._scale if scale is None else scale,
                                    q.data_ptr(), qs[0], qs[1], out.data_ptr(), os_[0], os_[1], ws.data_ptr(), ws.nbytes,
                                    _stream_of(cache._dev, q, out, ws))
    if code:
        _check("chunkkv_q8_attention", code)


def q8_attention(cache: Q8Cache, layer: int, q, *, scale: float | None = None, out=None, workspace=None):
    """Single-token attention over one layer's cache; allocates the output with torch unless given."""
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if workspace is None:
        workspace = torch.zeros(chunkkv_q8_workspace_size(cache, q.shape[1] // cache.Hkv), dtype=torch.uint8,
                                device=q.device)
    chunkkv_q8_attention(cache, layer, q, out, workspace, scale)
    return out


# ------------------------------------------------------------------ 4-bit cache

@dataclass
class Q4Cache:
    """The 4-bit cache of the layers that share one set of lengths (layouts as in chunkkv.h)."""
    B: int
    Hkv: int
    d: int
    pages: list              # per layer [n_pages, q4_page_bytes(d)] uint8
    table: torch.Tensor      # [B * Hkv, max_pages] int32
    lens: torch.Tensor       # [B * Hkv] int32
    ring: torch.Tensor       # [n_pages] int32
    state: torch.Tensor      # [4] int32: head, free pages, status of the last resize, 0
    rows: int = field(init=False, repr=False)
    _c: list = field(default_factory=list, repr=False)
    _refs: list = field(init=False, repr=False)     # as in Q8Cache
    _dev: int = field(init=False, repr=False)
    _scale: float = field(init=False, repr=False)

    def __post_init__(self):
        self.rows = self.B * self.Hkv
        n_pages = self.ring.numel()
        ints = (self.table, self.lens, self.ring, self.state)
        if any(t.dtype != torch.int32 or not t.is_contiguous() for t in ints):
            raise ValueError("table, lens, ring and state are contiguous int32")
        if self.table.dim() != 2 or self.table.shape[0] != self.rows or self.lens.numel() != self.rows or self.state.numel() != 4:
            raise ValueError("table [B * Hkv, max_pages], lens [B * Hkv], state [4]")
        if len({t.device for t in (*ints, *self.pages)}) != 1:
            raise ValueError("the tensors of a cache lie on one device")
        for p in self.pages:
            if p.shape != (n_pages, q4_page_bytes(self.d)) or p.dtype != torch.uint8 or not p.is_contiguous():
                raise ValueError("pages [n_pages, q4_page_bytes(d)] uint8, contiguous")
        for i in range(max(1, len(self.pages))):
            self._c.append(Q4CacheStruct(self.B, self.Hkv, self.d, n_pages, self.table.shape[1],
                                         self.pages[i].data_ptr() if self.pages else None, *[t.data_ptr() for t in ints]))
        self._refs = [ctypes.byref(c) for c in self._c]
        self._dev, self._scale = self.lens.get_device(), 1.0 / math.sqrt(self.d)

    @property
    def device(self):
        return self.lens.device

    def layer(self, i: int):
        """The chunkkv_q4_cache of layer i, by reference (the tensors' addresses as they were at construction)."""
        return self._refs[i]


def q4_cache(B: int, Hkv: int, d: int, *, n_pages: int, max_pages: int, n_layers: int = 1, device="cuda") -> Q4Cache:
    """An empty cache: pools for n_pages pages a layer, rows of up to max_pages pages, every page free."""
    dev = torch.device(device)
    return Q4Cache(B=B, Hkv=Hkv, d=d,
                   pages=[torch.zeros(n_pages, q4_page_bytes(d), dtype=torch.uint8, device=dev) for _ in range(n_layers)],
                   table=torch.full((B * Hkv, max_pages), -1, dtype=torch.int32, device=dev),
                   lens=torch.zeros(B * Hkv, dtype=torch.int32, device=dev),
                   ring=torch.arange(n_pages, dtype=torch.int32, device=dev),
                   state=torch.tensor([0, n_pages, 0, 0], dtype=torch.int32, device=dev))


def chunkkv_q4_resize(cache: Q4Cache, new_lens, slots=None) -> None:
    """Sets every row's length (device int32, one per row); slots: None or int64 [rows, n_cap] for the slot map."""
    _rows_i32(cache, new_lens, "new_lens")
    if slots is None:
        at, n_cap, stream = None, 0, _stream_of(cache._dev, new_lens)
    else:
        shape = slots.shape
        if slots.dtype != torch.int64 or len(shape) != 2 or shape[0] != cache.rows or not slots.is_contiguous():
            raise ValueError("slots: contiguous int64 [B * Hkv, n_cap]")
        at, n_cap, stream = slots.data_ptr(), shape[1], _stream_of(cache._dev, new_lens, slots)
    code = LIB.chunkkv_q4_resize(cache._refs[0], new_lens.data_ptr(), at, n_cap, stream)
    if code:
        _check("chunkkv_q4_resize", code)


def chunkkv_q4_append(cache: Q4Cache, layer: int, k, v, counts, slots) -> None:
    """Writes the first counts[b][h] of k, v [B, Hkv, n_cap, d] (any strides, d contiguous) to their slots."""
    shape, st, dt = k.shape, k.stride(), _DT.get(k.dtype)
    if dt is None or v.shape != shape or v.stride() != st or v.dtype != k.dtype:
        raise ValueError("k and v of one shape, type (float32 or bfloat16) and strides")
    n_cap = shape[2] if len(shape) == 4 else -1
    if shape != (cache.B, cache.Hkv, n_cap, cache.d) or st[3] != 1:
        raise ValueError("k, v [B, Hkv, n_cap, d], the head dimension contiguous")
    _rows_i32(cache, counts, "counts")
    if slots.dtype != torch.int64 or slots.shape != (cache.rows, n_cap) or not slots.is_contiguous():
        raise ValueError("slots: contiguous int64 [B * Hkv, n_cap]")
    code = LIB.chunkkv_q4_append(cache._refs[layer], dt, k.data_ptr(), v.data_ptr(), st[0], st[1], st[2],
                                 counts.data_ptr(), slots.data_ptr(), n_cap,
                                 _stream_of(cache._dev, k, v, counts, slots))
    if code:
        _check("chunkkv_q4_append", code)


def chunkkv_q4_load(cache: Q4Cache, layer: int, start, n_cap: int, k_out, v_out) -> None:
    """Reads rows back into k_out, v_out [tokens, d]: token i of row r to start[r] + i (int64), i < min(lens, n_cap).
    Tokens past the end of k_out are not written."""
    if start.dtype != torch.int64 or start.numel() != cache.rows or not start.is_contiguous():
        raise ValueError("start: one contiguous int64 per (sequence, KV head)")
    shape, st, dt = k_out.shape, k_out.stride(), _DT.get(k_out.dtype)
    if (dt is None or v_out.shape != shape or v_out.stride() != st or v_out.dtype != k_out.dtype
            or len(shape) != 2 or shape[1] != cache.d or st[1] != 1):
        raise ValueError("k_out, v_out [tokens, d] of one type and layout, the head dimension contiguous")
    code = LIB.chunkkv_q4_load(cache._refs[layer], dt, start.data_ptr(), n_cap, shape[0], k_out.data_ptr(),
                               v_out.data_ptr(), st[0], _stream_of(cache._dev, start, k_out, v_out))
    if code:
        _check("chunkkv_q4_load", code)


def chunkkv_q4_workspace_size(cache: Q4Cache, G: int, n_q: int = 1, dtype=torch.bfloat16) -> int:
    """Bytes of workspace for queries of n_q tokens a sequence, G heads a KV head, of this type."""
    n = ctypes.c_size_t()
    if dtype not in _DT:
        raise ValueError("float32 or bfloat16")
    _check("chunkkv_q4_workspace_size", LIB.chunkkv_q4_workspace_size(cache.layer(0), _DT[dtype], G, n_q, ctypes.byref(n)))
    return n.value


def chunkkv_q4_path(cache: Q4Cache, G: int, n_q: int = 1, dtype=torch.bfloat16) -> int:
    """0 or 1: the kernel for few or for many query rows (-1: invalid), for contiguous q and out.  Repeated axes (strides
    of 0) and strides of out of 2^22 elements and more take the one for few whatever this says."""
    return int(LIB.chunkkv_q4_path(cache.layer(0), _DT.get(dtype, -1), G, n_q))


def chunkkv_q4_attention(cache: Q4Cache, layer: int, q, out, ws, scale: float | None = None, q_lens=None) -> None:
    """out = attention of q over the rows of one layer's cache: [B, Hkv * G, d] for one query token a sequence, or
    [B, n_q, Hkv * G, d] for several, the last of each row's tokens being their own.  q_lens: how many of the n_q are
    real, device int32 [B] (None: all); the rest of out is left alone."""
    shape, qs, os_, dt = q.shape, q.stride(), out.stride(), _DT.get(q.dtype)
    if dt is None or out.shape != shape or out.dtype != q.dtype:
        raise ValueError("q and out of one shape and type, float32 or bfloat16")
    if len(shape) == 3:
        n_q, q_st, o_st = 1, 0, 0
    elif len(shape) == 4:
        n_q, q_st, o_st = shape[1], qs[1], os_[1]
    else:
        raise ValueError("q and out [B, Hq, d] or [B, n_q, Hq, d]")
    Hq = shape[-2]
    if shape[0] != cache.B or shape[-1] != cache.d or Hq % cache.Hkv or qs[-1] != 1 or os_[-1] != 1:
        raise ValueError("q and out [B, Hkv * G, d] or [B, n_q, Hkv * G, d], the head dimension contiguous")
    if q_lens is None:
        at, stream = None, _stream_of(cache._dev, q, out, ws)
    else:
        if q_lens.dtype != torch.int32 or q_lens.numel() != cache.B or not q_lens.is_contiguous():
            raise ValueError("q_lens: one contiguous int32 per sequence")
        at, stream = q_lens.data_ptr(), _stream_of(cache._dev, q, out, ws, q_lens)
    code = LIB.chunkkv_q4_attention(cache._refs[layer], dt, Hq // cache.Hkv, n_q, at, cache._scale if scale is None else scale,
                                    q.data_ptr(), qs[0], q_st, qs[-2], out.data_ptr(), os_[0], o_st, os_[-2],
                                    ws.data_ptr(), ws.nbytes, stream)
    if code:
        _check("chunkkv_q4_attention", code)


def q4_attention(cache: Q4Cache, layer: int, q, *, q_lens=None, scale: float | None = None, out=None, workspace=None):
    """Attention of one or several query tokens a sequence over one layer's cache; allocates the output with torch
    unless given (zeros at the query tokens that q_lens leaves out)."""
    if out is None:
        out = (torch.empty if q_lens is None else torch.zeros)(q.shape, dtype=q.dtype, device=q.device)
    if workspace is None:
        n_q = q.shape[1] if q.dim() == 4 else 1
        workspace = torch.zeros(chunkkv_q4_workspace_size(cache, max(1, q.shape[-2] // cache.Hkv), n_q, q.dtype),
                                dtype=torch.uint8, device=q.device)
    chunkkv_q4_attention(cache, layer, q, out, workspace, scale, q_lens)
    return out


__all__ = [
    "PrefillParams", "Q4Cache", "Q8Cache", "Q8_PAGE", "chunkkv_prefill_attention", "chunkkv_prefill_path",
    "chunkkv_prefill_workspace_size", "chunkkv_q4_append", "chunkkv_q4_attention", "chunkkv_q4_load", "chunkkv_q4_path",
    "chunkkv_q4_resize", "chunkkv_q4_workspace_size", "chunkkv_q8_append", "chunkkv_q8_attention", "chunkkv_q8_load",
    "chunkkv_q8_resize", "chunkkv_q8_workspace_size", "prefill_attention", "prefill_params_for", "q4_attention",
    "q4_cache", "q4_page_bytes", "q8_attention", "q8_cache",
]
