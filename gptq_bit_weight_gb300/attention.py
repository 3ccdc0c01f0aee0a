"""Rotary positions, a paged cache, and attention over it.

The classes marshal torch CUDA tensors to ``gptq_q4_attn_*`` (see
include/gptq_q4.h): ``PagedCache`` is one layer's keys and values,
``PagedCache4`` the same held in 4 bits, ``PagedBatch`` the requests of one
step (made once and used for every layer), ``PagedAttention`` the operators.
"""
from __future__ import annotations

import ctypes

import torch

from . import (GPTQ_Q4_ROPE_BANDS, GPTQ_Q4_ROPE_LINEAR, GPTQ_Q4_ROPE_NTK, GPTQ_Q4_ROPE_PLAIN, GPTQ_Q4_ROPE_YARN,
               _check, _lib, _release, gptq_q4_attn_device_error, gptq_q4_attn_free, gptq_q4_attn_make,
               gptq_q4_attn_set_rope, gptq_q4_batch, gptq_q4_cache, gptq_q4_cache4, gptq_q4_rope_freqs)
from .adapters import _code, _refuse, _rows, _stream

_append, _attend, _read = _lib.gptq_q4_attn_append, _lib.gptq_q4_attn_attend, _lib.gptq_q4_attn_read
_append4, _attend4, _read4 = _lib.gptq_q4_attn_append4, _lib.gptq_q4_attn_attend4, _lib.gptq_q4_attn_read4
_attend_sinks = _lib.gptq_q4_attn_attend_sinks

_KINDS = {"none": GPTQ_Q4_ROPE_PLAIN, "linear": GPTQ_Q4_ROPE_LINEAR, "ntk": GPTQ_Q4_ROPE_NTK,
          "bands": GPTQ_Q4_ROPE_BANDS, "yarn": GPTQ_Q4_ROPE_YARN}


class PagedCache:
    """k and v: [pages, kv_heads, page_size, head_dim], dense within a page."""

    def __init__(self, k, v):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.device != v.device or not k.is_cuda:
            _refuse("k and v must be CUDA tensors [pages, kv_heads, page_size, head_dim] of one shape and type")
        pages, heads, page, width = k.shape
        strides = []
        for t in (k, v):                     # a dimension of one has no stride of its own
            s = t.stride()
            if s[3] != 1 or s[2] != width or (heads > 1 and s[1] != page * width):
                _refuse("k and v must be dense within a page")
            strides.append(s[0] if pages > 1 else heads * page * width)
        if strides[0] != strides[1]:
            _refuse("k and v must have one stride from page to page")
        self.k, self.v = k, v
        self.kind = (k.dtype, k.device, *k.shape[1:])
        self.struct = gptq_q4_cache(k.data_ptr(), v.data_ptr(), pages, strides[0])
        self.ref = ctypes.byref(self.struct)


class PagedCache4:
    """A layer's keys and values in 4 bits: kv uint8 [pages, kv_heads, page_size,
    record], dense within a page, record = head_dim + 8 head_dim / group bytes
    (the layout stands at gptq_q4_cache4), for groups of 32 or 64 elements and
    a float16 or bfloat16 handle."""

    def __init__(self, kv, head_dim: int, group: int = 32, dtype=torch.float16):
        _code(dtype)
        if group not in (32, 64) or head_dim % group:
            _refuse(f"group {group} must be 32 or 64 and divide head_dim {head_dim}")
        record = self.record(head_dim, group)
        if kv.dim() != 4 or kv.dtype != torch.uint8 or not kv.is_cuda or kv.shape[3] != record:
            _refuse(f"kv must be a uint8 CUDA tensor [pages, kv_heads, page_size, {record}]")
        pages, heads, page, _ = kv.shape
        s = kv.stride()                      # a dimension of one has no stride of its own
        if s[3] != 1 or (page > 1 and s[2] != record) or (heads > 1 and s[1] != page * record):
            _refuse("kv must be dense within a page")
        self.kv, self.head_dim, self.group = kv, head_dim, group
        self.kind = (dtype, kv.device, heads, page, head_dim)
        self.struct = gptq_q4_cache4(kv.data_ptr(), pages, s[0] if pages > 1 else heads * page * record, group)
        self.ref = ctypes.byref(self.struct)

    @staticmethod
    def record(head_dim: int, group: int = 32) -> int:
        """Bytes of one token's keys and values of one head."""
        return head_dim + 8 * head_dim // group

    @classmethod
    def empty(cls, pages: int, kv_heads: int, page_size: int, head_dim: int, group: int = 32, dtype=torch.float16,
              device="cuda"):
        """A cache in new, uninitialised memory."""
        kv = torch.empty((pages, kv_heads, page_size, cls.record(head_dim, group)), dtype=torch.uint8, device=device)
        return cls(kv, head_dim, group, dtype)


class PagedBatch:
    """The requests of one step: cu_q int32 [batch + 1], kv_len int32 [batch]
    (the new tokens among them) and table int32 [batch, width], on the GPU;
    tokens: the step's rows; max_q: at least the most new tokens of a request
    (default: tokens)."""

    def __init__(self, cu_q, kv_len, table, tokens: int, max_q: int | None = None):
        for t, what in ((cu_q, "cu_q"), (kv_len, "kv_len"), (table, "table")):
            if t.dtype != torch.int32 or not t.is_cuda or t.device != cu_q.device or \
                    (t.dim() and t.numel() and t.shape[-1] > 1 and t.stride(-1) != 1):
                _refuse(f"{what} must be int32 on the GPU, dense in its last dimension")
        batch = kv_len.numel()
        if cu_q.dim() != 1 or kv_len.dim() != 1 or cu_q.numel() != batch + 1 or table.dim() != 2 or \
                table.shape[0] != batch:
            _refuse(f"cu_q {tuple(cu_q.shape)}, kv_len {tuple(kv_len.shape)} and table {tuple(table.shape)} "
                    "must be [batch + 1], [batch] and [batch, width]")
        self.tensors = (cu_q, kv_len, table)
        self.tokens, self.device = tokens, cu_q.device
        stride = table.stride(0) if batch > 1 else max(table.stride(0), table.shape[1])
        self.struct = gptq_q4_batch(cu_q.data_ptr(), kv_len.data_ptr(), table.data_ptr(), stride, table.shape[1],
                                    batch, tokens, tokens if max_q is None else max_q)
        self.ref = ctypes.byref(self.struct)


class PagedAttention:
    """Rotary positions, append and attention for q_heads query heads over
    kv_heads key/value heads; float16 or bfloat16."""

    def __init__(self, q_heads: int, kv_heads: int, head_dim: int, page_size: int, dtype=torch.float16):
        self.handle = None
        self.q_heads, self.kv_heads, self.head_dim, self.page_size = q_heads, kv_heads, head_dim, page_size
        self.dtype = dtype
        self.device = torch.device("cuda", torch.cuda.current_device())
        _release()
        self.handle = gptq_q4_attn_make(q_heads, kv_heads, head_dim, page_size, _code(dtype))
        self._q_width = q_heads * head_dim
        self._kind = (dtype, self.device, kv_heads, page_size, head_dim)
        self._scale = head_dim ** -0.5

    def set_rope(self, rotary_dim: int, max_pos: int, base: float = 10000.0, interleaved: bool = False,
                 scaling: str = "none", factor: float = 1.0, low: float = 1.0, high: float = 4.0, original: int = 1,
                 length_scale: float | None = None) -> None:
        """Rotary positions for `append`: scaling "none", "linear", "ntk",
        "bands" or "yarn" (the formulas stand at gptq_q4_rope_freqs; for
        "yarn" low and high are the numbers of turns, 1 and 32 as a rule).
        rotary_dim 0 turns rotation off."""
        if scaling not in _KINDS:
            _refuse(f"scaling {scaling!r} is none of {sorted(_KINDS)}")
        if rotary_dim == 0:
            gptq_q4_attn_set_rope(self.handle, 0, 0, None, 1.0, 0)
            return
        freqs, scale = gptq_q4_rope_freqs(rotary_dim, base, _KINDS[scaling], factor, low, high, original)
        gptq_q4_attn_set_rope(self.handle, rotary_dim, int(interleaved), freqs,
                              scale if length_scale is None else length_scale, max_pos)

    def _check(self, cache, batch: PagedBatch) -> None:
        if cache.kind != self._kind:
            dtype, device, *shape = cache.kind
            _refuse(f"the cache is {dtype} {['pages', *shape]} on {device}: {self.dtype} ['pages', {self.kv_heads}, "
                    f"{self.page_size}, {self.head_dim}] on {self.device} is wanted")
        if batch.device != self.device:
            _refuse(f"the batch is on {batch.device}, the handle on {self.device}")

    def append(self, qkv, cache, batch: PagedBatch, positions=None, q_out=None):
        """Rotate queries and keys and put keys and values into the cache, a
        PagedCache or PagedCache4 (which quantises them); qkv
        [tokens, (q_heads + 2 kv_heads) head_dim].  Returns the rotated
        queries [tokens, q_heads, head_dim]."""
        self._check(cache, batch)
        x, rows, xs = _rows(qkv, "qkv", (self.q_heads + 2 * self.kv_heads) * self.head_dim, self.dtype, self.device)
        if q_out is None:
            q_out = torch.empty((rows, self.q_heads, self.head_dim), dtype=self.dtype, device=self.device)
            q, q_rows, qs = q_out, rows, self._q_width
        else:
            q, q_rows, qs = self._token_rows(q_out, "q_out", self.q_heads, written=True)
        if rows != batch.tokens or q_rows != batch.tokens:
            _refuse(f"qkv has {rows} rows and q_out {q_rows}, the batch {batch.tokens} tokens")
        if positions is not None and (positions.dtype != torch.int32 or positions.device != self.device or
                                      positions.numel() != batch.tokens or not positions.is_contiguous()):
            _refuse(f"positions must be contiguous int32 [{batch.tokens}] on {self.device}")
        call = _append4 if type(cache.struct) is gptq_q4_cache4 else _append
        _check(call(self.handle, x.data_ptr(), xs, cache.ref, batch.ref,
                    None if positions is None else positions.data_ptr(), q.data_ptr(), qs,
                    _stream(self.device.index)))
        return q_out

    def read(self, cache, batch: PagedBatch, k_out=None, v_out=None):
        """What the cache holds for the batch's new tokens, as (keys, values)
        [tokens, kv_heads, head_dim] of the handle's type; of a PagedCache4 the
        values that its codes stand for."""
        self._check(cache, batch)
        if k_out is None and v_out is None:
            k_out = torch.empty((batch.tokens, self.kv_heads, self.head_dim), dtype=self.dtype, device=self.device)
            outs = k_out, torch.empty_like(k_out)
            width = self.kv_heads * self.head_dim
            args = k_out.data_ptr(), width, outs[1].data_ptr(), width
        else:
            outs, args = [], []
            for t, what in ((k_out, "k_out"), (v_out, "v_out")):
                if t is None:
                    t = torch.empty((batch.tokens, self.kv_heads, self.head_dim), dtype=self.dtype, device=self.device)
                o, rows, stride = self._token_rows(t, what, self.kv_heads, written=True)
                if rows != batch.tokens:
                    _refuse(f"{what} has {rows} rows, the batch {batch.tokens} tokens")
                outs.append(t)
                args += [o.data_ptr(), stride]
            outs = tuple(outs)
        call = _read4 if type(cache.struct) is gptq_q4_cache4 else _read
        _check(call(self.handle, cache.ref, batch.ref, *args, _stream(self.device.index)))
        return outs

    def attend(self, q, cache, batch: PagedBatch, scale: float | None = None, window: int = 0, out=None, sinks: int = 0):
        """Attention of the new tokens' queries q [tokens, q_heads, head_dim]
        over the cache, a PagedCache or PagedCache4; scale defaults to
        head_dim ** -0.5, window 0 is none; with a window, the first `sinks`
        tokens of each context stay visible, at their positions in the text."""
        self._check(cache, batch)
        x, rows, xs = self._token_rows(q, "q", self.q_heads)
        if out is None:
            out = torch.empty((rows, self.q_heads, self.head_dim), dtype=self.dtype, device=self.device)
            o, o_rows, os_ = out, rows, self._q_width
        else:
            o, o_rows, os_ = self._token_rows(out, "out", self.q_heads, written=True)
        if rows != batch.tokens or o_rows != batch.tokens:
            _refuse(f"q has {rows} rows and out {o_rows}, the batch {batch.tokens} tokens")
        args = [self.handle, x.data_ptr(), xs, cache.ref, batch.ref, self._scale if scale is None else scale, window]
        tail = [o.data_ptr(), os_, _stream(self.device.index)]
        if type(cache.struct) is gptq_q4_cache4:
            _check(_attend4(*args, sinks, *tail))
        elif sinks:
            _check(_attend_sinks(*args, sinks, *tail))
        else:
            _check(_attend(*args, *tail))
        return out

    def _token_rows(self, t, what: str, want: int, written: bool = False):
        """[tokens, want heads, head_dim] (a view of wider rows allowed) or [tokens, want * head_dim]."""
        if t.dim() != 3:
            return _rows(t, what, want * self.head_dim, self.dtype, self.device, written)
        rows, heads, width = t.shape
        stride, s1, s2 = t.stride()
        if heads != want or width != self.head_dim or (s1 != width and heads > 1) or s2 != 1:
            _refuse(f"{what} {tuple(t.shape)} must be [tokens, {want}, {self.head_dim}], dense in a token")
        if t.dtype != self.dtype or t.device != self.device:
            _refuse(f"{what} is {t.dtype} on {t.device}: {self.dtype} on {self.device} is wanted")
        return t, rows, stride if rows > 1 else want * self.head_dim

    def device_error(self) -> None:
        gptq_q4_attn_device_error(self.handle)

    def close(self) -> None:
        if getattr(self, "handle", None):
            handle, self.handle = self.handle, None
            _release(gptq_q4_attn_free, handle)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
