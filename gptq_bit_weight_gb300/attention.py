"""Rotary positions, a paged cache, and attention over it.

The classes marshal torch CUDA tensors to ``gptq_q4_attn_*`` (see
include/gptq_q4.h): ``PagedCache`` is one layer's keys and values,
``PagedBatch`` the requests of one step (made once and used for every layer),
``PagedAttention`` the operators.
"""
from __future__ import annotations

import ctypes

import torch

from . import (GPTQ_Q4_ROPE_BANDS, GPTQ_Q4_ROPE_LINEAR, GPTQ_Q4_ROPE_NTK, GPTQ_Q4_ROPE_PLAIN, GPTQ_Q4_ROPE_YARN,
               _check, _lib, gptq_q4_attn_device_error, gptq_q4_attn_free, gptq_q4_attn_make, gptq_q4_attn_set_rope,
               gptq_q4_batch, gptq_q4_cache, gptq_q4_rope_freqs)
from .adapters import _code, _refuse, _rows, _stream

_append, _attend = _lib.gptq_q4_attn_append, _lib.gptq_q4_attn_attend

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

    def _check(self, cache: PagedCache, batch: PagedBatch) -> None:
        if cache.kind != self._kind:
            dtype, device, *shape = cache.kind
            _refuse(f"the cache is {dtype} {['pages', *shape]} on {device}: {self.dtype} ['pages', {self.kv_heads}, "
                    f"{self.page_size}, {self.head_dim}] on {self.device} is wanted")
        if batch.device != self.device:
            _refuse(f"the batch is on {batch.device}, the handle on {self.device}")

    def append(self, qkv, cache: PagedCache, batch: PagedBatch, positions=None, q_out=None):
        """Rotate queries and keys and put keys and values into the cache; qkv
        [tokens, (q_heads + 2 kv_heads) head_dim].  Returns the rotated
        queries [tokens, q_heads, head_dim]."""
        self._check(cache, batch)
        x, rows, xs = _rows(qkv, "qkv", (self.q_heads + 2 * self.kv_heads) * self.head_dim, self.dtype, self.device)
        if q_out is None:
            q_out = torch.empty((rows, self.q_heads, self.head_dim), dtype=self.dtype, device=self.device)
            q, q_rows, qs = q_out, rows, self._q_width
        else:
            q, q_rows, qs = self._token_rows(q_out, "q_out", written=True)
        if rows != batch.tokens or q_rows != batch.tokens:
            _refuse(f"qkv has {rows} rows and q_out {q_rows}, the batch {batch.tokens} tokens")
        if positions is not None and (positions.dtype != torch.int32 or positions.device != self.device or
                                      positions.numel() != batch.tokens or not positions.is_contiguous()):
            _refuse(f"positions must be contiguous int32 [{batch.tokens}] on {self.device}")
        _check(_append(self.handle, x.data_ptr(), xs, cache.ref, batch.ref,
                       None if positions is None else positions.data_ptr(), q.data_ptr(), qs,
                       _stream(self.device.index)))
        return q_out

    def attend(self, q, cache: PagedCache, batch: PagedBatch, scale: float | None = None, window: int = 0, out=None):
        """Attention of the new tokens' queries q [tokens, q_heads, head_dim]
        over the cache; scale defaults to head_dim ** -0.5, window 0 is none."""
        self._check(cache, batch)
        x, rows, xs = self._token_rows(q, "q")
        if out is None:
            out = torch.empty((rows, self.q_heads, self.head_dim), dtype=self.dtype, device=self.device)
            o, o_rows, os_ = out, rows, self._q_width
        else:
            o, o_rows, os_ = self._token_rows(out, "out", written=True)
        if rows != batch.tokens or o_rows != batch.tokens:
            _refuse(f"q has {rows} rows and out {o_rows}, the batch {batch.tokens} tokens")
        _check(_attend(self.handle, x.data_ptr(), xs, cache.ref, batch.ref, self._scale if scale is None else scale,
                       window, o.data_ptr(), os_, _stream(self.device.index)))
        return out

    def _token_rows(self, t, what: str, written: bool = False):
        """[tokens, q_heads, head_dim] (a view of wider rows allowed) or [tokens, q_heads * head_dim]."""
        if t.dim() != 3:
            return _rows(t, what, self._q_width, self.dtype, self.device, written)
        rows, heads, width = t.shape
        stride, s1, s2 = t.stride()
        if heads != self.q_heads or width != self.head_dim or (s1 != width and heads > 1) or s2 != 1:
            _refuse(f"{what} {tuple(t.shape)} must be [tokens, {self.q_heads}, {self.head_dim}], dense in a token")
        if t.dtype != self.dtype or t.device != self.device:
            _refuse(f"{what} is {t.dtype} on {t.device}: {self.dtype} on {self.device} is wanted")
        return t, rows, stride if rows > 1 else self._q_width

    def device_error(self) -> None:
        gptq_q4_attn_device_error(self.handle)

    def close(self) -> None:
        if getattr(self, "handle", None):
            gptq_q4_attn_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
