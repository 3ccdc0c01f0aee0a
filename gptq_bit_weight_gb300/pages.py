"""The pages of a paged cache: free ones, forks, copies, compaction.

``PagePool`` marshals torch CUDA tensors to ``gptq_q4_pages_*`` (see
include/gptq_q4.h).  Nothing is counted on the side: which pages are in use
follows from the table and the lengths alone.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import (_check, _lib, _release, gptq_q4_buffer, gptq_q4_pages_device_error, gptq_q4_pages_free,
               gptq_q4_pages_make, gptq_q4_rows)
from .adapters import _refuse, _stream
from .attention import PagedCache4

_free_list, _fork = _lib.gptq_q4_pages_free_list, _lib.gptq_q4_pages_fork
_copy, _compact = _lib.gptq_q4_pages_copy, _lib.gptq_q4_pages_compact


class PagePool:
    """The pages of `caches`, the PagedCache or PagedCache4 of every layer: all
    of one number of pages and page size, sharing tables.  The pool keeps the
    caches alive.  table is int32 [batch, width], kv_len int32 [batch], as in
    PagedBatch; other index arguments are int32 on the same device."""

    def __init__(self, caches):
        self.handle = None
        self.caches = list(caches)
        if not self.caches:
            _refuse("a pool has at least one cache")
        kinds = {(c.struct.pages, c.kind[3], c.kind[1]) for c in self.caches}
        if len(kinds) != 1:
            _refuse(f"the caches differ in pages, page size or device: {sorted(map(str, kinds))}")
        self.pages, self.page_size, self.device = kinds.pop()
        buffers = []
        for c in self.caches:
            for t in (c.kv,) if isinstance(c, PagedCache4) else (c.k, c.v):
                size = math.prod(t.shape[1:]) * t.element_size()
                buffers.append(gptq_q4_buffer(t.data_ptr(), size, c.struct.page_stride * t.element_size()))
        _release()
        self.handle = gptq_q4_pages_make(buffers, self.pages, self.page_size)

    def _ints(self, t, what: str, n: int):
        if t.dtype != torch.int32 or t.device != self.device or t.dim() != 1 or not t.is_contiguous() or t.numel() != n:
            _refuse(f"{what} must be contiguous int32 [{n}] on {self.device}")
        return t.data_ptr()

    def _rows(self, table, kv_len):
        if table.dtype != torch.int32 or table.device != self.device or table.dim() != 2:
            _refuse(f"table must be int32 [batch, width] on {self.device}")
        batch, width = table.shape
        stride, inner = table.stride()
        if batch < 2:
            stride = max(stride, width)
        if (inner != 1 and width > 1 and batch) or stride < width:
            _refuse("table must be dense in its last dimension, its rows apart from each other")
        return gptq_q4_rows(table.data_ptr(), self._ints(kv_len, "kv_len", batch), stride, width, batch)

    def free(self, table, kv_len, window: int = 0, sinks: int = 0):
        """The pages that no row needs: (ids int32 [pages], ascending and then
        -1; count int32 [1]).  With a window, pages are needed that hold one of
        a row's last `window` tokens or of its first `sinks`."""
        rows = self._rows(table, kv_len)
        ids = torch.empty(self.pages, dtype=torch.int32, device=self.device)
        count = torch.empty(1, dtype=torch.int32, device=self.device)
        _check(_free_list(self.handle, ctypes.byref(rows), window, sinks, ids.data_ptr(), count.data_ptr(),
                          _stream(self.device.index)))
        return ids, count

    def fork(self, table, kv_len, parent, child, fresh) -> None:
        """Make rows child[i] of table and kv_len forks of rows parent[i]: they
        share full pages, and a partly filled last page is copied to page
        fresh[i] in every cache (else fresh[i] may be anything).  Negative
        numbers are no fork."""
        rows = self._rows(table, kv_len)
        n = parent.numel()
        _check(_fork(self.handle, ctypes.byref(rows), self._ints(parent, "parent", n), self._ints(child, "child", n),
                     self._ints(fresh, "fresh", n), n, _stream(self.device.index)))

    def copy(self, src, dst) -> None:
        """Copy pages src[i] to pages dst[i] in every cache; negative numbers are no copy."""
        n = src.numel()
        _check(_copy(self.handle, self._ints(src, "src", n), self._ints(dst, "dst", n), n, _stream(self.device.index)))

    def compact(self, table, kv_len, table_out=None, window: int = 0, sinks: int = 0):
        """Move the pages in use to the lowest numbers, in every cache, and
        write the table that names them to table_out (default: table itself).
        Returns their count, int32 [1]."""
        rows = self._rows(table, kv_len)
        out = table if table_out is None else table_out
        if out.shape != table.shape:
            _refuse(f"table_out {tuple(out.shape)} must be {tuple(table.shape)}")
        out_rows = self._rows(out, kv_len)
        count = torch.empty(1, dtype=torch.int32, device=self.device)
        _check(_compact(self.handle, ctypes.byref(rows), window, sinks, out_rows.table, out_rows.table_stride,
                        count.data_ptr(), _stream(self.device.index)))
        return count

    def device_error(self) -> None:
        gptq_q4_pages_device_error(self.handle)

    def close(self) -> None:
        if getattr(self, "handle", None):
            handle, self.handle = self.handle, None
            _release(gptq_q4_pages_free, handle)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
