"""Low-rank adapters of many requests beside a shared projection.

``LoraPool`` marshals torch CUDA tensors to ``gptq_q4_lora_*`` (see
include/gptq_q4.h); the library does the work and keeps its own copy of the
adapters.
"""
from __future__ import annotations

import torch

from . import (GPTQ4Error, GPTQ_Q4_DTYPE_BF16, GPTQ_Q4_DTYPE_FP16, GPTQ_Q4_DTYPE_FP32, GPTQ_Q4_INVALID_ARGUMENT,
               _check, _lib, _release, gptq_q4_lora_device_error, gptq_q4_lora_free, gptq_q4_lora_make,
               gptq_q4_lora_reserve, gptq_q4_lora_set)

_CODES = {torch.float16: GPTQ_Q4_DTYPE_FP16, torch.bfloat16: GPTQ_Q4_DTYPE_BF16, torch.float32: GPTQ_Q4_DTYPE_FP32}


def _refuse(message: str):
    raise GPTQ4Error(GPTQ_Q4_INVALID_ARGUMENT, message)


def _code(dtype) -> int:
    if dtype not in _CODES:
        _refuse(f"dtype {dtype} is not float16 or bfloat16")
    return _CODES[dtype]


# A small call's host time is most of it: these two spare a call a Stream object and a wrapper.
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_add = _lib.gptq_q4_lora_add


def _flat(t, what: str, width: int, written: bool):
    """`t`, not of two dimensions, as [rows, width]; a copy only where it is not written to."""
    n, at = 1, t.dim()
    while at and n < width:                              # the last dimensions that make up a row
        at -= 1
        n *= t.shape[at]
    if n != width and not (t.dim() == 1 and n % width == 0):
        _refuse(f"{what} {tuple(t.shape)} does not end in rows of {width} elements")
    flat = t.reshape(-1, width)
    if written and flat.data_ptr() != t.data_ptr():
        _refuse(f"{what} {tuple(t.shape)} cannot be viewed as rows")
    return flat


def _rows(t, what: str, width: int, dtype, device, written: bool = False):
    """`t` as rows of `width` elements, dense within a row: (tensor [rows, width], rows, row stride)."""
    if t.dtype != dtype or t.device != device:
        _refuse(f"{what} is {t.dtype} on {t.device}: {dtype} on {device} is wanted")
    if t.dim() != 2:
        t = _flat(t, what, width, written)
    rows, have = t.shape
    stride, inner = t.stride()
    if have != width:
        _refuse(f"{what} has rows of {have} elements: {width} are wanted")
    if inner != 1:
        _refuse(f"{what} is not dense within its rows")
    # one row, or none, has no stride of its own
    return t, rows, stride if rows > 1 else width


class LoraPool:
    """Up to `slots` adapters of one projection (K inputs, N outputs), each of
    its own rank up to max_rank; float16 or bfloat16."""

    def __init__(self, K: int, N: int, slots: int, max_rank: int, dtype=torch.float16):
        self.handle = None
        self.K, self.N, self.slots, self.max_rank, self.dtype = K, N, slots, max_rank, dtype
        self.device = torch.device("cuda", torch.cuda.current_device())
        _release()
        self.handle = gptq_q4_lora_make(K, N, slots, max_rank, _code(dtype))

    def set(self, slot: int, a, b, scale: float = 1.0) -> None:
        """Put an adapter into a slot: a [rank, K], b [N, rank]; the pool keeps a copy."""
        if a.dim() != 2 or b.dim() != 2 or a.shape[1] != self.K or b.shape != (self.N, a.shape[0]):
            _refuse(f"a {tuple(a.shape)} and b {tuple(b.shape)} must be [rank, {self.K}] and [{self.N}, rank]")
        for t, what in ((a, "a"), (b, "b")):
            if t.dtype != self.dtype or t.device != self.device:
                _refuse(f"{what} is {t.dtype} on {t.device}: {self.dtype} on {self.device} is wanted")
        a, b = a.contiguous(), b.contiguous()
        gptq_q4_lora_set(self.handle, slot, a.data_ptr(), b.data_ptr(), a.shape[0], scale,
                         _stream(self.device.index))

    def clear(self, slot: int) -> None:
        gptq_q4_lora_set(self.handle, slot, None, None, 0, 0.0,
                         _stream(self.device.index))

    def reserve(self, max_m: int) -> None:
        gptq_q4_lora_reserve(self.handle, max_m)

    def add(self, x, row_slot, y, out=None):
        """y plus each row's adapter: x [.., K] is the projection's input, y
        [.., N] its output, row_slot int32 [rows] each row's slot (negative:
        none).  out=y adds in place; rows of x, y and out may be strided."""
        dtype, device = self.dtype, self.device
        x2, M, xs = _rows(x, "x", self.K, dtype, device)
        y2, my, ys = _rows(y, "y", self.N, dtype, device)
        if out is None:
            out = torch.empty(y.shape, dtype=dtype, device=device)
            at, mo, os_ = out.data_ptr(), my, self.N
        else:
            o2, mo, os_ = _rows(out, "out", self.N, dtype, device, written=True)
            at = o2.data_ptr()
        if my != M or mo != M or row_slot.numel() != M:
            _refuse(f"x has {M} rows, y {my}, out {mo}, row_slot {row_slot.numel()}")
        if row_slot.dtype != torch.int32 or row_slot.device != device or not row_slot.is_contiguous():
            _refuse(f"row_slot must be contiguous int32 on {device}")
        _check(_add(self.handle, x2.data_ptr(), xs, row_slot.data_ptr(), M, y2.data_ptr(), ys, at, os_,
                    _stream(device.index)))
        return out

    def device_error(self) -> None:
        gptq_q4_lora_device_error(self.handle)

    def close(self) -> None:
        if getattr(self, "handle", None):
            handle, self.handle = self.handle, None
            _release(gptq_q4_lora_free, handle)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
