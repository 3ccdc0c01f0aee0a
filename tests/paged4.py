"""What the tests of the 4-bit cache, of windows with sinks and of the pages share: a step's requests over either
cache, the 4-bit format by its definition, and attention in 64 bits.

Tolerance of an attention output: that of test_gpu_attention.py, whose terms hold for any 16-bit keys and values, and
so for the values that codes stand for; and kv / 16 2^-23 of A (test_gpu_attention_long.py) for running sums."""
import gc
import math

import pytest
import torch

DEV = "cuda:0"
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}


def quantise(x, group):
    """(codes, step, least) of a 16-bit tensor [.., D], from the definition, in 64 bits."""
    y = x.double().unflatten(-1, (-1, group))
    lo, hi = y.amin(-1), y.amax(-1)
    span = hi - lo
    ok = torch.isfinite(y).all(-1) & (span <= torch.finfo(torch.float32).max)
    step = (span / 15).to(x.dtype)
    c = torch.where((step > 0)[..., None], ((y - lo[..., None]) / step.double()[..., None]).round().clamp(0, 15),
                    torch.zeros_like(y))
    nan = torch.full_like(lo, float("nan"))
    c = torch.where(ok[..., None], c, torch.zeros_like(c)).flatten(-2)
    return c.to(torch.int64), torch.where(ok, step.double(), nan).to(x.dtype), torch.where(ok, lo, nan).to(x.dtype)


def values(code, step, least):
    y = code.double().unflatten(-1, (step.shape[-1], -1)) * step.double()[..., None] + least.double()[..., None]
    return y.flatten(-2).to(step.dtype)


def record(k, v):
    """Bytes of (code, step, least) of keys and values."""
    parts = []
    for code, _, _ in (k, v):
        words = torch.zeros((*code.shape[:-1], code.shape[-1] // 8), dtype=torch.int64)
        for e in range(8):
            words |= code[..., e::8] << (4 * (e // 2) + 16 * (e % 2))
        words = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
        parts.append(words.contiguous().view(torch.uint8))
    for _, step, least in (k, v):
        parts.append(torch.stack([step, least], -1).flatten(-2).contiguous().view(torch.uint8))
    return torch.cat(parts, -1)


class Step:
    """A step's requests and one layer's cache: of 16 bits (group None) or of 4.  Slots that no token holds read as NaN,
    as do pages that no request owns; table entries past a request's pages, and of pages between the first tokens and
    the window, are not valid indexes."""

    def __init__(self, q4, lens, Hkv, D, page, dtype, group=None, seed=0, lead=0, tail=0, window=0, sinks=0, device=DEV):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.Hkv, self.D, self.page, self.dtype, self.group = lens, Hkv, D, page, dtype, group
        need = [-(-kv // page) for _, kv in lens]
        width, total = max(need + [1]), sum(need)
        order = torch.randperm(total + 2, generator=g)
        self.table = torch.full((len(lens), width), -1, dtype=torch.int32)
        self.keys, self.values, at = [], [], 0
        if group:
            pool = torch.full((total + 2, Hkv, page, D + 8 * D // group), 255, dtype=torch.uint8)
        else:
            pool = torch.full((2, total + 2, Hkv, page, D), float("nan"), dtype=dtype)
        for b, (ql, kv) in enumerate(lens):
            k = (torch.randn(kv, Hkv, D, generator=g) + torch.randn(Hkv, D, generator=g)).to(dtype)
            v = torch.randn(kv, Hkv, D, generator=g).to(dtype)
            if group:
                kc, vc = quantise(k, group), quantise(v, group)
                k, v, rec = values(*kc), values(*vc), record(kc, vc)
            self.keys.append(k), self.values.append(v)
            oldest = max(0, kv - ql - window + 1) if window else 0             # of the window of the first new token
            for i in range(need[b]):
                n = min(page, kv - i * page)
                if window and (i + 1) * page <= oldest and i * page >= sinks:
                    continue
                p = int(order[at + i])
                self.table[b, i] = p
                rows = slice(i * page, i * page + n)
                if group:
                    pool[p, :, :n] = rec[rows].transpose(0, 1)
                else:
                    pool[0, p, :, :n], pool[1, p, :, :n] = k[rows].transpose(0, 1), v[rows].transpose(0, 1)
            at += need[b]
        self.cu = [lead]
        for ql, _ in lens:
            self.cu.append(self.cu[-1] + ql)
        self.tokens = self.cu[-1] + tail
        self.pool = pool.to(device)
        self.cache = q4.PagedCache4(self.pool, D, group, dtype) if group else q4.PagedCache(self.pool[0], self.pool[1])
        self.max_q = max([ql for ql, _ in lens] + [0])
        self.device = device
        self.batch = self.make_batch(q4, self.max_q)

    def make_batch(self, q4, max_q):
        return q4.PagedBatch(torch.tensor(self.cu, dtype=torch.int32, device=self.device),
                             torch.tensor([kv for _, kv in self.lens], dtype=torch.int32, device=self.device),
                             self.table.to(self.device), tokens=self.tokens, max_q=max_q)


def attention(step, q, scale, window=0, sinks=0):
    """(result, tolerance) [tokens, Hq, D] in 64 bits; rows without a request stay NaN."""
    T, Hq, D = q.shape
    G, dt = Hq // step.Hkv, q.dtype
    ref = torch.full((T, Hq, D), float("nan"), dtype=torch.float64)
    tol = torch.zeros_like(ref)
    for b, (ql, kv) in enumerate(step.lens):
        if not ql:
            continue
        rows = slice(step.cu[b], step.cu[b] + ql)
        qd = q[rows].double().view(ql, step.Hkv, G, D)
        k, v = step.keys[b].double(), step.values[b].double()
        i, j = torch.arange(kv - ql, kv)[:, None], torch.arange(kv)[None, :]
        seen = j <= i
        if window:
            seen = seen & ((j > i - window) | (j < sinks))
        s = (torch.einsum("thgd,jhd->hgtj", qd, k) * scale).masked_fill(~seen, -math.inf)
        mag = torch.einsum("thgd,jhd->hgtj", qd.abs(), k.abs()).masked_fill(~seen, 0) * abs(scale)
        top = s.amax(-1, keepdim=True).clamp(min=-1e300) if kv else torch.zeros(s.shape[:-1] + (1,), dtype=s.dtype)
        p = (s - top).exp()
        tot = p.sum(-1, keepdim=True)
        p = torch.where(tot > 0, p / tot.clamp(min=1e-300), torch.zeros_like(p))
        o, A = torch.einsum("hgtj,jhd->thgd", p, v), torch.einsum("hgtj,jhd->thgd", p, v.abs())
        d = D * 2.0 ** -23 * (mag.amax(-1) if kv else mag.sum(-1)).permute(2, 0, 1)[..., None]
        vmax = float(v.abs().max()) if v.numel() else 0.0
        t = U[dt] * o.abs() + (U[dt] + 2 * d + 2.0 ** -12 + kv / 16 * 2.0 ** -23) * A + TINY[dt] * (1 + kv * vmax) * (o.abs() > 0)
        ref[rows], tol[rows] = o.reshape(ql, Hq, D), t.reshape(ql, Hq, D)
    return ref, tol


@pytest.fixture(scope="module", autouse=True)
def no_handles_left():
    """Handles that a failed call's traceback keeps in a cycle are freed here, not while a later test captures a graph
    (freeing one synchronizes, which ends a capture)."""
    yield
    gc.collect()


def refused(q4, call, status=None):
    """Whether the call raises the library's error; keeps no traceback."""
    try:
        call()
    except q4.GPTQ4Error as e:
        return status is None or e.status == status
    return False


def check(got, ref, tol, what):
    got = got.double().cpu()
    own = ~torch.isnan(ref)
    err = (got - ref).abs()
    bad = own & ~(err <= tol)
    worst = float((err[own] / tol[own].clamp(min=1e-300)).max()) if own.any() else 0.0
    assert not bad.any(), f"{what}: {int(bad.sum())} of {int(own.sum())} outside, worst error / tolerance {worst:.3f}"
