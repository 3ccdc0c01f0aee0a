"""Attention over a context whose one dominant key hides a long, flat tail: each of the tail's weights is below fp16's
least number beside the dominant one, all of them together are not below its precision.

The dominant key's value is zero, so the result is the tail's.  Tolerance, with o the result and A = sum p |v| = o (the
values have one sign): u o for the result's rounding, and (u + 2 d + 2^-12 + kv / 16 2^-23) A for weights of the normal
range, scores and sums, as in paged4.py; kv 2^-32 for weights below it, which are held at 2^7 times their size or more
and there off by at most 2^-25 each (values are at most 1)."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from paged4 import DEV, U, no_handles_left, quantise, record, values  # noqa: E402, F401


@pytest.fixture(scope="module")
def q4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gptq_bit_weight_gb300 as q4mod
    return q4mod


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("at", [0, 9000], ids=["first", "inside"])
@pytest.mark.parametrize("window", [0, 30000])
@pytest.mark.parametrize("max_q", [2, 100000], ids=["stream", "chunk"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group", [32, None], ids=["4bit", "16bit"])
def test_a_tail_below_a_dominant_key(q4, group, D, max_q, window, at, dtype):
    """Twenty requests of two tokens over one context: an item for each request and head, whole or nearly so in a CTA."""
    kv, Hq, Hkv, page, n, ql, sinks = 32768, 64, 8, 64, 20, 2, 4
    if window:
        at = max(at, 2 * page) if at else at           # a first token, or one of the window
    k, v = torch.zeros(kv, Hkv, D), torch.ones(kv, Hkv, D)
    v *= 0.5 + 0.5 * torch.rand(kv, Hkv, 1, generator=torch.Generator().manual_seed(1))
    v[at] = 0
    k[at, :, 0] = 4
    k, v = k.to(dtype), v.to(dtype)
    if group:
        kc, vc = quantise(k, group), quantise(v, group)
        rec = record(kc, vc)
        k, v = values(*kc), values(*vc)
        pool = rec.view(kv // page, page, Hkv, -1).transpose(1, 2).contiguous().to(DEV)
        cache = q4.PagedCache4(pool, D, group, dtype)
    else:
        cache = q4.PagedCache(*(t.view(kv // page, page, Hkv, D).transpose(1, 2).contiguous().to(DEV) for t in (k, v)))
    q = torch.zeros(n * ql, Hq, D, dtype=dtype)
    for t in range(n * ql):                            # 2^-25.2 to 2^-25.9 of the dominant weight, row by row
        q[t, :, 0] = torch.linspace(25.2, 25.9, Hq) * math.log(2) / 4 * D ** 0.5
    i32 = dict(dtype=torch.int32, device=DEV)
    batch = q4.PagedBatch(torch.arange(n + 1, **i32) * ql, torch.full((n,), kv, **i32),
                          torch.arange(kv // page, **i32).repeat(n, 1), tokens=n * ql, max_q=max_q)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    got = att.attend(q.to(DEV), cache, batch, window=window, sinks=sinks if window else 0).double().cpu()
    att.device_error()
    i, j = torch.arange(kv - ql, kv)[:, None], torch.arange(kv)[None, :]
    seen = j <= i
    if window:
        seen = seen & ((j > i - window) | (j < sinks))
    x = q[:ql].double().view(ql, Hkv, -1, D)
    s = (torch.einsum("thgd,jhd->hgtj", x, k.double()) * D ** -0.5).masked_fill(~seen, -math.inf)
    o = torch.einsum("hgtj,jhd->thgd", torch.softmax(s, -1), v.double()).reshape(ql, Hq, D)
    d = D * 2.0 ** -23 * float(s.max())
    tol = o * (2 * U[dtype] + 2 * d + 2.0 ** -12 + kv / 16 * 2.0 ** -23) + kv * 2.0 ** -32
    assert float(o.min()) > 20 * float(tol.max() - (o * U[dtype]).max())        # the tail is there to be seen
    err = (got.view(n, ql, Hq, D) - o).abs() / tol
    assert bool((err <= 1).all()), f"worst error / tolerance {float(err.max()):.3f}"


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("max_q", [1, 100000], ids=["stream", "chunk"])
@pytest.mark.parametrize("step", [4, 8, 32])
@pytest.mark.parametrize("group", [32, None], ids=["4bit", "16bit"])
def test_weights_stay_finite_under_huge_scores(q4, group, step, max_q, dtype):
    """Scores of about 2^25 that rise a little every other tile: fp32 holds them in steps of 4, so a reference may be off
    by units of the exponent.  Whatever the weights are then, the result lies between the values."""
    kv, H, D, page, n, ql = 1024, 16, 64, 64, 160, 2                  # an item whole, or nearly so, in a CTA
    k, v = torch.zeros(kv, 1, D), 0.5 + 0.5 * torch.rand(kv, 1, 1, generator=torch.Generator().manual_seed(2)).expand(kv, 1, D)
    k[:, :, 0] = 4096
    k[:, :, 32] = (torch.arange(kv) // 256 * step / 4)[:, None]       # a group of its own
    k, v = k.to(dtype), v.to(dtype)
    if group:
        kc, vc = quantise(k, group), quantise(v, group)
        cache = q4.PagedCache4(record(kc, vc).view(kv // page, page, 1, -1).transpose(1, 2).contiguous().to(DEV), D, group, dtype)
        v = values(*vc)
    else:
        cache = q4.PagedCache(*(t.reshape(kv // page, page, 1, D).transpose(1, 2).contiguous().to(DEV) for t in (k, v)))
    q = torch.zeros(n * ql, H, D)
    q[:, :, 0] = 8192 + 64 * (torch.arange(n * ql * H) % 61).view(n * ql, H)
    q[:, :, 32] = 4
    i32 = dict(dtype=torch.int32, device=DEV)
    att = q4.PagedAttention(H, 1, D, page, dtype=dtype)
    batch = q4.PagedBatch(torch.arange(n + 1, **i32) * ql, torch.full((n,), kv, **i32), torch.arange(kv // page, **i32).repeat(n, 1),
                          tokens=n * ql, max_q=max_q)
    for scale in (1.366, 1.0, 0.5):
        got = att.attend(q.to(dtype).to(DEV), cache, batch, scale=scale).float().cpu()
        edge = 1 + 4 * U[dtype]
        assert bool(((got >= float(v.min()) / edge) & (got <= float(v.max()) * edge)).all()), scale
    att.device_error()
