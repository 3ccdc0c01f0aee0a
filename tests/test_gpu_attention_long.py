"""Attention where a CTA goes through many key tiles of an item, and where a
call has more requests than a warp looks at: the loops over key tiles with
their running maximum, the ring of stages used over and over, the shares of
large batches.  The tolerance is that of test_gpu_attention.py, plus kv / 16
2^-23 of A: each product of 16 keys is added to a running sum that may lose a
unit in its last place."""
import math
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
TYPES = pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])


@pytest.fixture(scope="module")
def q4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gptq_bit_weight_gb300 as q4mod
    return q4mod


def shares(lens, Hkv, G, window, stream):
    """How the units of a call fall to the CTAs: the units of a CTA, and for each item (request, head, its first key
    tile, its number of them, its row tile, its first unit).  Items are a request's row tiles for each key/value head:
    16 rows (streaming kernel) or two of 128 / G whole tokens."""
    items, u = [], 0
    for b, (ql, kv) in enumerate(lens):
        step = 2 * (128 // G)
        for h in range(Hkv):
            for i in range(-(-ql * G // 16) if stream else -(-ql // step)):
                if stream:
                    t0, t1 = 16 * i // G, (min(16 * i + 16, ql * G) - 1) // G
                else:
                    t0, t1 = i * step, min((i + 1) * step, ql) - 1
                hi = min(kv - ql + t1 + 1, kv)
                first = (max(0, kv - ql + t0 - window + 1) if window else 0) // 128
                n = -(-hi // 128) - first if hi > 0 else 1
                items.append((b, h, first, n, i, u))
                u += n
    ctas = torch.cuda.get_device_properties(0).multi_processor_count
    return max(1, -(-u // ctas)), items


class Call:
    """Requests with keys and values scattered over pages; slots that no token holds, pages that no request owns and
    pages before the window are NaN, and have no index in the table."""

    def __init__(self, q4, lens, Hkv, D, page, dtype, seed, window=0, level=None):
        g = torch.Generator(device=DEV).manual_seed(seed)
        need = [-(-kv // page) for _, kv in lens]
        order = torch.randperm(sum(need) + 2, generator=torch.Generator().manual_seed(seed))
        table = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32)
        pool = [torch.full((sum(need) + 2, Hkv, page, D), float("nan"), dtype=dtype, device=DEV) for _ in "kv"]
        self.lens, self.kv, at, self.cu = lens, [], 0, [0]
        for b, (ql, kv) in enumerate(lens):
            self.cu.append(self.cu[-1] + ql)
            own = [torch.randn(kv, Hkv, D, generator=g, device=DEV).to(dtype) for _ in "kv"]
            if level is not None:                        # the first coordinate of a key is its tile's level
                own[0] = (own[0].float() * 0.25).to(dtype)
                own[0][:, :, 0] = level(b).to(dtype)
            self.kv.append(own)
            gone = min(max(0, kv - ql - window + 1) // page, need[b]) if window else 0
            pages = order[at:at + need[b]]
            for to, t in zip(pool, own):
                padded = torch.full((need[b] * page, Hkv, D), float("nan"), dtype=dtype, device=DEV)
                padded[:kv] = t
                to[pages[gone:].to(DEV)] = padded.view(need[b], page, Hkv, D).transpose(1, 2)[gone:]
            table[b, gone:need[b]] = pages[gone:].to(torch.int32)
            at += need[b]
        i32 = dict(dtype=torch.int32, device=DEV)
        self.cache = q4.PagedCache(*pool)
        self.batch = lambda max_q: q4.PagedBatch(torch.tensor(self.cu, **i32), torch.tensor([kv for _, kv in lens], **i32),
                                                 table.to(DEV), tokens=self.cu[-1], max_q=max_q)

    def check(self, got, q, window, what):
        T, Hq, D = q.shape
        dt, scale, got = q.dtype, D ** -0.5, got.double()
        for b, (ql, kv) in enumerate(self.lens):
            rows = slice(self.cu[b], self.cu[b] + ql)
            if not ql:
                continue
            i, j = torch.arange(kv - ql, kv, device=DEV)[:, None], torch.arange(kv, device=DEV)[None, :]
            hidden = (j > i) | (j <= i - window if window else torch.zeros_like(j, dtype=torch.bool))
            Hkv = self.kv[b][0].shape[1]
            for h in range(Hkv):
                k, v = (t[:, h].double() for t in self.kv[b])
                x = q[rows].view(ql, Hkv, -1, D)[:, h].double().transpose(0, 1)               # [G, ql, D]
                p = torch.softmax((x @ k.t() * scale).masked_fill(hidden, -math.inf), -1)
                mag = ((x.abs() @ k.abs().t()) * scale).masked_fill(hidden, 0).amax(-1)
                o, A = p @ v, p @ v.abs()
                d = D * 2.0 ** -23 * mag[..., None]
                tol = U[dt] * o.abs() + (U[dt] + 2 * d + 2.0 ** -12 + kv / 16 * 2.0 ** -23) * A + \
                    TINY[dt] * (1 + kv * float(v.abs().max()))
                mine = got[rows].view(ql, Hkv, -1, D)[:, h].transpose(0, 1)
                err = (mine - o).abs()
                assert bool((err <= tol).all()), f"{what}, request {b}, head {h}: {float((err / tol).max()):.3f} tolerances"


# new tokens over 30000, query heads over 8: single tokens, drafts; one row tile, whose key tiles take two buffers in
# turn, with few rows (all threads add up the pieces) and more; two row tiles
LONG = {"token": (1, 8), "draft": (3, 32), "few_rows": (20, 16), "one_tile": (40, 16), "two_tiles": (100, 16)}


@TYPES
@pytest.mark.parametrize("window", [0, 20011])
@pytest.mark.parametrize("rising", [False, True], ids=["plain", "rising"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", list(LONG))
def test_many_key_tiles_of_an_item(q4, kind, D, rising, window, dtype):
    """Rising: the scores of some rows grow by 2^10 at the second, the fifth and the last key tile that a CTA has of
    an item, those of others half as much, or fall, or stay; neighbouring rows differ."""
    (ql, Hq), Hkv, page = LONG[kind], 8, 64
    lens, G, stream = [(ql, 30000)], Hq // Hkv, ql * Hq // Hkv <= 16
    per, items = shares(lens, Hkv, G, window, stream)
    assert per >= 8 and all(n >= 2 * per for _, _, _, n, _, _ in items)          # some CTA has `per` key tiles of each

    def level(b):
        x = torch.zeros(lens[b][1], Hkv)
        for _, h, first, n, _, u in items:
            for j in range(n):
                at = (u + j) % per
                x[(first + j) * 128:(first + j + 1) * 128, h] = 7 * ((at >= 1) + (at >= 4) + (at == per - 1))
        return x.to(DEV)

    call = Call(q4, lens, Hkv, D, page, dtype, seed=D + ql, window=window, level=level if rising else None)
    q = (torch.randn(ql, Hq, D, generator=torch.Generator().manual_seed(1)) * 2).to(dtype)
    if rising:
        way = torch.tensor([1.0, -1.0, 0.0, 0.5])[torch.arange(ql * Hq) * 7 // 5 % 4].view(ql, Hq)
        q[:, :, 0] = (way * D ** 0.5).to(dtype)
    q = q.to(DEV)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    batch = call.batch(ql)
    out = att.attend(q, call.cache, batch, window=window)
    call.check(out, q, window, kind)
    assert torch.equal(att.attend(q, call.cache, batch, window=window), out)
    att.device_error()


@TYPES
@pytest.mark.parametrize("window", [0, 700])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [33, 48, 330, 400])
def test_large_batches_of_any_lengths(q4, n, D, window, dtype):
    """Single tokens over contexts of up to 3000 beside chunks of several hundred, drafts and empty requests; more
    requests than a warp, and than a block, has threads."""
    r = random.Random(n + D)
    lens = []
    for b in range(n):
        kind = r.random()
        kv = r.randint(1, 3000 if n < 100 else 900)
        lens.append((1, kv) if kind < 0.7 else (r.randint(2, 9), max(9, kv)) if kind < 0.9 else (0, r.choice([0, kv])))
    chunks = {n // 3: (500, 1777), n - 2: (301, 301), 5: (130, 2500)}
    for b, c in chunks.items():
        lens[b] = c
    Hq, Hkv, page = 8, 2, 16
    call = Call(q4, lens, Hkv, D, page, dtype, seed=n, window=window)
    q = (torch.randn(call.cu[-1], Hq, D, generator=torch.Generator().manual_seed(2)) * 2).to(dtype).to(DEV)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    for max_q, stream in ((1, True), (500, False)):          # max_q chooses the kernel
        per, items = shares(lens, Hkv, Hq // Hkv, window, stream)
        cut = [x for x in items if x[5] // per != (x[5] + x[3] - 1) // per]
        assert len(cut) > 20 and any(x[4] > 0 for x in cut) and len({x[0] for x in items if x[4] > 0}) >= 3
        out = att.attend(q, call.cache, call.batch(max_q), window=window)
        call.check(out, q, window, f"max_q {max_q}")
        assert torch.equal(att.attend(q, call.cache, call.batch(max_q), window=window), out)
    att.device_error()
