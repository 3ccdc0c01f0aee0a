"""Rotary positions with the append to the paged cache, and attention over
it, against the definitions in 64 bits.

Tolerance of an attention output, with A = sum_j p_j |v_j| over the visible
keys and u the type's unit roundoff: u |ref| for the one rounding of the
result; u A for weights p rounded to 16 bits (and 2^-25 n max|v| for weights
below fp16's normal range); and (2 d + 2^-12) A for the scores' fp32 sums
(d = head_dim 2^-23 scale sum|q k|, the bound of any order of summation, at
twice the unit roundoff for truncating adders), exponentials and sums of
exponentials (2^-12 together, far above their 2^-21).  A rotated element is
off by its rounding and 4 2^-24 (|a| + |b|) length_scale for the fp32
products, sum, cosine and sine."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}


@pytest.fixture(scope="module")
def q4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gptq_bit_weight_gb300 as q4mod
    return q4mod


class Step:
    """A step's requests and one layer's cache.  Slots that no token holds are NaN, and so are the
    pages that no request owns; table entries past a request's pages are not valid indexes."""

    def __init__(self, q4, lens, Hkv, D, page, dtype, seed=0, lead=0, tail=0, window=0, interleave=False):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.Hkv, self.D, self.page = lens, Hkv, D, page
        need = [-(-kv // page) for _, kv in lens]
        width, total = max(need + [1]), sum(need)
        order = torch.randperm(total + 2, generator=g)
        self.table = torch.full((len(lens), width), -1, dtype=torch.int32)
        nan = torch.full((total + 2, Hkv, page, D), float("nan"), dtype=dtype)
        self.k, self.v, at = nan, nan.clone(), 0
        self.keys, self.values = [], []
        for b, (ql, kv) in enumerate(lens):
            k, v = torch.randn(kv, Hkv, D, generator=g).to(dtype), torch.randn(kv, Hkv, D, generator=g).to(dtype)
            self.keys.append(k), self.values.append(v)
            first = max(0, kv - ql - window + 1) // page if window else 0      # pages before the window are gone
            for i in range(need[b]):
                p = int(order[at + i])
                n = min(page, kv - i * page)
                if i >= first:
                    self.table[b, i] = p
                    self.k[p, :, :n], self.v[p, :, :n] = k[i * page:i * page + n].transpose(0, 1), v[i * page:i * page + n].transpose(0, 1)
            at += need[b]
        cu = [lead]
        for ql, _ in lens:
            cu.append(cu[-1] + ql)
        self.cu, self.tokens = cu, cu[-1] + tail
        if interleave:                       # keys and values of a page side by side in one tensor
            both = torch.stack([self.k, self.v], 1).to(DEV)
            self.cache = q4.PagedCache(both[:, 0], both[:, 1])
        else:
            self.cache = q4.PagedCache(self.k.to(DEV), self.v.to(DEV))
        self.max_q = max([ql for ql, _ in lens] + [0])
        self.batch = self.make_batch(q4, self.max_q)

    def make_batch(self, q4, max_q):
        return q4.PagedBatch(torch.tensor(self.cu, dtype=torch.int32, device=DEV),
                             torch.tensor([kv for _, kv in self.lens], dtype=torch.int32, device=DEV),
                             self.table.to(DEV), tokens=self.tokens, max_q=max_q)


def attention_reference(step, q, scale, window):
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
        s = torch.einsum("thgd,jhd->hgtj", qd, k) * scale
        mag = torch.einsum("thgd,jhd->hgtj", qd.abs(), k.abs()) * abs(scale)
        i, j = torch.arange(kv - ql, kv)[:, None], torch.arange(kv)[None, :]
        seen = j <= i
        if window:
            seen &= j > i - window
        s = s.masked_fill(~seen, -math.inf)
        top = s.amax(-1, keepdim=True).clamp(min=-1e300) if kv else torch.zeros(s.shape[:-1] + (1,), dtype=s.dtype)
        p = (s - top).exp()
        tot = p.sum(-1, keepdim=True)
        p = torch.where(tot > 0, p / tot.clamp(min=1e-300), torch.zeros_like(p))
        o = torch.einsum("hgtj,jhd->thgd", p, v)
        A = torch.einsum("hgtj,jhd->thgd", p, v.abs())
        d = D * 2.0 ** -23 * (mag.masked_fill(~seen, 0).amax(-1) if kv else mag.sum(-1))
        d = d.permute(2, 0, 1)[..., None]
        vmax = float(v.abs().max()) if v.numel() else 0.0
        ref[rows] = o.reshape(ql, Hq, D)
        t = U[dt] * o.abs() + (U[dt] + 2 * d + 2.0 ** -12) * A + TINY[dt] * (1 + kv * vmax) * (o.abs() > 0)
        tol[rows] = t.reshape(ql, Hq, D)
    return ref, tol


def check(got, ref, tol, what):
    got = got.double().cpu()
    own = ~torch.isnan(ref)
    err = (got - ref).abs()
    bad = own & ~(err <= tol)
    worst = float((err[own] / tol[own].clamp(min=1e-300)).max()) if own.any() else 0.0
    assert not bad.any(), f"{what}: {int(bad.sum())} of {int(own.sum())} outside, worst error / tolerance {worst:.3f}"


LENS = {
    "one": [(1, 1)],
    "one_long": [(1, 1500)],
    "tile_edges": [(1, n) for n in (7, 8, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257)],
    "empty_requests": [(0, 40), (1, 33), (0, 0), (3, 3), (0, 1)],
    "rows_that_see_nothing": [(5, 2), (4, 0), (1, 0), (2, 9)],
    "few_tokens": [(4, 200), (7, 7), (2, 65), (9, 300)],
    "chunk": [(130, 130)],
    "chunk_over_cache": [(65, 700), (33, 513)],
    "mixed": [(1, 300), (70, 400), (1, 17), (2, 2), (129, 129), (1, 600), (0, 5), (16, 16)],
    "late_chunk_sees_nothing_first": [(150, 20), (40, 300)],
}
SHAPES = [  # Hq, Hkv, D, page
    (4, 4, 128, 16),
    (16, 2, 128, 32),
    (6, 2, 64, 8),
    (5, 1, 128, 64),
    (8, 1, 64, 128),
    (20, 1, 128, 16),
    (48, 1, 64, 32),
    (128, 1, 128, 256),
]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("lens", list(LENS), ids=str)
def test_attend(q4, lens, shape, dtype):
    Hq, Hkv, D, page = shape
    if Hq * max(ql for ql, _ in LENS[lens]) > 9000:
        pytest.skip("the same tiles as the smaller head counts")
    step = Step(q4, LENS[lens], Hkv, D, page, dtype, seed=Hq + page, lead=2, tail=3)
    q = (torch.randn(step.tokens, Hq, D, generator=torch.Generator().manual_seed(1)) * 2).to(dtype)
    ref, tol = attention_reference(step, q, D ** -0.5, 0)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    qd = q.to(DEV)
    first = None
    # max_q chooses the kernel: as it is, and as large as allowed
    for batch in (step.batch, step.make_batch(q4, 100000)):
        out = torch.full_like(qd, float("nan"))
        att.attend(qd, step.cache, batch, out=out)
        check(out, ref, tol, f"max_q {batch.struct.max_q}")
        assert torch.isnan(out.cpu()[torch.isnan(ref)]).all()        # rows of no request are left alone
        again = torch.full_like(qd, float("nan"))
        att.attend(qd, step.cache, batch, out=again)
        assert torch.equal(torch.nan_to_num(out), torch.nan_to_num(again))
    att.device_error()


@pytest.mark.parametrize("max_q", [None, 100000])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("window", [1, 16, 100, 257])
@pytest.mark.parametrize("shape", [(4, 4, 128, 16), (16, 2, 64, 32), (10, 2, 128, 64)], ids=lambda s: "x".join(map(str, s)))
def test_window(q4, shape, window, dtype, max_q):
    """Pages before the window are not there any more (their table entries are no page)."""
    Hq, Hkv, D, page = shape
    step = Step(q4, [(1, 500), (1, 30), (3, 400), (140, 350), (150, 150), (4, 2)], Hkv, D, page, dtype, seed=3,
                window=window)
    q = (torch.randn(step.tokens, Hq, D, generator=torch.Generator().manual_seed(2)) * 2).to(dtype)
    ref, tol = attention_reference(step, q, D ** -0.5, window)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    batch = step.batch if max_q is None else step.make_batch(q4, max_q)
    check(att.attend(q.to(DEV), step.cache, batch, window=window), ref, tol, f"window {window}")
    att.device_error()


@pytest.mark.parametrize("max_q", [1, 100000])
@pytest.mark.parametrize("window", [2 ** 30 - 1, 2 ** 30, 2 ** 31 - 1])
@pytest.mark.parametrize("D", [64, 128])
def test_window_longer_than_any_context(q4, D, window, max_q):
    """The largest windows hide nothing, for requests with more new tokens than context among them (their first rows
    have negative indexes, of which a window is subtracted)."""
    Hq, Hkv, page, dtype = 4, 2, 16, torch.bfloat16
    step = Step(q4, [(10, 5), (5, 2), (1, 300), (160, 20), (40, 0), (3, 200)], Hkv, D, page, dtype, seed=14)
    q = torch.randn(step.tokens, Hq, D, generator=torch.Generator().manual_seed(13)).to(dtype)
    ref, tol = attention_reference(step, q, D ** -0.5, 0)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    check(att.attend(q.to(DEV), step.cache, step.make_batch(q4, max_q), window=window), ref, tol, f"window {window}")
    att.device_error()


@pytest.mark.parametrize("lens", [[(1, 400), (1, 70)], [(140, 400), (1, 70)]], ids=["tokens", "chunk"])
def test_strided_rows_scale_and_stream(q4, lens):
    """q as columns of wider rows, out as columns of wider rows, keys and values side by side in a
    page, another scale, on a side stream."""
    Hq, Hkv, D, page, dtype = 8, 2, 128, 16, torch.bfloat16
    step = Step(q4, lens, Hkv, D, page, dtype, seed=4, interleave=True)
    wide = torch.randn(step.tokens, Hq * D + 264, generator=torch.Generator().manual_seed(3)).to(dtype)
    q = wide[:, 8:8 + Hq * D].reshape(-1, Hq, D)
    ref, tol = attention_reference(step, q, 0.2, 0)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    wd = wide.to(DEV)
    out = torch.full((step.tokens, Hq * D + 64), 7.0, dtype=dtype, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        att.attend(wd[:, 8:8 + Hq * D], step.cache, step.batch, scale=0.2, out=out[:, 16:16 + Hq * D])
    side.synchronize()
    check(out[:, 16:16 + Hq * D].reshape(-1, Hq, D), ref, tol, "strided")
    assert (out[:, :16] == 7).all() and (out[:, 16 + Hq * D:] == 7).all()
    att.device_error()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("lens", [[(1, 900)], [(140, 600)], [(1, 64), (130, 130)]], ids=["token", "chunk", "both"])
def test_rising_and_extreme_scores(q4, lens, dtype):
    """Scores that rise along the context (the running maximum moves at every tile), spread over
    hundreds, with equal largest ones; and a request whose keys make every score the same."""
    Hq, Hkv, D, page = 4, 2, 128, 16
    step = Step(q4, lens, Hkv, D, page, dtype, seed=5)
    g = torch.Generator().manual_seed(6)
    for b, (ql, kv) in enumerate(lens):
        ramp = torch.linspace(-1, 1, kv)[:, None, None]
        k = (ramp * torch.ones(1, Hkv, D) + 0.02 * torch.randn(kv, Hkv, D, generator=g)).to(dtype)
        if b == 1:
            k = torch.ones(kv, Hkv, D, dtype=dtype)
        step.keys[b] = k
        for i in range(-(-kv // page)):
            n = min(page, kv - i * page)
            step.cache.k[int(step.table[b, i]), :, :n] = k[i * page:i * page + n].transpose(0, 1).to(DEV)
    q = torch.full((step.tokens, Hq, D), 3.0).to(dtype)
    q[:, 1] = -3.0                                        # and falling ones
    q[:, 2] = 0.0                                         # and none: the plain mean
    ref, tol = attention_reference(step, q, 1.0, 0)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    check(att.attend(q.to(DEV), step.cache, step.batch, scale=1.0), ref, tol, "rising scores")
    check(att.attend(q.to(DEV), step.cache, step.make_batch(q4, 100000), scale=1.0), ref, tol, "rising scores")
    att.device_error()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("max_q", [1, 100000])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_see_nothing_beside_values_without_number(q4, D, max_q, bad):
    """More new tokens than context, and no number in a value that only the later ones see: the first ones' outputs
    are zeros, in items of one CTA and in those that two share (of 300 tokens, at two key tiles a CTA)."""
    Hq, Hkv, page, dtype = 4, 4, 16, torch.bfloat16
    lens = [(9, 4), (300, 290), (1510, 1500), (70, 66), (4, 4)]
    step = Step(q4, lens, Hkv, D, page, dtype, seed=17)
    for b, at in ((0, 3), (1, 4), (1, 200), (1, 289), (2, 4), (2, 1499), (3, 60)):
        step.cache.v[int(step.table[b, at // page]), :, at % page] = bad
    q = torch.randn(step.tokens, Hq, D, generator=torch.Generator().manual_seed(16)).to(dtype)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    out = att.attend(q.to(DEV), step.cache, step.make_batch(q4, max_q)).cpu()
    for b, (ql, kv) in enumerate(lens):
        rows = out[step.cu[b]:step.cu[b] + ql]
        assert (rows[:ql - kv] == 0).all(), b                # they see nothing
        if b == 4:
            assert torch.isfinite(rows).all()                # another request's values are not its own
        else:
            assert not torch.isfinite(rows[-1]).any(), b
    att.device_error()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("max_q,tile", [(1, 16), (100000, 256)])
@pytest.mark.parametrize("D", [64, 128])
def test_values_without_number_stay_in_their_tiles(q4, D, max_q, tile, window, bad):
    """A NaN or infinity in one value: rows that see it have no number, rows of other tiles (tokens, at one query head
    for each key/value head) and of other requests and heads are right."""
    Hq, Hkv, page, dtype, at = 2, 2, 16, torch.float16, 300
    step = Step(q4, [(600, 600), (9, 500)], Hkv, D, page, dtype, seed=20)
    q = torch.randn(step.tokens, Hq, D, generator=torch.Generator().manual_seed(18)).to(dtype)
    ref, tol = attention_reference(step, q, D ** -0.5, window)
    step.cache.v[int(step.table[0, at // page]), 1, at % page] = bad
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    out = att.attend(q.to(DEV), step.cache, step.make_batch(q4, max_q), window=window).cpu()
    end = at + window if window else 600                  # the first row that no longer sees it
    assert not torch.isfinite(out[at:end, 1]).any()
    ref[at // tile * tile:min(-(-end // tile) * tile, 600), 1] = float("nan")       # no claim for the rest of the tiles
    check(out, ref, tol, f"beside {bad}")
    att.device_error()


@pytest.mark.parametrize("max_q", [1, 100000])
def test_cache_past_32_bit_offsets(q4, max_q):
    """Pages that begin more than 2^32 bytes into the cache."""
    Hq, Hkv, D, page, dtype = 8, 2, 128, 16, torch.float16
    step = Step(q4, [(1, 100), (1, 37)], Hkv, D, page, dtype, seed=7)
    n, stride = step.k.shape[0], 1 << 28
    size = (n - 1) * stride + Hkv * page * D
    inner = (page * D, D, 1)
    k, v = (torch.empty(size, dtype=dtype, device=DEV).as_strided((n, Hkv, page, D), (stride, *inner)) for _ in "kv")
    k.copy_(step.k), v.copy_(step.v)
    q = torch.randn(step.tokens, Hq, D, generator=torch.Generator().manual_seed(4)).to(dtype)
    ref, tol = attention_reference(step, q, D ** -0.5, 0)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    check(att.attend(q.to(DEV), q4.PagedCache(k, v), step.make_batch(q4, max_q)), ref, tol, "large offsets")
    att.device_error()


def test_many_requests(q4):
    """More requests than a block has threads, most of them tiny."""
    Hq, Hkv, D, page, dtype = 4, 2, 64, 8, torch.float16
    g = torch.Generator().manual_seed(8)
    lens = [(int(a), int(a) + int(b)) for a, b in zip(torch.randint(0, 3, (1500,), generator=g), torch.randint(0, 40, (1500,), generator=g))]
    step = Step(q4, lens, Hkv, D, page, dtype, seed=8)
    q = torch.randn(step.tokens, Hq, D, generator=g).to(dtype)
    ref, tol = attention_reference(step, q, D ** -0.5, 0)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    qd = q.to(DEV)
    for max_q in (2, 100000):
        check(att.attend(qd, step.cache, step.make_batch(q4, max_q)), ref, tol, "many requests")
    att.device_error()


@pytest.mark.parametrize("max_q", [1, 100000])
def test_lengths_and_pages_out_of_range_are_reported(q4, max_q):
    """Bad device data ends in a status, and leaves the other requests right."""
    Hq, Hkv, D, page, dtype = 4, 2, 128, 16, torch.float16
    step = Step(q4, [(1, 100), (1, 50)], Hkv, D, page, dtype, seed=9)
    q = torch.randn(step.tokens, Hq, D, generator=torch.Generator().manual_seed(5)).to(dtype)
    ref, tol = attention_reference(step, q, D ** -0.5, 0)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    qd = q.to(DEV)
    for what in ("kv", "page", "page_high", "kv_negative", "cu"):
        cu, kv, table = (t.clone() for t in step.batch.tensors)
        if what == "kv":
            kv[0] = 100000
            table[0].clamp_(min=0)
        if what == "kv_negative":
            kv[0] = -3
        if what == "page":
            table[0, 2] = -1
        if what == "page_high":
            table[0, 2] = 10 ** 9
        if what == "cu":
            cu[2] = 1000
        out = att.attend(qd, step.cache, q4.PagedBatch(cu, kv, table, tokens=step.tokens, max_q=max_q))
        if what != "cu":
            check(out[1:], ref[1:], tol[1:], what)
        with pytest.raises(q4.GPTQ4Error) as e:
            att.device_error()
        assert e.value.status == q4.GPTQ_Q4_DEVICE_FAULT
    check(att.attend(qd, step.cache, step.make_batch(q4, max_q)), ref, tol, "afterwards")
    att.device_error()


@pytest.mark.parametrize("max_q", [1, 100000])
def test_any_row_ranges_are_cut_to_the_rows(q4, max_q):
    """Row ranges at the ends of 32 bits: reported, nothing is written outside the rows, and nothing is appended."""
    Hq, Hkv, D, page, dtype = 2, 1, 64, 8, torch.float16
    low, high = -2 ** 31, 2 ** 31 - 1
    step = Step(q4, [(3, 20), (2, 9)], Hkv, D, page, dtype, seed=15)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    x = torch.randn(step.tokens, 4 * D, generator=torch.Generator().manual_seed(14)).to(dtype).to(DEV)
    for cu in ([0, 3, low], [0, low, low], [2, low, high], [low, high, low], [high, low, 3], [0, high, 5], [low, low, low]):
        batch = q4.PagedBatch(torch.tensor(cu, dtype=torch.int32, device=DEV), *step.batch.tensors[1:],
                              tokens=step.tokens, max_q=max_q)
        room = torch.full((step.tokens + 64, Hq * D), 7.0, dtype=dtype, device=DEV)
        att.attend(x[:, :Hq * D], step.cache, batch, out=room[32:32 + step.tokens])
        assert (room[:32] == 7).all() and (room[32 + step.tokens:] == 7).all()
        with pytest.raises(q4.GPTQ4Error) as e:
            att.device_error()
        assert e.value.status == q4.GPTQ_Q4_DEVICE_FAULT
        cache = q4.PagedCache(step.k.to(DEV), step.v.to(DEV))
        att.append(x, cache, batch, q_out=room[32:32 + step.tokens])
        if cu == [0, 3, low]:                             # the first request's range is right
            p, o = int(step.table[0, 2]), slice(1, 4)
            cache.k[p, :, o] = cache.v[p, :, o] = float("nan")
            step.k[p, :, o] = step.v[p, :, o] = float("nan")
        assert torch.equal(torch.nan_to_num(cache.k.cpu(), nan=99.0), torch.nan_to_num(step.k, nan=99.0))
        assert torch.equal(torch.nan_to_num(cache.v.cpu(), nan=99.0), torch.nan_to_num(step.v, nan=99.0))
        assert (room[:32] == 7).all() and (room[32 + step.tokens:] == 7).all()
        try:
            att.device_error()
        except q4.GPTQ4Error as e:                        # if the range held a row
            assert e.status == q4.GPTQ_Q4_DEVICE_FAULT


@pytest.mark.parametrize("max_q", [1, 100000])
def test_more_work_than_a_call_counts_is_reported_and_not_done(q4, max_q):
    """2^31 tiles of work, from lengths alone: nothing is read or written."""
    heads, D, page = 128, 64, 1024
    i32 = torch.int32
    att = q4.PagedAttention(heads, heads, D, page)
    k = torch.zeros(1, heads, page, D, dtype=torch.float16, device=DEV)
    batch = q4.PagedBatch(torch.tensor([0, 600], dtype=i32, device=DEV), torch.tensor([2 ** 30], dtype=i32, device=DEV),
                          torch.zeros(1, 2 ** 20, dtype=i32, device=DEV), tokens=600, max_q=max_q)
    out = torch.full((600, heads, D), 5.0, dtype=torch.float16, device=DEV)
    att.attend(torch.zeros_like(out), q4.PagedCache(k, k), batch, out=out)
    with pytest.raises(q4.GPTQ4Error) as e:
        att.device_error()
    assert e.value.status == q4.GPTQ_Q4_DEVICE_FAULT
    assert (out == 5).all()


# ------------------------------------------------------------------ append

def rotate_reference(x, pos, freqs, length, interleaved, dtype):
    """(result, tolerance) of rotated heads x [T, H, D]."""
    xd, rot = x.double(), 2 * len(freqs)
    f = torch.tensor(freqs, dtype=torch.float64)
    angle = pos.double()[:, None] * f
    c, s = (angle.cos() * length)[:, None], (angle.sin() * length)[:, None]
    i0 = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    i1 = i0 + (1 if interleaved else rot // 2)
    a, b = xd[..., i0], xd[..., i1]
    out, tol = xd.clone(), torch.zeros_like(xd)
    out[..., i0], out[..., i1] = a * c - b * s, b * c + a * s
    slack = 4 * 2.0 ** -24 * (a.abs() + b.abs()) * length
    tol[..., i0] = U[dtype] * out[..., i0].abs() + slack + TINY[dtype]
    tol[..., i1] = U[dtype] * out[..., i1].abs() + slack + TINY[dtype]
    return out, tol


ROPES = [  # rotary_dim, interleaved, keywords
    (128, False, {}),
    (64, True, {"base": 500000.0, "scaling": "bands", "factor": 8.0, "low": 1.0, "high": 4.0, "original": 512}),
    (32, False, {"scaling": "linear", "factor": 4.0}),
    (16, True, {"scaling": "ntk", "factor": 2.0}),
    (48, False, {"scaling": "yarn", "factor": 4.0, "low": 1.0, "high": 32.0, "original": 256}),
    (0, False, {}),
]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("rope", ROPES, ids=lambda r: f"{r[0]}{'i' if r[1] else 'h'}{r[2].get('scaling', '')}")
@pytest.mark.parametrize("shape", [(4, 4, 128, 16), (8, 1, 64, 8), (10, 2, 128, 64)], ids=lambda s: "x".join(map(str, s)))
def test_append(q4, shape, rope, dtype):
    Hq, Hkv, D, page = shape
    rot, interleaved, kw = rope
    rot = min(rot, D)
    step = Step(q4, LENS["mixed"], Hkv, D, page, dtype, seed=10, lead=1, tail=2)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    att.set_rope(rot, 2000, interleaved=interleaved, **kw)
    freqs, length = [], 1.0
    if rot:
        kind = {"linear": 1, "ntk": 2, "bands": 3, "yarn": 4}.get(kw.get("scaling"), 0)
        freqs, length = q4.gptq_q4_rope_freqs(rot, kw.get("base", 10000.0), kind, kw.get("factor", 1.0),
                                              kw.get("low", 1.0), kw.get("high", 4.0), kw.get("original", 1))
    T, W = step.tokens, (Hq + 2 * Hkv) * D
    wide = torch.randn(T, W + 24, generator=torch.Generator().manual_seed(6)).to(dtype)
    heads = wide[:, 8:8 + W].reshape(T, Hq + 2 * Hkv, D)
    index = torch.full((T,), -1)
    for b, (ql, kv) in enumerate(step.lens):
        index[step.cu[b]:step.cu[b] + ql] = torch.arange(kv - ql, kv)
    for positions in (None, torch.randint(0, 2000, (T,), generator=torch.Generator().manual_seed(7), dtype=torch.int32)):
        pos = (index if positions is None else positions).clamp(min=0)
        turned, tol = (rotate_reference(heads[:, :Hq + Hkv], pos, freqs, length, interleaved, dtype) if rot
                       else (heads[:, :Hq + Hkv].double(), torch.zeros(T, Hq + Hkv, D, dtype=torch.float64)))
        cache = q4.PagedCache(step.k.to(DEV), step.v.to(DEV))
        wd = wide.to(DEV)
        q_out = torch.full((T, Hq, D), float("nan"), dtype=dtype, device=DEV)
        att.append(wd[:, 8:8 + W], cache, step.batch, positions=None if positions is None else positions.to(DEV), q_out=q_out)
        mine = index >= 0
        got = q_out.double().cpu()
        assert ((got - turned[:, :Hq]).abs() <= tol[:, :Hq])[mine].all()
        assert torch.isnan(got[~mine]).all()
        # the cache: new tokens written, everything else untouched
        want_v, k, v = step.v.clone(), cache.k.cpu(), cache.v.cpu()
        old_k = step.k.clone()
        for b, (ql, kv) in enumerate(step.lens):
            for t in range(ql):
                i, row = kv - ql + t, step.cu[b] + t
                p, o = int(step.table[b, i // page]), i % page
                want_v[p, :, o] = heads[row, Hq + Hkv:]
                assert ((k[p, :, o].double() - turned[row, Hq:]).abs() <= tol[row, Hq:]).all()
                k[p, :, o] = old_k[p, :, o] = 0
        assert torch.equal(torch.nan_to_num(v, nan=99.0), torch.nan_to_num(want_v, nan=99.0))
        assert torch.equal(torch.nan_to_num(k, nan=99.0), torch.nan_to_num(old_k, nan=99.0))
        # in place: the queries' columns of qkv themselves
        att.append(wd[:, 8:8 + W], cache, step.batch, positions=None if positions is None else positions.to(DEV),
                   q_out=wd[:, 8:8 + Hq * D])
        assert torch.equal(wd[:, 8:8 + Hq * D].reshape(T, Hq, D)[mine.to(DEV)], q_out[mine.to(DEV)])
        assert torch.equal(wd[:, 8 + Hq * D:].cpu(), wide[:, 8 + Hq * D:])
    att.device_error()


def test_positions_of_a_long_context(q4):
    """A million tokens in, an angle in fp32 would be off by hundredths of a turn."""
    Hq, Hkv, D, page, dtype = 2, 1, 64, 8, torch.float16
    step = Step(q4, [(2, 10)], Hkv, D, page, dtype, seed=11)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    att.set_rope(64, 1 << 20)
    x = torch.randn(2, 4, D, generator=torch.Generator().manual_seed(8)).to(dtype)
    pos = torch.tensor([(1 << 20) - 1, 999983], dtype=torch.int32)
    q = att.append(x.view(2, -1).to(DEV), step.cache, step.batch, positions=pos.to(DEV))
    freqs, _ = q4.gptq_q4_rope_freqs(64, 10000.0, 0)
    ref, tol = rotate_reference(x[:, :2], pos, freqs, 1.0, False, dtype)
    assert ((q.double().cpu() - ref).abs() <= tol).all()
    att.device_error()


def test_append_out_of_range_is_reported_and_not_written(q4):
    Hq, Hkv, D, page, dtype = 2, 1, 64, 8, torch.float16
    step = Step(q4, [(1, 10), (1, 5)], Hkv, D, page, dtype, seed=12)
    x = torch.randn(2, 4 * D, generator=torch.Generator().manual_seed(9)).to(dtype).to(DEV)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    att.set_rope(64, 16)
    ok_rows = {}
    for what in ("fine", "position", "page", "short", "long"):
        cu, kv, table = (t.clone() for t in step.batch.tensors)
        pos = torch.tensor([9, 4], dtype=torch.int32, device=DEV)
        if what == "position":
            pos[0] = 16
        if what == "page":
            table[0, 1] = step.k.shape[0]
        if what == "short":
            kv[0] = 0
        if what == "long":
            kv[0] = 1000
        cache = q4.PagedCache(step.k.to(DEV), step.v.to(DEV))
        q = torch.zeros(2, Hq, D, dtype=dtype, device=DEV)
        att.append(x, cache, q4.PagedBatch(cu, kv, table, tokens=2), positions=pos, q_out=q)
        ok_rows[what] = (q[1].cpu(), cache.k.cpu()[int(step.table[1, 0])])
        assert torch.equal(ok_rows[what][0], ok_rows["fine"][0])
        assert torch.equal(torch.nan_to_num(ok_rows[what][1]), torch.nan_to_num(ok_rows["fine"][1]))
        if what == "fine":
            att.device_error()
            continue
        if what != "long":
            assert (q[0] == 0).all()
        with pytest.raises(q4.GPTQ4Error) as e:
            att.device_error()
        assert e.value.status == q4.GPTQ_Q4_DEVICE_FAULT


def test_a_captured_append_outlives_its_rotary_table(q4):
    """set_rope after a capture: another table leaves the graph its own, which nobody else is given; the same sizes
    change the angles of the graph as well."""
    Hq, Hkv, D, page, dtype = 4, 2, 128, 16, torch.float16
    step = Step(q4, [(3, 40), (1, 700)], Hkv, D, page, dtype, seed=16)
    x = torch.randn(step.tokens, Hq + 2 * Hkv, D, generator=torch.Generator().manual_seed(15)).to(dtype)
    xd = x.view(step.tokens, -1).to(DEV)
    pos = torch.tensor([37, 38, 39, 699])
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)

    def right(q, rot, base, interleaved, what):
        ref, tol = rotate_reference(x[:, :Hq], pos, q4.gptq_q4_rope_freqs(rot, base, 0)[0], 1.0, interleaved, dtype)
        assert ((q.double().cpu() - ref).abs() <= tol).all(), what

    att.set_rope(128, 1000)
    q = torch.empty(step.tokens, Hq, D, dtype=dtype, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        att.append(xd, step.cache, step.batch, q_out=q)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            att.append(xd, step.cache, step.batch, q_out=q)
    torch.cuda.synchronize()
    others = []
    for rot, base, interleaved, max_pos in ((128, 10000.0, True, 1000), (64, 500.0, False, 1000), (64, 900.0, False, 1000),
                                            (128, 500000.0, False, 4000), (0, 1.0, False, 0)):
        att.set_rope(rot, max_pos, base=base, interleaved=interleaved)
        others += [torch.full((n,), 77, dtype=torch.int8, device=DEV) for n in [512000] * 6 + [1 << 21] * 2]
        if rot:
            right(att.append(xd, step.cache, step.batch), rot, base, interleaved, (rot, base))
        else:
            assert torch.equal(att.append(xd, step.cache, step.batch).cpu(), x[:, :Hq])
        q.fill_(float("nan"))
        graph.replay()
        right(q, 128, 10000.0, False, "replayed")
    assert all((o == 77).all() for o in others)
    att.device_error()

    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    att.set_rope(128, 1000)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        att.append(xd, step.cache, step.batch, q_out=q)
    att.set_rope(128, 1000, base=300.0)
    graph.replay()
    right(q, 128, 300.0, False, "written anew")
    att.device_error()


@pytest.mark.parametrize("what", ["one_past", "long", "huge", "chunk", "cu_past", "cu_back"])
def test_a_request_past_its_limits_writes_nothing(q4, what):
    """A request that overruns its table, whose last entries are padding on another request's page, or whose rows are
    out of range: neither its pages nor anybody's change, and the other request is served."""
    Hq, Hkv, D, page, dtype = 2, 1, 64, 8, torch.float16
    step = Step(q4, [(4, 16), (2, 21)], Hkv, D, page, dtype, seed=13)
    assert step.table.shape == (2, 3)
    step.table[0, 2] = step.table[1, 0]                   # the first request's padding
    cu, kv, table = (t.clone() for t in (*step.batch.tensors[:2], step.table.to(DEV)))
    good = 0 if what == "cu_past" else 1
    if what == "one_past":                               # 24 tokens fit the table
        kv[0] = 25
    if what == "long":
        kv[0] = 1000
    if what == "huge":
        kv[0] = 2 ** 31 - 1
    if what == "chunk":                                  # its first new tokens would fit, its last would not
        kv[0] = 26
    if what == "cu_past":
        cu[2] = 1000
    if what == "cu_back":                                # the first request's rows begin before the step's
        cu[0] = -7
    x = torch.randn(6, 4 * D, generator=torch.Generator().manual_seed(12)).to(dtype)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    cache = q4.PagedCache(step.k.to(DEV), step.v.to(DEV))
    q = torch.zeros(6, Hq, D, dtype=dtype, device=DEV)
    att.append(x.to(DEV), cache, q4.PagedBatch(cu, kv, table, tokens=6), q_out=q)
    want_k, want_v, want_q = step.k.clone(), step.v.clone(), torch.zeros(6, Hq, D, dtype=dtype)
    heads = x.view(6, 4, D)
    ql, n = step.lens[good]
    for t in range(ql):
        i, row = n - ql + t, step.cu[good] + t
        p = int(step.table[good, i // page])
        want_k[p, :, i % page], want_v[p, :, i % page], want_q[row] = heads[row, 2:3], heads[row, 3:4], heads[row, :2]
    for got, want in ((cache.k, want_k), (cache.v, want_v), (q, want_q)):
        assert torch.equal(torch.nan_to_num(got.cpu(), nan=99.0), torch.nan_to_num(want, nan=99.0))
    with pytest.raises(q4.GPTQ4Error) as e:
        att.device_error()
    assert e.value.status == q4.GPTQ_Q4_DEVICE_FAULT


def test_decode_loop_matches_one_prompt(q4):
    """Appending and attending token by token, or in uneven chunks, gives what one prompt gives."""
    Hq, Hkv, D, page, dtype, n = 8, 2, 128, 16, torch.bfloat16, 200
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    att.set_rope(128, 512)
    qkv = torch.randn(n, (Hq + 2 * Hkv) * D, generator=torch.Generator().manual_seed(10)).to(dtype).to(DEV)
    table = torch.randperm(13, generator=torch.Generator().manual_seed(11)).to(torch.int32)[None].to(DEV)

    def run(chunks):
        cache = q4.PagedCache(*(torch.full((13, Hkv, page, D), float("nan"), dtype=dtype, device=DEV) for _ in "kv"))
        out, at = [], 0
        for c in chunks:
            at += c
            batch = q4.PagedBatch(torch.tensor([0, c], dtype=torch.int32, device=DEV),
                                  torch.tensor([at], dtype=torch.int32, device=DEV), table, tokens=c)
            q = att.append(qkv[at - c:at], cache, batch)
            out.append(att.attend(q, cache, batch))
        return torch.cat(out), cache

    whole, c0 = run([n])
    assert not torch.isnan(whole).any()
    for chunks in ([1] * n, [130, 1, 1, 3, 17, 48], [64, 136]):
        got, c1 = run(chunks)
        assert torch.equal(torch.nan_to_num(c0.k), torch.nan_to_num(c1.k))
        # two results within the tolerance of one value: weights and outputs rounded to bf16, |v| a few
        assert ((got.float() - whole.float()).abs() <= 2 * (2 * U[dtype] + 2.0 ** -12) * 4).all()
    att.device_error()


def test_dimensions_of_one_have_any_stride(q4):
    """One head, one page or one request, cut out of tensors that give such a dimension another stride."""
    D, page, dtype = 64, 16, torch.float16
    g = torch.Generator().manual_seed(19)
    i32 = torch.int32
    new = lambda *s: torch.randn(*s, generator=g).to(dtype).to(DEV)                    # noqa: E731
    att = q4.PagedAttention(1, 1, D, page, dtype=dtype)
    one, lens = torch.tensor([0, 3], dtype=i32, device=DEV), torch.tensor([[13, 1], [9, 1]], dtype=i32, device=DEV)
    q, k, v = new(1, 3, D), new(1, page, 1, D), new(1, page, 1, D)
    dense = q4.PagedCache(k.transpose(1, 2).contiguous(), v.transpose(1, 2).contiguous())
    table = torch.zeros(1, 1, dtype=i32, device=DEV)
    want = att.attend(q[0][:, None].contiguous(), dense, q4.PagedBatch(one, lens[0, :1].contiguous(), table, 3))
    # one key/value head between the tokens and their elements; one page, of keys and values that lie apart
    caches = [q4.PagedCache(k.transpose(1, 2), v.transpose(1, 2)),
              q4.PagedCache(k.transpose(1, 2).as_strided((1, 1, page, D), (8, D, D, 1)),
                            torch.stack([v, v], 1)[:, 1].transpose(1, 2))]
    # one query head; a request's length out of a column, its table's only column out of a row
    batches = [q4.PagedBatch(one, lens[:1, 0], table.expand(7, 1)[:1], 3),
               q4.PagedBatch(one, lens.t()[:1, 0], torch.zeros(1, 9, dtype=i32, device=DEV).t()[:1], 3)]
    for cache in caches:
        for batch in batches:
            assert torch.equal(att.attend(q.transpose(0, 1), cache, batch), want)
    out = torch.zeros(1, 3, D, dtype=dtype, device=DEV)
    att.attend(q.transpose(0, 1), caches[0], batches[0], out=out.transpose(0, 1))
    assert torch.equal(out[0], want[:, 0])
    two = new(3, 2, page, D)
    for a, b in ((two[:, :, :, :32], two[:, :, :, :32]), (two[:, :, ::2], two[:, :, ::2]), (two[::2], two[:2]),
                 (two.transpose(0, 1), two.transpose(0, 1))):
        with pytest.raises(q4.GPTQ4Error):
            q4.PagedCache(a, b)
    att.device_error()


@pytest.mark.parametrize("max_q", [1, 100000])
def test_contexts_without_a_page(q4, max_q):
    """A table of no columns: no row sees anything, and a token has no place to go."""
    Hq, Hkv, D, page, dtype = 4, 2, 64, 16, torch.float16
    i32 = torch.int32
    k = torch.full((2, Hkv, page, D), float("nan"), dtype=dtype, device=DEV)
    cache = q4.PagedCache(k, k.clone())
    batch = q4.PagedBatch(torch.tensor([0, 5, 5, 6], dtype=i32, device=DEV), torch.zeros(3, dtype=i32, device=DEV),
                          torch.empty(3, 0, dtype=i32, device=DEV), tokens=7, max_q=max_q)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    out = torch.full((7, Hq, D), 5.0, dtype=dtype, device=DEV)
    att.attend(torch.ones_like(out), cache, batch, out=out)
    assert (out[:6] == 0).all() and (out[6] == 5).all()
    att.device_error()
    q = torch.full_like(out, 5.0)
    att.append(torch.ones(7, (Hq + 2 * Hkv) * D, dtype=dtype, device=DEV), cache, batch, q_out=q)
    assert (q == 5).all() and torch.isnan(cache.k).all() and torch.isnan(cache.v).all()
    with pytest.raises(q4.GPTQ4Error) as e:
        att.device_error()
    assert e.value.status == q4.GPTQ_Q4_DEVICE_FAULT


def test_results_go_where_they_were_asked_for(q4):
    """Outputs of more dimensions are written in place, or refused where their rows do not lie in a row each (they
    were computed into a copy); inputs of any layout are taken, but not other shapes with as many elements."""
    Hq, Hkv, D, page, dtype = 4, 2, 64, 16, torch.float16
    step = Step(q4, [(2, 30), (4, 9)], Hkv, D, page, dtype, seed=18)
    qkv = torch.randn(6, (Hq + 2 * Hkv) * D, generator=torch.Generator().manual_seed(17)).to(dtype).to(DEV)
    q = qkv[:, :Hq * D].reshape(6, Hq, D)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    att.append(qkv, step.cache, step.batch)
    want = att.attend(q, step.cache, step.batch)
    for shape in ((2, 3, Hq, D), (1, 6, Hq * D // 2, 2), (6, Hq * D)):
        out = torch.full(shape, float("nan"), dtype=dtype, device=DEV)
        assert att.attend(q, step.cache, step.batch, out=out) is out and torch.equal(out.view_as(want), want)
        out.fill_(float("nan"))
        assert att.append(qkv, step.cache, step.batch, q_out=out) is out and torch.equal(out.view_as(q), q)
    apart = torch.zeros(3, 2, Hq, D, dtype=dtype, device=DEV).transpose(0, 1)       # rows in another order
    assert torch.equal(att.attend(apart.copy_(q.view(2, 3, Hq, D)), step.cache, step.batch), want)
    for f in (lambda: att.attend(q, step.cache, step.batch, out=apart),
              lambda: att.append(qkv, step.cache, step.batch, q_out=apart),
              lambda: att.attend(q.view(6, 1, 2 * Hq, D // 2).transpose(2, 3), step.cache, step.batch, out=apart)):
        with pytest.raises(q4.GPTQ4Error) as e:
            f()
        assert e.value.status == q4.GPTQ_Q4_INVALID_ARGUMENT
    for shape in ((3, 2, Hq * D // 3), (12, 1, Hq * D // 2 + 1), (7, 3, 5, 2)):
        with pytest.raises(q4.GPTQ4Error) as e:
            att.append(torch.zeros(shape, dtype=dtype, device=DEV), step.cache, step.batch)
        assert e.value.status == q4.GPTQ_Q4_INVALID_ARGUMENT
    att.device_error()


def test_refusals(q4):
    bad, no = q4.GPTQ_Q4_INVALID_ARGUMENT, q4.GPTQ_Q4_UNSUPPORTED

    def refused(status, f, *args, **kw):
        with pytest.raises(q4.GPTQ4Error) as e:
            f(*args, **kw)
        assert e.value.status == status and e.value.message

    for status, args in ((bad, (0, 1, 64, 16)), (bad, (6, 4, 64, 16)), (bad, (129, 1, 64, 16)), (no, (4, 2, 96, 16)),
                         (no, (4, 2, 64, 12)), (no, (4, 2, 64, 4)), (no, (4, 2, 64, 2048))):
        refused(status, q4.PagedAttention, *args)
    refused(no, q4.PagedAttention, 4, 2, 64, 16, dtype=torch.float32)
    att = q4.PagedAttention(4, 2, 64, 16)
    refused(bad, att.set_rope, 72, 100)
    refused(bad, att.set_rope, 24, 100)
    refused(bad, att.set_rope, 64, 0)
    refused(bad, att.set_rope, 64, 100, base=1.0)
    refused(bad, att.set_rope, 64, 100, scaling="other")
    refused(bad, att.set_rope, 64, 100, scaling="linear", factor=0.5)
    refused(bad, att.set_rope, 64, 100, scaling="bands", factor=2.0, low=4.0, high=1.0)
    h = torch.float16
    z = lambda *s, dtype=h: torch.zeros(*s, dtype=dtype, device=DEV)                 # noqa: E731
    k, v = z(3, 2, 16, 64), z(3, 2, 16, 64)
    refused(bad, q4.PagedCache, k, v[:2])
    refused(bad, q4.PagedCache, k.transpose(1, 2), v.transpose(1, 2))
    refused(bad, q4.PagedCache, k.cpu(), v.cpu())
    i32 = torch.int32
    cu, kv, table = torch.tensor([0, 2], dtype=i32, device=DEV), torch.tensor([5], dtype=i32, device=DEV), z(1, 2, dtype=i32)
    refused(bad, q4.PagedBatch, cu.long(), kv, table, 2)
    refused(bad, q4.PagedBatch, cu, kv, table[0], 2)
    refused(bad, q4.PagedBatch, cu[:1], kv, table, 2)
    cache, batch = q4.PagedCache(k, v), q4.PagedBatch(cu, kv, table, 2)
    q, qkv = z(2, 4, 64), z(2, 8 * 64)
    refused(bad, att.attend, z(3, 4, 64), cache, batch)
    refused(bad, att.attend, q.bfloat16(), cache, batch)
    refused(bad, att.attend, q, q4.PagedCache(k.bfloat16(), v.bfloat16()), batch)
    refused(bad, att.attend, q, q4.PagedCache(z(3, 2, 32, 64), z(3, 2, 32, 64)), batch)
    refused(bad, att.attend, q, cache, batch, window=-1)
    refused(bad, att.attend, q, cache, batch, scale=float("inf"))
    refused(bad, att.attend, z(2, 260)[:, 2:258], cache, batch)
    refused(bad, att.attend, q, cache, q4.PagedBatch(cu, kv, table, -2))
    refused(bad, att.append, z(2, 7 * 64), cache, batch)
    refused(bad, att.append, qkv, cache, batch, positions=z(2, dtype=torch.int64))
    refused(bad, att.append, qkv, cache, batch, q_out=z(2, 4, 32))
    many = 4097
    refused(no, att.attend, z(many, 4, 64), cache,
            q4.PagedBatch(torch.arange(many + 1, dtype=i32, device=DEV), torch.ones(many, dtype=i32, device=DEV),
                          z(many, 1, dtype=i32), many))
    raw, hd, c, b = q4.gptq_q4_attn_attend, att.handle, cache.struct, batch.struct
    refused(bad, raw, None, q.data_ptr(), 256, c, b, 1.0, 0, q.data_ptr(), 256, 0)
    refused(bad, raw, hd, None, 256, c, b, 1.0, 0, q.data_ptr(), 256, 0)
    refused(bad, raw, hd, q.data_ptr(), 248, c, b, 1.0, 0, q.data_ptr(), 256, 0)
    refused(bad, raw, hd, q.data_ptr(), 256, q4.gptq_q4_cache(None, None, 3, 2048), b, 1.0, 0, q.data_ptr(), 256, 0)
    refused(bad, raw, hd, q.data_ptr(), 256, q4.gptq_q4_cache(c.k, c.v, 3, 2040), b, 1.0, 0, q.data_ptr(), 256, 0)
    # a step without requests or tokens is no work
    none = q4.PagedBatch(z(1, dtype=i32), z(0, dtype=i32), z(0, 2, dtype=i32), 0)
    assert att.attend(q[:0], cache, none).shape == (0, 4, 64)
    assert att.append(qkv[:0], cache, none).shape == (0, 4, 64)
    att.device_error()
    att.close()
