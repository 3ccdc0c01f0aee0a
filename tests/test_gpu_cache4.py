"""The paged cache in 4 bits: the append that quantises into it, reading it back, and attention over it, against the
definitions in 64 bits (paged4.py).

An appended code is the definition's, bit for bit, where the rotated key is: the kernel rounds the exact sum of its
products once to fp32 and once to 16 bits, as `x.double() .. .float().to(dtype)` does.  Queries are off by one
rounding, as in test_gpu_attention.py."""
import gc

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from paged4 import DEV, U, Step, attention, check, no_handles_left, quantise, record, refused, values  # noqa: E402, F401

TYPES = pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
GROUPS = pytest.mark.parametrize("group", [32, 64])


@pytest.fixture(scope="module")
def q4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gptq_bit_weight_gb300 as q4mod
    return q4mod


# ------------------------------------------------------------------ append and read

def rotated(x, pos, rot, interleaved, base=10000.0):
    """x [tokens, heads, D] turned by positions pos, from fp32 cosines and sines, exact until the roundings."""
    f = torch.tensor([base ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    angle = pos.double()[:, None] * f
    c, s = angle.cos().float().double()[:, None], angle.sin().float().double()[:, None]
    first = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    second = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    y, a, b = x.clone(), x[..., first].double(), x[..., second].double()
    y[..., first], y[..., second] = (a * c - b * s).float().to(x.dtype), (b * c + a * s).float().to(x.dtype)
    return y


def same_records(got, want, D, dtype):
    """Codes are equal; parameters are equal as numbers (or both NaN)."""
    assert torch.equal(got[..., :D], want[..., :D])
    a, b = (t[..., D:].contiguous().view(dtype).float() for t in (got, want))
    assert torch.equal(torch.nan_to_num(a, nan=1e9), torch.nan_to_num(b, nan=1e9))


APPEND = {
    "single": [(1, 1)],
    "decode": [(1, n) for n in (1, 7, 16, 17, 33, 64, 100)],
    "prompts": [(40, 40), (0, 9), (33, 50), (1, 20)],
    "many": [(37, 37 + i % 50) for i in range(90)],          # several tokens in a block
}


@TYPES
@GROUPS
@pytest.mark.parametrize("rope", [(0, False), (64, False), (64, True), (128, False), (128, True), (32, False)], ids=str)
@pytest.mark.parametrize("lens", list(APPEND), ids=str)
def test_append_and_read(q4, lens, rope, group, dtype):
    rot, interleaved = rope
    Hq, Hkv, D, page = (5, 1, 128, 16) if rot != 32 else (6, 2, 64, 8)
    lens = APPEND[lens]
    step = Step(q4, lens, Hkv, D, page, dtype, group, seed=1, lead=2, tail=3)
    g = torch.Generator().manual_seed(2)
    x = (torch.randn(step.tokens, Hq + 2 * Hkv, D, generator=g) * torch.exp(torch.randn(step.tokens, Hq + 2 * Hkv, 1, generator=g))).to(dtype)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    if rot:
        att.set_rope(rot, 200, interleaved=interleaved)
    before = step.pool.cpu()
    pos = torch.zeros(step.tokens, dtype=torch.int64)
    want = before.clone()
    owner = torch.zeros(step.tokens, dtype=torch.bool)
    for b, (ql, kv) in enumerate(lens):
        pos[step.cu[b]:step.cu[b] + ql] = torch.arange(kv - ql, kv)
        owner[step.cu[b]:step.cu[b] + ql] = True
    y = rotated(x[:, :Hq + Hkv], pos, rot, interleaved) if rot else x[:, :Hq + Hkv]
    k, v = quantise(y[:, Hq:], group), quantise(x[:, Hq + Hkv:], group)
    rec = record(k, v)
    for b, (ql, kv) in enumerate(lens):
        for t in range(ql):
            j = kv - ql + t
            want[int(step.table[b, j // page]), :, j % page] = rec[step.cu[b] + t]
    q = torch.full((step.tokens, Hq, D), 7.0, dtype=dtype, device=DEV)
    xd = x.view(step.tokens, -1).to(DEV)
    att.append(xd, step.cache, step.batch, q_out=q)
    att.device_error()
    same_records(step.pool.cpu(), want, D, dtype)
    near = (q.cpu().double() - y[:, :Hq].double()).abs() <= 2 * U[dtype] * y[:, :Hq].double().abs() + 2.0 ** -22 * x[:, :Hq].double().abs().amax(-1, keepdim=True)
    assert near[owner].all() and (q.cpu()[~owner] == 7).all()
    kr, vr = (torch.full((step.tokens, Hkv, D), 7.0, dtype=dtype, device=DEV) for _ in "kv")
    att.read(step.cache, step.batch, k_out=kr, v_out=vr)
    att.device_error()
    for got, ref in ((kr, values(*k)), (vr, values(*v))):
        assert torch.equal(got.cpu()[owner], ref[owner]) and (got.cpu()[~owner] == 7).all()
    # in place: q_out is qkv itself
    att.append(xd, step.cache, step.batch, q_out=xd[:, :Hq * D])
    assert torch.equal(xd.view(step.tokens, -1, D)[:, :Hq].cpu()[owner], q.cpu()[owner])
    same_records(step.pool.cpu(), want, D, dtype)


@TYPES
def test_append_at_other_positions(q4, dtype):
    """Rotary positions of their own; one past the table is reported, and its token left out."""
    Hq, Hkv, D, page, lens = 4, 2, 128, 16, [(3, 20), (2, 5)]
    step = Step(q4, lens, Hkv, D, page, dtype, 32, seed=15)
    x = torch.randn(5, Hq + 2 * Hkv, D, generator=torch.Generator().manual_seed(16)).to(dtype)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    att.set_rope(D, 500)
    pos = torch.tensor([0, 499, 7, 7, 123], dtype=torch.int32)
    att.append(x.view(5, -1).to(DEV), step.cache, step.batch, positions=pos.to(DEV))
    att.device_error()
    k, v = att.read(step.cache, step.batch)
    want = rotated(x[:, Hq:Hq + Hkv], pos, D, False)
    assert torch.equal(k.cpu(), values(*quantise(want, 32))) and torch.equal(v.cpu(), values(*quantise(x[:, Hq + Hkv:], 32)))
    before = step.pool.clone()
    pos[2] = 500
    q = torch.full((5, Hq, D), 7.0, dtype=dtype, device=DEV)
    att.append(-x.view(5, -1).to(DEV), step.cache, step.batch, positions=pos.to(DEV), q_out=q)
    assert refused(q4, att.device_error)
    assert (q[2] == 7).all() and not (q[1] == 7).all()
    p, slot = int(step.table[0, 19 // page]), 19 % page
    assert torch.equal(step.pool[p, :, slot], before[p, :, slot]) and not torch.equal(step.pool[p, :, slot - 1], before[p, :, slot - 1])


def test_two_captured_graphs_of_one_handle(q4):
    """They share the handle's workspace, one after the other, beside calls outside."""
    Hq, Hkv, D, page, dtype = 8, 1, 128, 16, torch.bfloat16
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    steps = [Step(q4, lens, Hkv, D, page, dtype, group, seed=17) for lens, group in (([(1, 9000), (1, 300)], 32), ([(60, 5000)], 64), ([(1, 7000)], None))]
    g = torch.Generator().manual_seed(18)
    qs = [torch.randn(s.tokens, Hq, D, generator=g).to(dtype).to(DEV) for s in steps]
    want = [att.attend(q, s.cache, s.batch, window=4000, sinks=9).clone() for q, s in zip(qs, steps)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    gc.collect()
    with torch.cuda.stream(side):
        for q, s in zip(qs, steps):
            torch.cuda.synchronize()
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=side):
                outs.append(att.attend(q, s.cache, s.batch, window=4000, sinks=9))
        for i in (0, 1, 2, 1, 0, 2, 2):
            graphs[i].replay()
            again = att.attend(qs[2 - i], steps[2 - i].cache, steps[2 - i].batch, window=4000, sinks=9)
            assert torch.equal(outs[i], want[i]) and torch.equal(again, want[2 - i])
    torch.cuda.synchronize()
    att.device_error()


@TYPES
@GROUPS
def test_append_of_extreme_values(q4, group, dtype):
    """Constant groups, subnormal and largest steps, borders between codes, infinities and NaN, -0; each group by itself."""
    Hq, Hkv, D, page = 1, 1, 128, 8
    big = torch.finfo(dtype).max
    tiny = 2.0 ** -24 if dtype == torch.float16 else 2.0 ** -133
    rows = [torch.zeros(D), torch.full((D,), -0.0), torch.full((D,), 3.25), torch.linspace(-1, 1, D),
            torch.arange(D) % 16 * 1.0, torch.arange(D) % 31 * 0.5, torch.arange(D) % 16 * tiny, torch.arange(D) % 4 * tiny,
            torch.where(torch.arange(D) % 2 == 0, big, 0.0), torch.where(torch.arange(D) % 2 == 0, big, -big) * 0.5,
            torch.where(torch.arange(D) == 5, float("inf"), 1.0), torch.where(torch.arange(D) == 70, float("nan"), 2.0),
            torch.where(torch.arange(D) == 127, -float("inf"), -1.0), 1e3 + torch.linspace(0, 1, D),
            torch.where(torch.arange(D) % 2 == 0, big, -big)]
    T = len(rows)
    g = torch.Generator().manual_seed(3)
    kv = torch.stack(rows).to(dtype)
    x = torch.stack([torch.randn(T, D, generator=g).to(dtype), kv, kv.flip(0)], 1)
    step = Step(q4, [(T, T)], Hkv, D, page, dtype, group, seed=4)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    att.append(x.view(T, -1).to(DEV), step.cache, step.batch)
    k, v = att.read(step.cache, step.batch)
    att.device_error()
    kc, vc = quantise(x[:, 1:2], group), quantise(x[:, 2:3], group)
    rec = record(kc, vc)
    got = torch.stack([step.pool.cpu()[int(step.table[0, t // page]), :, t % page] for t in range(T)])
    same_records(got, rec, D, dtype)
    for a, b in ((k, values(*kc)), (v, values(*vc))):
        assert torch.equal(torch.nan_to_num(a.cpu().float(), nan=1e9), torch.nan_to_num(b.float(), nan=1e9))


@GROUPS
def test_quantisation_error_is_half_a_step(q4, group):
    """What comes back is within half a step, the rounding of the step (15 codes of it) and that of the value."""
    Hq, Hkv, D, page, dtype = 2, 2, 128, 16, torch.float16
    step = Step(q4, [(50, 50)], Hkv, D, page, dtype, group, seed=5)
    x = torch.randn(50, Hq + 2 * Hkv, D, generator=torch.Generator().manual_seed(6)).to(dtype)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    att.append(x.view(50, -1).to(DEV), step.cache, step.batch)
    for got, want in zip(att.read(step.cache, step.batch), (x[:, 2:4], x[:, 4:])):
        y = want.double().unflatten(-1, (-1, group))
        s = (y.amax(-1) - y.amin(-1)) / 15
        err = (got.cpu().double() - want.double()).abs().unflatten(-1, (-1, group))
        assert (err <= (0.5 + 16 * U[dtype]) * s[..., None] + U[dtype] * (y.abs() + s[..., None])).all()


@pytest.mark.parametrize("page", [8, 16, 256])
@TYPES
def test_read_of_the_16_bit_cache(q4, page, dtype):
    """Whole contexts, in another order than their pages', into columns of wider rows."""
    lens = [(n, n) for n in (1, 40, 0, 17, 300)]
    step = Step(q4, lens, 3, 64, page, dtype, seed=7, lead=1, tail=2)
    att = q4.PagedAttention(6, 3, 64, page, dtype=dtype)
    wide = torch.full((step.tokens, 2 * 3 * 64 + 16), 7.0, dtype=dtype, device=DEV)
    att.read(step.cache, step.batch, k_out=wide[:, 8:200], v_out=wide[:, 200:392])
    att.device_error()
    w = wide.cpu()
    for b, (ql, _) in enumerate(lens):
        rows = w[step.cu[b]:step.cu[b] + ql]
        assert torch.equal(rows[:, 8:200], step.keys[b].reshape(ql, 192)) and torch.equal(rows[:, 200:392], step.values[b].reshape(ql, 192))
    assert (w[0] == 7).all() and (w[-2:] == 7).all() and (w[:, :8] == 7).all() and (w[:, 392:] == 7).all()


# ------------------------------------------------------------------ attention

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
SHAPES = [  # Hq, Hkv, D, page, group
    (4, 4, 128, 16, 32),
    (16, 2, 128, 32, 64),
    (6, 2, 64, 8, 32),
    (5, 1, 128, 64, 32),
    (8, 1, 64, 128, 64),
    (20, 1, 128, 16, 64),
    (48, 1, 64, 32, 32),
    (128, 1, 128, 256, 32),
    (3, 3, 64, 512, 64),
]


@TYPES
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("lens", list(LENS), ids=str)
def test_attend(q4, lens, shape, dtype):
    Hq, Hkv, D, page, group = shape
    if Hq * max(ql for ql, _ in LENS[lens]) > 9000:
        pytest.skip("the same tiles as the smaller head counts")
    step = Step(q4, LENS[lens], Hkv, D, page, dtype, group, seed=Hq + page, lead=2, tail=3)
    q = (torch.randn(step.tokens, Hq, D, generator=torch.Generator().manual_seed(1)) * 2).to(dtype)
    ref, tol = attention(step, q, D ** -0.5)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    qd = q.to(DEV)
    for batch in (step.batch, step.make_batch(q4, 100000)):          # max_q chooses the kernel
        out = torch.full_like(qd, float("nan"))
        att.attend(qd, step.cache, batch, out=out)
        check(out, ref, tol, f"max_q {batch.struct.max_q}")
        assert torch.isnan(out.cpu()[torch.isnan(ref)]).all()        # rows of no request are left alone
        again = torch.full_like(qd, float("nan"))
        att.attend(qd, step.cache, batch, out=again)
        assert torch.equal(torch.nan_to_num(out), torch.nan_to_num(again))
    att.device_error()


WINDOWS = [(1, 0), (1, 1), (16, 4), (100, 16), (257, 130), (100, 1000), (64, 2 ** 31 - 1), (2 ** 31 - 1, 5)]


@TYPES
@pytest.mark.parametrize("max_q", [None, 100000])
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("shape", [(4, 4, 128, 16, 32), (16, 2, 64, 32, 32), (10, 2, 128, 64, 64), (2, 1, 64, 8, 64), (8, 8, 128, 16, None),
                                   (16, 2, 64, 32, None), (10, 2, 128, 64, None), (3, 1, 64, 256, None)],
                         ids=lambda s: "x".join(map(str, s)))
def test_window_and_sinks(q4, shape, window, sinks, max_q, dtype):
    """Both caches; pages between the first tokens and the window are not there any more."""
    Hq, Hkv, D, page, group = shape
    step = Step(q4, [(1, 500), (1, 30), (3, 400), (140, 350), (150, 150), (4, 2), (1, 1000), (2, 129)], Hkv, D, page, dtype, group,
                seed=3, window=window, sinks=sinks)
    q = (torch.randn(step.tokens, Hq, D, generator=torch.Generator().manual_seed(2)) * 2).to(dtype)
    ref, tol = attention(step, q, D ** -0.5, window, sinks)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    batch = step.batch if max_q is None else step.make_batch(q4, max_q)
    check(att.attend(q.to(DEV), step.cache, batch, window=window, sinks=sinks), ref, tol, f"window {window}, sinks {sinks}")
    att.device_error()


@pytest.mark.parametrize("group", [32, None])
@pytest.mark.parametrize("max_q", [1, 100000])
def test_sinks_without_a_window_are_plain_attention(q4, max_q, group):
    Hq, Hkv, D, page, dtype = 8, 2, 128, 16, torch.bfloat16
    step = Step(q4, [(1, 300), (20, 400)], Hkv, D, page, dtype, group, seed=8)
    q = torch.randn(step.tokens, Hq, D, generator=torch.Generator().manual_seed(9)).to(dtype).to(DEV)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    batch = step.make_batch(q4, max_q)
    assert torch.equal(att.attend(q, step.cache, batch, sinks=7), att.attend(q, step.cache, batch))
    att.device_error()


@pytest.mark.parametrize("group", [32, 64, None])
@pytest.mark.parametrize("lens", [[(1, 400), (1, 70)], [(140, 400), (1, 70)]], ids=["tokens", "chunk"])
def test_strided_rows_scale_and_stream(q4, lens, group):
    """q and out as columns of wider rows, another scale, on a side stream; also a scale below zero."""
    Hq, Hkv, D, page, dtype = 8, 2, 128, 16, torch.bfloat16
    step = Step(q4, lens, Hkv, D, page, dtype, group, seed=4)
    wide = torch.randn(step.tokens, Hq * D + 264, generator=torch.Generator().manual_seed(3)).to(dtype)
    q = wide[:, 8:8 + Hq * D].reshape(-1, Hq, D)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    wd = wide.to(DEV)
    for scale in (0.2, -0.1, 0.0):
        ref, tol = attention(step, q, scale, 100, 20)
        out = torch.full((step.tokens, Hq * D + 64), 7.0, dtype=dtype, device=DEV)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            att.attend(wd[:, 8:8 + Hq * D], step.cache, step.batch, scale=scale, out=out[:, 16:16 + Hq * D], window=100, sinks=20)
        side.synchronize()
        check(out[:, 16:16 + Hq * D].reshape(-1, Hq, D), ref, tol, f"strided, scale {scale}")
        assert (out[:, :16] == 7).all() and (out[:, 16 + Hq * D:] == 7).all()
    att.device_error()


@pytest.mark.parametrize("group", [32, None])
@pytest.mark.parametrize("max_q", [1, 100000])
def test_cache_past_32_bit_offsets(q4, max_q, group):
    """Pages that begin more than 2^32 bytes into the cache."""
    Hq, Hkv, D, page, dtype = 8, 2, 128, 16, torch.float16
    step = Step(q4, [(1, 100), (1, 37)], Hkv, D, page, dtype, group, seed=7)
    q = torch.randn(step.tokens, Hq, D, generator=torch.Generator().manual_seed(4)).to(dtype)
    ref, tol = attention(step, q, D ** -0.5, 50, 3)
    stride = 1 << 29
    if group:
        n, *rest = step.pool.shape
        far = torch.empty((n - 1) * stride + step.pool[0].numel(), dtype=torch.uint8, device=DEV)
        kv = far.as_strided(step.pool.shape, (stride, *step.pool.stride()[1:]))
        kv.copy_(step.pool)
        cache = q4.PagedCache4(kv, D, group, dtype)
    else:
        n = step.pool.shape[1]
        k, v = (torch.empty((n - 1) * (stride // 2) + step.pool[0, 0].numel(), dtype=dtype, device=DEV)
                .as_strided(step.pool.shape[1:], (stride // 2, *step.pool.stride()[2:])) for _ in "kv")
        k.copy_(step.pool[0]), v.copy_(step.pool[1])
        cache = q4.PagedCache(k, v)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    batch = step.make_batch(q4, max_q)
    check(att.attend(q.to(DEV), cache, batch, window=50, sinks=3), ref, tol, "large offsets")
    kr, _ = att.read(cache, batch)
    assert torch.equal(kr.cpu()[0], step.keys[0][-1])
    x = torch.randn(2, (Hq + 2 * Hkv) * D, generator=torch.Generator().manual_seed(5)).to(dtype).to(DEV)
    att.append(x, cache, batch)
    vr = att.read(cache, batch)[1].cpu()
    want = x.view(2, -1, D)[:, Hq + Hkv:].cpu()
    assert torch.equal(vr, values(*quantise(want, group)) if group else want)
    att.device_error()


@pytest.mark.parametrize("group", [64, None])
def test_many_requests(q4, group):
    """More requests than a block has threads, most of them tiny."""
    Hq, Hkv, D, page, dtype = 4, 2, 64, 8, torch.float16
    g = torch.Generator().manual_seed(8)
    lens = [(int(a), int(a) + int(b)) for a, b in zip(torch.randint(0, 3, (1500,), generator=g), torch.randint(0, 40, (1500,), generator=g))]
    step = Step(q4, lens, Hkv, D, page, dtype, group, seed=8, window=9, sinks=4)
    q = torch.randn(step.tokens, Hq, D, generator=g).to(dtype)
    ref, tol = attention(step, q, D ** -0.5, 9, 4)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    for max_q in (2, 100000):
        check(att.attend(q.to(DEV), step.cache, step.make_batch(q4, max_q), window=9, sinks=4), ref, tol, "many requests")
    att.device_error()


@TYPES
@pytest.mark.parametrize("group", [32, 64, None])
@pytest.mark.parametrize("max_q", [1, 3, 100000])
def test_long_contexts(q4, max_q, group, dtype):
    """A CTA goes through many key tiles of an item, and items are cut between CTAs."""
    Hq, Hkv, D, page = 8, 1, 128, 64
    step = Step(q4, [(1, 30000), (3, 9000), (2, 20011)], Hkv, D, page, dtype, group, seed=9)
    q = torch.randn(step.tokens, Hq, D, generator=torch.Generator().manual_seed(10)).to(dtype)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    for window, sinks in ((0, 0), (7000, 300)):
        ref, tol = attention(step, q, D ** -0.5, window, sinks)
        check(att.attend(q.to(DEV), step.cache, step.make_batch(q4, max_q), window=window, sinks=sinks), ref, tol, f"window {window}")
    att.device_error()


@TYPES
@pytest.mark.parametrize("group", [32, None])
@pytest.mark.parametrize("max_q", [1, 100000])
def test_extreme_scores(q4, max_q, group, dtype):
    """Scores that rise along the context, fall, and are all equal, with the sinks' far above and far below the window's."""
    Hq, Hkv, D, page, kv = 4, 1, 128, 16, 900
    step = Step(q4, [(2, kv)], Hkv, D, page, dtype, group, seed=11)
    ramp = torch.linspace(-1, 1, kv)[:, None, None] + 0.02 * torch.randn(kv, Hkv, D, generator=torch.Generator().manual_seed(12))
    ramp[:5] = torch.tensor([5.0, -5.0, 3.0, 0.0, 5.0])[:, None, None]
    k, v = ramp.to(dtype), step.values[0]
    if group:
        kc, vc = quantise(k, group), quantise(v, group)
        k, v, rec = values(*kc), values(*vc), record(kc, vc)
    step.keys[0], step.values[0] = k, v
    for j in range(kv):
        p = int(step.table[0, j // page])
        if group:
            step.pool[p, :, j % page] = rec[j].to(DEV)
        else:
            step.pool[0, p, :, j % page] = k[j].to(DEV)
    q = torch.full((2, Hq, D), 3.0).to(dtype)
    q[:, 1], q[:, 2] = -3.0, 0.0
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    for window, sinks in ((0, 0), (500, 3), (300, 5)):
        ref, tol = attention(step, q, 1.0, window, sinks)
        check(att.attend(q.to(DEV), step.cache, step.make_batch(q4, max_q), scale=1.0, window=window, sinks=sinks), ref, tol, f"{window}, {sinks}")
    att.device_error()


@pytest.mark.parametrize("group", [32, None])
@pytest.mark.parametrize("max_q", [1, 100000])
@pytest.mark.parametrize("D", [64, 128])
def test_values_without_number(q4, D, max_q, group):
    """A NaN in hidden tokens (between sinks and window) reaches no row of a single token; one that is seen reaches its
    head and request only; rows that see nothing are zeros."""
    Hq, Hkv, page, dtype = 2, 2, 16, torch.float16
    lens = [(1, 500), (1, 400), (9, 4)]
    step = Step(q4, lens, Hkv, D, page, dtype, group, seed=20)
    q = torch.randn(step.tokens, Hq, D, generator=torch.Generator().manual_seed(18)).to(dtype)
    ref, tol = attention(step, q, D ** -0.5, 100, 10)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)

    def spoil(b, at, head):
        p = int(step.table[b, at // page])
        if group:
            step.pool[p, head, at % page] = 255
        else:
            step.pool[:, p, head, at % page] = float("nan")
    for at in (10, 15, 16, 200, 399, 400 - 1):
        spoil(0, at, 0)
    batch = step.make_batch(q4, max_q)
    check(att.attend(q.to(DEV), step.cache, batch, window=100, sinks=10), ref, tol, "hidden")
    spoil(0, 9, 0), spoil(1, 300, 1)
    out = att.attend(q.to(DEV), step.cache, batch, window=100, sinks=10).cpu()
    assert torch.isnan(out[0, 0]).all() and torch.isnan(out[1, 1]).all()
    ref[0, 0], ref[1, 1] = float("nan"), float("nan")
    check(out, ref, tol, "seen")
    assert (out[2:7] == 0).all()
    att.device_error()


@pytest.mark.parametrize("group", [32, None])
@pytest.mark.parametrize("max_q", [1, 100000])
def test_bad_batches_are_reported(q4, max_q, group):
    """Bad device data ends in a status, leaves the other requests right and writes nothing for the bad one."""
    Hq, Hkv, D, page, dtype = 4, 2, 128, 16, torch.float16
    step = Step(q4, [(1, 100), (1, 50)], Hkv, D, page, dtype, group, seed=9)
    q = torch.randn(step.tokens, Hq, D, generator=torch.Generator().manual_seed(5)).to(dtype)
    ref, tol = attention(step, q, D ** -0.5, 40, 4)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    x = torch.randn(2, (Hq + 2 * Hkv) * D, generator=torch.Generator().manual_seed(6)).to(dtype).to(DEV)
    good = step.table.clone()
    for change in ("page", "negative", "length"):
        step.table = good.clone()
        lens = list(step.lens)
        if change == "page":
            step.table[0, 6] = 10 ** 6
        elif change == "negative":
            step.table[0, 6] = -7
        else:
            step.lens = [(1, 10 ** 6), (1, 50)]
        batch = step.make_batch(q4, max_q)
        step.lens = lens
        out = att.attend(q.to(DEV), step.cache, batch, window=40, sinks=4)
        assert refused(q4, att.device_error, q4.GPTQ_Q4_DEVICE_FAULT)
        check(out[1:], ref[1:], tol[1:], "the other request")
        att.device_error()
        before = step.pool.clone()
        kr, vr = (torch.full((2, Hkv, D), 7.0, dtype=dtype, device=DEV) for _ in "kv")
        att.read(step.cache, batch, k_out=kr, v_out=vr)
        assert refused(q4, att.device_error)
        assert (kr[0] == 7).all() and torch.equal(kr[1].cpu(), step.keys[1][-1])
        att.append(x, step.cache, batch)
        assert refused(q4, att.device_error)
        changed = (step.pool != before) & ~(torch.isnan(step.pool) & torch.isnan(before)) if group is None else step.pool != before
        where = changed.reshape(-1, *changed.shape[-4:]).any(0).flatten(1).any(1).nonzero().flatten().tolist()
        assert where == [int(good[1, 3])]
        step.pool.copy_(before)


@pytest.mark.parametrize("group", [32, 64, None])
def test_captured_step(q4, group):
    """A decode step in a graph: lengths grow on the GPU, the new token is appended and attended."""
    Hq, Hkv, D, page, dtype = 8, 2, 128, 16, torch.float16
    lens = [(1, 30), (1, 61)]
    step = Step(q4, [(1, 80), (1, 111)], Hkv, D, page, dtype, group, seed=13)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    att.set_rope(D, 4096)
    kv = torch.tensor([n for _, n in lens], dtype=torch.int32, device=DEV)
    batch = q4.PagedBatch(torch.arange(3, dtype=torch.int32, device=DEV), kv, step.table.to(DEV), tokens=2, max_q=1)
    x = torch.randn(2, (Hq + 2 * Hkv) * D, generator=torch.Generator().manual_seed(14)).to(dtype).to(DEV)

    def one():
        kv.add_(1)
        return att.attend(att.append(x, step.cache, batch), step.cache, batch, window=50, sinks=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gc.collect()
    with torch.cuda.stream(side):
        one()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            out = one()
        for _ in range(40):
            graph.replay()
    torch.cuda.synchronize()
    got, pool = out.clone(), step.pool.clone()
    kv.copy_(torch.tensor([n for _, n in lens], dtype=torch.int32))
    for _ in range(41):
        want = one()
    assert torch.equal(got, want) and torch.equal(torch.nan_to_num(pool.float()), torch.nan_to_num(step.pool.float()))
    att.device_error()
