"""The adapter pool against the definition in 64 bits.

Tolerance of an output: one rounding of the result to 16 bits (u |ref|, u the
type's unit roundoff), plus, on S = scale sum_r (sum_k |x a|) |b|: 2^-16 for the
sums x . A^T being carried as two 16-bit parts, and 4 sqrt(K + rank) 2^-23 for
fp32 sums (each step off by at most 2^-23 of a partial sum, errors of either
sign)."""
import numpy as np
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


def adapters(g, ranks, K, N, dtype, std=0.3):
    out = []
    for r in ranks:
        a = (torch.randn(r, K, generator=g) * K ** -0.5).to(dtype)
        b = (torch.randn(N, r, generator=g) * std).to(dtype)
        out.append((a, b, 0.5 + 0.25 * len(out)))
    return out


def reference(x, y, rows, ads, K):
    """(result, tolerance) in 64 bits."""
    ref, S = y.double().clone(), torch.zeros(y.shape, dtype=torch.float64)
    n = torch.ones(y.shape[0], 1, dtype=torch.float64)
    for s, (a, b, scale) in enumerate(ads):
        m = rows == s
        if not m.any() or not a.shape[0]:
            continue
        xd, ad, bd = x[m].double(), a.double(), b.double()
        ref[m] += scale * (xd @ ad.t()) @ bd.t()
        S[m] = scale * (xd.abs() @ ad.abs().t()) @ bd.abs().t()
        n[m] = K + a.shape[0]
    dt = y.dtype
    return ref, U[dt] * ref.abs() + TINY[dt] + (2.0 ** -16 + 4 * n.sqrt() * 2.0 ** -23) * (S + y.double().abs())


def check(got, ref, tol, what):
    err = (got.double().cpu() - ref).abs()
    if not err.numel():
        return
    worst = float((err / tol.clamp(min=1e-300)).max())
    assert bool((err <= tol).all()), f"{what}: worst error / tolerance {worst:.3f}"


def pool_of(q4, ads, K, N, slots, max_rank, dtype):
    pool = q4.LoraPool(K, N, slots, max_rank, dtype=dtype)
    for s, (a, b, scale) in enumerate(ads):
        if a.shape[0]:
            pool.set(s, a.to(DEV), b.to(DEV), scale)
    return pool


CASES = [  # (M, K, N, ranks, rows: "one", "mixed", "runs")
    (1, 8, 8, [1], "one"),
    (1, 256, 512, [16], "one"),
    (3, 64, 72, [4, 9], "mixed"),
    (16, 512, 264, [8, 16, 17, 64], "mixed"),
    (17, 520, 1000, [8, 16, 17, 64], "mixed"),
    (64, 1024, 640, [16] * 20, "mixed"),
    (65, 328, 2056, [33, 48, 5], "mixed"),
    (200, 4096, 256, [64, 8, 32, 1], "mixed"),
    (257, 256, 1288, [64, 128], "runs"),
    (600, 1032, 520, [64, 8, 0, 16], "runs"),
    (1031, 2048, 776, [32], "one"),
    (1500, 200, 136, [16, 64, 40, 8, 24], "runs"),
    (300, 192, 200, [256, 200], "runs"),
    (130, 456, 392, [16] * 24, "mixed"),
    (128, 64, 64, [64], "one"),
    (1280, 64, 24576, [16, 8], "runs"),      # a dozen column tiles for each SM
    (513, 4104, 1160, [128, 16, 100], "mixed"),
    (1, 1000, 1288, [16], "one"),            # one row of a small adapter: one launch
    (1, 2056, 328, [40], "one"),
    (1, 96, 4104, [24, 5], "mixed"),
    (1, 2048, 264, [256], "one"),
    (1, 8, 40968, [100], "one"),
    (1, 4096, 512, [256], "one"),            # and of a larger one: two
    (4, 1000, 1288, [16] * 10, "mixed"),
    (16, 4096, 512, [33, 16, 64], "mixed"),
    (256, 512, 392, [16, 5, 64, 33] * 8, "mixed"),
    (255, 1024, 264, [48], "one"),
    (256, 1024, 8200, [16, 5, 64, 33] * 6, "mixed"),   # one chunk of many adapters
    (290, 8192, 2056, [64, 8, 33, 16] * 5, "runs"),    # two; more rows of an adapter than a unit takes
    (133, 2048, 14344, [64] * 64, "mixed"),
    (320, 328, 520, [16, 40, 64], "runs"),
    (70, 64, 64, [8] * 70, "mixed"),
    (700, 256, 264, [200, 16, 256], "mixed"),          # ranks too high for the tiles
    (700, 264, 520, [64, 16, 33] * 8, "mixed"),        # each tile has too many adapters
    (9000, 64, 72, [64, 16, 33] * 8, "mixed"),         # more tiles than a warp looks at together
]


def row_slots(g, M, n, kind):
    if kind == "one":
        return torch.zeros(M, dtype=torch.int32)
    if kind == "mixed":
        return torch.randint(-1, n, (M,), generator=g, dtype=torch.int32)
    rows = torch.empty(M, dtype=torch.int32)
    at = 0
    while at < M:
        k = int(torch.randint(1, max(2, M // 4), (1,), generator=g))
        rows[at:at + k] = int(torch.randint(-1, n, (1,), generator=g))
        at += k
    return rows


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("M,K,N,ranks,kind", CASES)
def test_matches_definition(q4, M, K, N, ranks, kind, dtype):
    g = torch.Generator().manual_seed(M * 7919 + K + N)
    ads = adapters(g, ranks, K, N, dtype)
    rows = row_slots(g, M, len(ranks), kind)
    x, y = torch.randn(M, K, generator=g).to(dtype), torch.randn(M, N, generator=g).to(dtype)
    pool = pool_of(q4, ads, K, N, len(ranks) + 1, max(ranks), dtype)
    ref, tol = reference(x, y, rows, ads, K)
    xd, yd, rd = x.to(DEV), y.to(DEV), rows.to(DEV)
    out = pool.add(xd, rd, yd)
    again = pool.add(xd, rd, yd)
    check(out, ref, tol, "out of place")
    assert torch.equal(out, again)                       # the same call gives the same bits
    assert torch.equal(yd.cpu(), y) and torch.equal(xd.cpu(), x)
    none = (rows < 0).nonzero().flatten()
    assert torch.equal(out.cpu()[none], y[none])         # a row without an adapter is y itself
    pool.add(xd, rd, yd, out=yd)
    assert torch.equal(yd, out)                          # in place: the same
    pool.device_error()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
def test_a_prompt_beside_single_tokens(q4, dtype):
    """Tiles of one adapter and tiles of many in one call, the rows of both kinds in one tile among them."""
    K, N, M = 520, 1032, 1700
    g = torch.Generator().manual_seed(15)
    ads = adapters(g, [64, 40, 16, 64] * 6, K, N, dtype)
    rows = torch.full((M,), 3, dtype=torch.int32)
    rows[200:500] = torch.randint(-1, 24, (300,), generator=g, dtype=torch.int32)
    rows[1300:] = torch.randint(-1, 24, (400,), generator=g, dtype=torch.int32)
    x, y = torch.randn(M, K, generator=g).to(dtype), torch.randn(M, N, generator=g).to(dtype)
    pool = pool_of(q4, ads, K, N, 24, 64, dtype)
    ref, tol = reference(x, y, rows, ads, K)
    xd, yd, rd = x.to(DEV), y.to(DEV), rows.to(DEV)
    out = pool.add(xd, rd, yd)
    check(out, ref, tol, "out of place")
    assert torch.equal(out, pool.add(xd, rd, yd))
    assert torch.equal(out.cpu()[rows < 0], y[rows < 0])
    pool.add(xd, rd, yd, out=yd)
    assert torch.equal(yd, out)
    pool.device_error()


@pytest.mark.parametrize("ranks", [[96] * 5, [64] * 8, [112, 97, 100, 128], [176, 161], [16] * 32, [48] * 10],
                         ids=lambda r: f"{len(r)}x{max(r)}")
def test_tiles_that_take_passes(q4, ranks):
    """Rows of a pool that is served by passes over a tile's output mix all its adapters; then some of those have no
    number in B, which takes a pass for each."""
    K, N, M, dtype = 264, 392, 700, torch.float16
    assert len(ranks) * ((max(ranks) + 15) // 16 * 16) <= 512
    g = torch.Generator().manual_seed(19)
    ads = adapters(g, ranks, K, N, dtype)
    rows = torch.randint(-1, len(ranks), (M,), generator=g, dtype=torch.int32)
    x, y = torch.randn(M, K, generator=g).to(dtype), torch.randn(M, N, generator=g).to(dtype)
    ref, tol = reference(x, y, rows, ads, K)
    xd, yd, rd = x.to(DEV), y.to(DEV), rows.to(DEV)
    pool = pool_of(q4, ads, K, N, len(ranks), max(ranks), dtype)
    out = pool.add(xd, rd, yd)
    check(out, ref, tol, "mixed")
    assert torch.equal(pool.add(xd, rd, yd, out=yd.clone()), out)
    broken = list(range(0, len(ranks), 2))
    for s in broken:
        ads[s][1][5, 1] = float("nan")
        pool.set(s, ads[s][0].to(DEV), ads[s][1].to(DEV), ads[s][2])
    out = pool.add(xd, rd, yd).cpu()
    whole = ~torch.isin(rows, torch.tensor(broken, dtype=torch.int32))
    check(out[whole], ref[whole], tol[whole], "beside broken adapters")
    fine = torch.arange(N) != 5
    check(out[:, fine], ref[:, fine], tol[:, fine], "their other columns")
    assert torch.isnan(out[~whole][:, 5]).all()
    pool.device_error()


@pytest.mark.parametrize("M", [2, 40, 300])
def test_strided_columns_of_a_fused_projection(q4, M):
    """One part of a fused projection: columns of a wider y, x a view of wider rows, on a side stream."""
    K, N, lead, wide = 192, 136, 64, 416
    dtype = torch.bfloat16
    g = torch.Generator().manual_seed(5)
    ads = adapters(g, [16, 40], K, N, dtype)
    rows = row_slots(g, M, 2, "mixed")
    x, y = torch.randn(M, K + 40, generator=g).to(dtype), torch.randn(M, wide, generator=g).to(dtype)
    pool = pool_of(q4, ads, K, N, 2, 40, dtype)
    ref, tol = reference(x[:, 8:8 + K], y[:, lead:lead + N], rows, ads, K)
    xd, yd, rd = x.to(DEV), y.to(DEV), rows.to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        view = yd[:, lead:lead + N]
        pool.add(xd[:, 8:8 + K], rd, view, out=view)
    side.synchronize()
    check(yd[:, lead:lead + N], ref, tol, "columns")
    assert torch.equal(yd[:, :lead].cpu(), y[:, :lead]) and torch.equal(yd[:, lead + N:].cpu(), y[:, lead + N:])


def test_slots_are_replaced_and_cleared(q4):
    K, N, dtype = 256, 320, torch.float16
    g = torch.Generator().manual_seed(8)
    ads = adapters(g, [64, 3, 16], K, N, dtype)
    x, y = torch.randn(20, K, generator=g).to(dtype), torch.randn(20, N, generator=g).to(dtype)
    rows = torch.zeros(20, dtype=torch.int32)
    xd, yd, rd = x.to(DEV), y.to(DEV), rows.to(DEV)
    pool = q4.LoraPool(K, N, 2, 64, dtype=dtype)
    assert torch.equal(pool.add(xd, rd, yd), yd)         # an empty slot
    for a, b, scale in ads:                              # a smaller rank leaves nothing of the last one
        pool.set(0, a.to(DEV), b.to(DEV), scale)
        ref, tol = reference(x, y, rows, [(a, b, scale)], K)
        check(pool.add(xd, rd, yd), ref, tol, f"rank {a.shape[0]}")
    pool.clear(0)
    assert torch.equal(pool.add(xd, rd, yd), yd)
    assert pool.add(xd[:0], rd[:0], yd[:0]).shape == (0, N)
    pool.device_error()


@pytest.mark.parametrize("M", [5, 400])
def test_large_sums_and_foreign_nan(q4, M):
    """x . A^T past fp16's range with a small B, and NaN or infinity in one row that reach no other row."""
    K, N, dtype = 512, 264, torch.float16
    g = torch.Generator().manual_seed(9)
    a = torch.full((16, K), 8.0).to(dtype) + torch.randn(16, K, generator=g).to(dtype)
    b = (torch.randn(N, 16, generator=g) * 2e-5).to(dtype)
    x = (torch.randn(M, K, generator=g).abs() * 60).to(dtype)           # sums about 2e5
    y = torch.randn(M, N, generator=g).to(dtype)
    rows = torch.zeros(M, dtype=torch.int32)
    pool = pool_of(q4, [(a, b, 1.0)], K, N, 1, 16, dtype)
    ref, tol = reference(x, y, rows, [(a, b, 1.0)], K)
    check(pool.add(x.to(DEV), rows.to(DEV), y.to(DEV)), ref, tol, "large sums")
    x[1], x[3] = float("nan"), float("inf")
    out = pool.add(x.to(DEV), rows.to(DEV), y.to(DEV)).cpu()
    clean = torch.tensor([i for i in range(M) if i not in (1, 3)])
    check(out[clean], ref[clean], tol[clean], "beside NaN")
    assert not torch.isfinite(out[1]).any() and not torch.isfinite(out[3]).any()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("M", [3, 400])
def test_an_infinity_keeps_its_sign(q4, M, dtype):
    """An adapter of rank 1, stored with 15 ranks of zeros beside it: infinity in x times those is NaN."""
    K, N = 128, 264
    g = torch.Generator().manual_seed(14)
    away = lambda *n: (lambda t: (t.sign() * (t.abs() + 0.1)).to(dtype))(torch.randn(*n, generator=g))
    a, b = away(1, K), away(N, 1)
    x, y = torch.randn(M, K, generator=g).to(dtype), torch.randn(M, N, generator=g).to(dtype)
    x[1, 5] = float("inf")
    rows = torch.zeros(M, dtype=torch.int32)
    ref, tol = reference(x, y, rows, [(a, b, 0.5)], K)
    assert torch.isinf(ref[1]).all()
    pool = pool_of(q4, [(a, b, 0.5)], K, N, 1, 1, dtype)
    out = pool.add(x.to(DEV), rows.to(DEV), y.to(DEV)).double().cpu()
    assert torch.equal(out[1], ref[1])
    clean = torch.arange(M) != 1
    check(out[clean], ref[clean], tol[clean], "other rows")


@pytest.mark.parametrize("M", [9, 200, 500])
def test_a_broken_adapter_stays_with_its_rows(q4, M):
    """An infinity in one adapter's B, NaN in another's A: rows of other adapters, and of none, in the same tile."""
    K, N, dtype = 320, 400, torch.bfloat16
    g = torch.Generator().manual_seed(13)
    ads = adapters(g, [16, 16, 32, 64], K, N, dtype)
    rows = row_slots(g, M, 4, "mixed")
    x, y = torch.randn(M, K, generator=g).to(dtype), torch.randn(M, N, generator=g).to(dtype)
    ref, tol = reference(x, y, rows, ads, K)
    ads[1][1][7, 3] = float("inf")
    ads[2][0][5, 11] = float("nan")
    pool = pool_of(q4, ads, K, N, 4, 64, dtype)
    out = pool.add(x.to(DEV), rows.to(DEV), y.to(DEV)).cpu()
    whole = (rows != 1) & (rows != 2)
    check(out[whole], ref[whole], tol[whole], "beside broken adapters")
    assert torch.isnan(out[rows == 2]).all()
    bad, fine = out[rows == 1][:, 7], out[rows == 1][:, :7]
    assert not torch.isfinite(bad).any()
    check(fine, ref[rows == 1][:, :7], tol[rows == 1][:, :7], "other columns of a broken adapter")
    pool.device_error()


def test_slot_out_of_range_is_reported(q4):
    K, N, dtype = 64, 64, torch.float16
    g = torch.Generator().manual_seed(10)
    ads = adapters(g, [8], K, N, dtype)
    pool = pool_of(q4, ads, K, N, 1, 8, dtype)
    x, y = torch.randn(3, K, generator=g).to(dtype).to(DEV), torch.randn(3, N, generator=g).to(dtype).to(DEV)
    out = pool.add(x, torch.tensor([0, 1, -5], dtype=torch.int32, device=DEV), y)
    assert torch.equal(out[1:], y[1:]) and not torch.equal(out[0], y[0])
    with pytest.raises(q4.GPTQ4Error) as e:
        pool.device_error()
    assert e.value.status == q4.GPTQ_Q4_DEVICE_FAULT
    pool.device_error()                                  # reading it cleared it


def test_rows_past_32_bit_offsets(q4):
    """Rows that begin more than 2^32 bytes into their tensors."""
    K = N = 64
    stride, M, dtype = 1 << 29, 6, torch.float16         # 6 GB
    g = torch.Generator().manual_seed(11)
    ads = adapters(g, [16], K, N, dtype)
    pool = pool_of(q4, ads, K, N, 1, 16, dtype)
    big = torch.empty(stride * M, dtype=dtype, device=DEV)
    xv, yv = big.as_strided((M, K), (stride, 1)), big.as_strided((M, N), (stride, 1), 64)
    x, y = torch.randn(M, K, generator=g).to(dtype), torch.randn(M, N, generator=g).to(dtype)
    xv.copy_(x), yv.copy_(y)
    rows = torch.zeros(M, dtype=torch.int32)
    pool.add(xv, rows.to(DEV), yv, out=yv)
    ref, tol = reference(x, y, rows, ads, K)
    check(yv, ref, tol, "large offsets")


def test_beside_the_quantised_projection(q4):
    """y of a packed layer plus the adapters, as a decoder layer would run it."""
    import synthetic
    K, N, gs, M = 512, 256, 128, 9
    layer = synthetic.make_layer(K, N, gs, key=(77,))
    mat = q4.Q4Matrix(*(torch.from_numpy(np.ascontiguousarray(t)).to(DEV) for t in (layer.qweight, layer.qzeros, layer.scales)),
                      None, None, gs)
    g = torch.Generator().manual_seed(12)
    ads = adapters(g, [16, 8], K, N, torch.float16)
    pool = pool_of(q4, ads, K, N, 2, 16, torch.float16)
    x = torch.randn(M, K, generator=g).half()
    rows = torch.randint(-1, 2, (M,), generator=g, dtype=torch.int32)
    y = mat(x.to(DEV))
    ref, tol = reference(x, y.cpu(), rows, ads, K)
    check(pool.add(x.to(DEV), rows.to(DEV), y), ref, tol, "beside the projection")


def test_shapes_of_more_dimensions(q4):
    """x [.., K] and y [.., N] of any leading dimensions; another shape with as many elements is refused, not read as
    other rows."""
    K, N, dtype = 64, 96, torch.float16
    g = torch.Generator().manual_seed(18)
    ads = adapters(g, [8], K, N, dtype)
    pool = pool_of(q4, ads, K, N, 1, 8, dtype)
    x, y = torch.randn(6, K, generator=g).to(dtype).to(DEV), torch.randn(6, N, generator=g).to(dtype).to(DEV)
    rows = torch.zeros(6, dtype=torch.int32, device=DEV)
    want = pool.add(x, rows, y)
    got = pool.add(x.view(2, 3, K), rows, y.view(3, 1, 2, N))
    assert got.shape == (3, 1, 2, N) and torch.equal(got.view(6, N), want)
    assert torch.equal(pool.add(x.view(6, 8, 8), rows, y.view(6, 4, 24)).view(6, N), want)     # heads of a row
    assert torch.equal(pool.add(x[0], rows[:1], y[0]), want[0])
    assert torch.equal(pool.add(x.view(-1), rows, y), want)
    apart = y.view(2, 3, N).transpose(0, 1).contiguous().transpose(0, 1)                       # rows in another order
    assert torch.equal(pool.add(x, rows, apart).view(6, N), want)
    for args in ((x.view(3, 4, K // 2), rows, y), (x.view(3, 2, 2, K // 2), rows[:4], y), (x, rows, y.view(2, 6, N // 2)),
                 (x[:5].reshape(-1)[:-1], rows[:5], y[:5]), (x, rows, y, apart)):
        with pytest.raises(q4.GPTQ4Error) as e:
            pool.add(*args)
        assert e.value.status == q4.GPTQ_Q4_INVALID_ARGUMENT
    pool.device_error()


def captured(f):
    """f() captured into a graph, after one call outside it."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            f()
    torch.cuda.synchronize()
    return graph


@pytest.mark.parametrize("M", [3, 40])
@pytest.mark.parametrize("grow", ["call", "reserve"])
def test_a_captured_step_outlives_a_larger_call(q4, M, grow):
    """A step captured at few rows, then calls that need larger workspaces: the graph goes on giving its result, and
    writes nothing into memory that others have been given since."""
    K, N, dtype = 264, 520, torch.bfloat16
    g = torch.Generator().manual_seed(16)
    ads = adapters(g, [256, 40, 16], K, N, dtype)
    pool = pool_of(q4, ads, K, N, 3, 256, dtype)
    x, y = torch.randn(2000, K, generator=g).to(dtype), torch.randn(2000, N, generator=g).to(dtype)
    rows = row_slots(g, 2000, 3, "mixed")
    ref, tol = reference(x, y, rows, ads, K)
    xd, yd, rd = x.to(DEV), y.to(DEV), rows.to(DEV)
    out = torch.empty(M, N, dtype=dtype, device=DEV)
    graph = captured(lambda: pool.add(xd[:M], rd[:M], yd[:M], out=out))
    if grow == "reserve":
        pool.reserve(700)
        pool.reserve(2000)
    for m in (65, 300, 700, 2000):
        check(pool.add(xd[:m], rd[:m], yd[:m]), ref[:m], tol[:m], f"{m} rows")
    others = [torch.full((n,), 77, dtype=torch.int8, device=DEV) for n in [1 << 16] * 40 + [1 << 21] * 4]
    torch.cuda.synchronize()
    for _ in range(2):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check(out, ref[:M], tol[:M], "replayed")
    assert all((o == 77).all() for o in others)
    pool.device_error()


@pytest.mark.parametrize("M", [200, 900])
def test_a_workspace_grown_while_capturing(q4, M):
    """The captured call is the first that needs the larger workspace; calls outside the graph use it too, before and
    after the graph has gone."""
    K, N, dtype = 264, 520, torch.float16
    g = torch.Generator().manual_seed(17)
    ads = adapters(g, [64, 40, 16], K, N, dtype)
    pool = pool_of(q4, ads, K, N, 3, 64, dtype)
    x, y = torch.randn(M, K, generator=g).to(dtype), torch.randn(M, N, generator=g).to(dtype)
    rows = row_slots(g, M, 3, "mixed")
    ref, tol = reference(x, y, rows, ads, K)
    xd, yd, rd = x.to(DEV), y.to(DEV), rows.to(DEV)
    out, side, graph = torch.empty_like(yd), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        pool.add(xd, rd, yd, out=out)
    check(pool.add(xd, rd, yd), ref, tol, "before a replay")
    graph.replay()
    check(out, ref, tol, "replayed")
    del graph
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    check(pool.add(xd, rd, yd), ref, tol, "after the graph")
    pool.device_error()


def test_refusals(q4):
    bad = q4.GPTQ_Q4_INVALID_ARGUMENT

    def refused(status, f, *args, **kw):
        with pytest.raises(q4.GPTQ4Error) as e:
            f(*args, **kw)
        assert e.value.status == status and e.value.message

    for args in ((60, 64, 1, 8), (64, 0, 1, 8), (64, 64, 0, 8), (64, 64, 5000, 8), (64, 64, 1, 0), (64, 64, 1, 257)):
        refused(bad, q4.LoraPool, *args)
    refused(q4.GPTQ_Q4_UNSUPPORTED, q4.LoraPool, 64, 64, 1, 8, dtype=torch.float32)
    refused(bad, q4.LoraPool, 64, 64, 1, 8, dtype=torch.int32)
    pool = q4.LoraPool(64, 128, 2, 8)
    a, b = torch.zeros(8, 64, dtype=torch.float16, device=DEV), torch.zeros(128, 8, dtype=torch.float16, device=DEV)
    refused(bad, pool.set, 2, a, b)
    refused(bad, pool.set, 0, a, b[:, :7])
    refused(bad, pool.set, 0, a.float(), b.float())
    refused(bad, pool.set, 0, a, b, float("nan"))
    refused(bad, pool.set, 0, torch.zeros(9, 64, dtype=torch.float16, device=DEV),
            torch.zeros(128, 9, dtype=torch.float16, device=DEV))
    refused(bad, q4.gptq_q4_lora_set, pool.handle, 0, a.cpu().data_ptr(), b.data_ptr(), 8, 1.0, 0)
    refused(bad, pool.reserve, -1)
    x, y = torch.zeros(4, 64, dtype=torch.float16, device=DEV), torch.zeros(4, 128, dtype=torch.float16, device=DEV)
    rows = torch.zeros(4, dtype=torch.int32, device=DEV)
    refused(bad, pool.add, x, rows.long(), y)
    refused(bad, pool.add, x, rows[:3], y)
    refused(bad, pool.add, x[:, :56], rows, y)
    refused(bad, pool.add, x.bfloat16(), rows, y)
    refused(bad, pool.add, x, rows, y, out=y[:, :64])
    refused(bad, pool.add, x.cpu(), rows, y)
    wide = torch.zeros(4, 140, dtype=torch.float16, device=DEV)
    refused(bad, pool.add, x, rows, wide[:, 4:132])      # neither aligned nor strided by 8
    add, h = q4.gptq_q4_lora_add, pool.handle
    refused(bad, add, None, x.data_ptr(), 64, rows.data_ptr(), 4, y.data_ptr(), 128, y.data_ptr(), 128, 0)
    refused(bad, add, h, x.data_ptr(), 64, rows.data_ptr(), -1, y.data_ptr(), 128, y.data_ptr(), 128, 0)
    refused(bad, add, h, 0, 64, rows.data_ptr(), 4, y.data_ptr(), 128, y.data_ptr(), 128, 0)
    refused(bad, add, h, x.data_ptr(), 56, rows.data_ptr(), 4, y.data_ptr(), 128, y.data_ptr(), 128, 0)
    refused(bad, add, h, x.data_ptr(), 64, rows.data_ptr(), 4, y.data_ptr(), 128, y.data_ptr(), 136, 0)
    pool.device_error()
    wider = q4.LoraPool(64, 128, 1, 256)
    with pytest.raises(q4.GPTQ4Error) as e:              # 2 TB: past any GPU's memory
        wider.reserve(2_000_000_000)
    assert e.value.status == q4.GPTQ_Q4_OUT_OF_MEMORY
    assert torch.equal(wider.add(x, rows, y), y)         # and the pool still works
    pool.close()
