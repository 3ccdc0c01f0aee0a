"""Pages of a cache: free lists, forks, copies and compaction, against a plain model of a table on the host; contents
are compared byte by byte."""
import gc
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from paged4 import no_handles_left, refused  # noqa: E402, F401

DEV = "cuda:0"


@pytest.fixture(scope="module")
def q4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gptq_bit_weight_gb300 as q4mod
    return q4mod


class Pool:
    """Caches of several layers (16 bits and 4 bits, of other shapes) with random bytes, and requests over them."""

    def __init__(self, q4, pages, page, B, kv, layers=3, seed=0, shared=True, extra=2, gap=False):
        r = random.Random(seed)
        g = torch.Generator().manual_seed(seed)
        self.pages, self.page = pages, page
        byte = lambda *s: torch.randint(0, 256, s, dtype=torch.uint8, generator=g)         # noqa: E731
        self.buffers, caches = [], []
        for i in range(layers):
            if i % 2:
                t = byte(pages, 2 + i, page, 160).to(DEV)
                self.buffers.append(t)
                caches.append(q4.PagedCache4(t, 128, 32, torch.float16))
            else:
                wide = byte(pages, 2, 1 + i, page, 64 * 2).to(DEV)                         # keys and values side by side
                k, v = (wide[:, j].view(torch.bfloat16) for j in (0, 1))
                self.buffers.append(wide)
                caches.append(q4.PagedCache(k, v))
        self.pool = q4.PagePool(caches)
        ids = list(range(pages))
        r.shuffle(ids)
        self.kv = [r.randint(0, kv) for _ in range(B)]
        self.rows = []
        for b, n in enumerate(self.kv):
            row = [ids.pop() for _ in range(-(-n // page))]
            if shared and b and r.random() < 0.5:
                m = min(len(row), len(self.rows[-1])) // 2
                ids += row[:m]
                row[:m] = self.rows[-1][:m]
            self.rows.append(row)
        width = max([len(x) for x in self.rows] + [1]) + extra
        full = torch.full((B, width + 3), -5, dtype=torch.int32)
        self.full = full.to(DEV)
        self.table = self.full[:, 1:1 + width]                                             # rows of a wider tensor
        for b, row in enumerate(self.rows):
            self.table[b, :len(row)] = torch.tensor(row, dtype=torch.int32, device=DEV)
            self.table[b, len(row):] = r.choice([-1, 10 ** 9, 0])                          # never looked at
        self.lens = torch.tensor(self.kv, dtype=torch.int32, device=DEV)

    def needed(self, b, window=0, sinks=0):
        n, p = self.kv[b], self.page
        return [j for j in range(-(-n // p)) if not window or j * p < sinks or (j + 1) * p > n - window]

    def used(self, window=0, sinks=0):
        return sorted({self.rows[b][j] for b in range(len(self.kv)) for j in self.needed(b, window, sinks)})

    def snapshot(self):
        return [t.cpu().clone() for t in self.buffers]


SIZES = [(1, 16, 1, 10), (40, 16, 3, 100), (1000, 8, 40, 150), (5000, 32, 70, 2000), (33000, 64, 20, 900), (31, 1, 4, 7), (128, 24, 9, 300), (6000, 32, 300, 900), (32768, 16, 5, 100), (32769, 16, 5, 100)]


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 0), (40, 20), (1, 1), (10 ** 6, 3)])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_free_list(q4, size, window, sinks):
    pages, page, B, kv = size
    p = Pool(q4, pages, page, B, kv, layers=1, seed=1)
    ids, count = p.pool.free(p.table, p.lens, window=window, sinks=sinks)
    used = set(p.used(window, sinks))
    free = [i for i in range(pages) if i not in used]
    assert count.tolist() == [len(free)] and ids.tolist() == free + [-1] * (pages - len(free))
    p.pool.device_error()


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 20)])
@pytest.mark.parametrize("size", SIZES[:4] + SIZES[5:], ids=str)
def test_compact(q4, size, window, sinks, in_place):
    pages, page, B, kv = size
    if page == 64 or page == 1 or page == 24:
        p = Pool(q4, pages, page, B, kv, layers=2, seed=2)
    else:
        p = Pool(q4, pages, page, B, kv, layers=3, seed=2)
    before = p.snapshot()
    old = p.table.clone()
    out = p.table if in_place else torch.full_like(p.table, 77)
    count = p.pool.compact(p.table, p.lens, None if in_place else out, window=window, sinks=sinks)
    used = p.used(window, sinks)
    n = len(used)
    holes = [i for i in range(n) if i not in set(used)]
    to = {i: i for i in used} | dict(zip([i for i in used if i >= n], holes))
    assert count.tolist() == [n]
    want = torch.full(old.shape, -1, dtype=torch.int32)
    for b, row in enumerate(p.rows):
        for j in p.needed(b, window, sinks):
            want[b, j] = to[row[j]]
    assert torch.equal(out.cpu(), want)
    if not in_place:
        assert torch.equal(p.table, old)
    assert (p.full[:, 0] == -5).all() and (p.full[:, -2:] == -5).all()
    for a, b in zip(before, p.snapshot()):
        ref = a.clone()
        for src, dst in to.items():
            ref[dst] = a[src]
        assert torch.equal(b, ref)
    # a second compaction moves nothing
    now = p.snapshot()
    assert p.pool.compact(out, p.lens, window=window, sinks=sinks).tolist() == [n]
    assert torch.equal(out.cpu(), want) and all(torch.equal(a, b) for a, b in zip(now, p.snapshot()))
    p.pool.device_error()


@pytest.mark.parametrize("size", [(60, 16, 6, 100), (900, 32, 40, 500), (200, 8, 16, 64)], ids=str)
def test_fork(q4, size):
    """Several children of one parent, lengths at page ends, empty parents, rows that stay; the free list feeds it."""
    pages, page, B, kv = size
    p = Pool(q4, pages, page, B, kv, seed=3)
    r = random.Random(4)
    p.kv[1] = p.kv[1] // page * page
    p.lens[1] = p.kv[1]
    p.rows[1] = p.rows[1][:p.kv[1] // page]
    who = r.sample(range(B), B)
    child, parents = who[:B // 2], who[B // 2:]
    parent = [parents[0]] * 2 + [r.choice(parents) for _ in child[2:]]
    child = child + [parents[0], 0, -1]
    parent = parent + [parents[0], -1, parents[0]]                       # a row that stays, and no forks
    fresh, _ = p.pool.free(p.table, p.lens)
    fresh = fresh[:len(child)].contiguous()
    f = fresh.tolist()
    before, old = p.snapshot(), p.table.cpu().clone()
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)       # noqa: E731
    p.pool.fork(p.table, p.lens, ints(parent), ints(child), fresh)
    p.pool.device_error()
    want, lens, moved = old.clone(), list(p.kv), []
    for i, (a, c) in enumerate(zip(parent, child)):
        if a < 0 or c < 0 or a == c:
            continue
        row = list(p.rows[a])
        if p.kv[a] % page:
            moved.append((row[-1], f[i]))
            row[-1] = f[i]
        want[c] = -1
        want[c, :len(row)] = torch.tensor(row, dtype=torch.int32)
        lens[c] = p.kv[a]
    assert torch.equal(p.table.cpu(), want) and p.lens.tolist() == lens
    for a, b in zip(before, p.snapshot()):
        ref = a.clone()
        for src, dst in moved:
            ref[dst] = a[src]
        assert torch.equal(b, ref)


def test_forks_that_cannot_be_done_are_left_out(q4):
    """Each fault by itself beside a good fork, which is done."""
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)       # noqa: E731
    for parent, child, fresh, length, bad_row in [
            ([0, 2], [1, 4], [50, 51], None, None),                      # none is at fault
            ([0, 99], [1, 4], [50, 51], None, None),                     # rows past the table
            ([0, 2], [1, 99], [50, 51], None, None),
            ([0, 2], [1, 0], [50, 51], None, None),                      # a parent as a child
            ([0, 2], [1, 1], [50, 51], None, None),                      # a child twice
            ([0, 2], [1, 4], [50, 50], None, None),                      # a fresh page twice
            ([0, 2], [1, 4], [50, 600], None, None),                     # no fresh page
            ([0, 2], [1, 4], [50, -1], None, None),
            ([0, 2], [1, 4], [50, 51], 10 ** 6, None),                   # the parent's length
            ([0, 2], [1, 4], [50, 51], -3, None),
            ([0, 2], [1, 4], [50, 51], None, 10 ** 6),                   # its last page
            ([0, 2], [1, 4], [50, 51], None, -1)]:
        p = Pool(q4, 64, 16, 6, 5, seed=5, shared=False)
        p.kv = [17, 5, 20, 3, 9, 1]
        p.lens.copy_(ints(p.kv))
        p.table[:, :2] = torch.arange(12, dtype=torch.int32, device=DEV).view(6, 2)
        if length is not None:
            p.lens[2] = length
        if bad_row is not None:
            p.table[2, 1] = bad_row
        before, old, lens = p.snapshot(), p.table.cpu().clone(), p.lens.tolist()
        p.pool.fork(p.table, p.lens, ints(parent), ints(child), ints(fresh))
        fine = (parent, child, fresh, length, bad_row) == ([0, 2], [1, 4], [50, 51], None, None)
        if fine:
            p.pool.device_error()
        else:
            assert refused(q4, p.pool.device_error, q4.GPTQ_Q4_DEVICE_FAULT)
            p.pool.device_error()
        clash = child[1] == 0
        want = old.clone()
        if not clash or fine:
            want[1] = -1
            want[1, :2] = torch.tensor([0, 50])
            lens[1] = 17
        if fine or clash:
            c = child[1]
            want[c] = -1
            want[c, :2] = torch.tensor([4, 51])
            lens[c] = 20
        if clash:                                                        # row 0 is a parent: the second fork is left out
            want, lens = old.clone(), [17, 17, 20, 3, 9, 1]
            want[1] = -1
            want[1, :2] = torch.tensor([0, 50])
        assert torch.equal(p.table.cpu(), want) and p.lens.tolist() == lens, (parent, child, fresh)
        for a, b in zip(before, p.snapshot()):
            ref = a.clone()
            ref[50] = a[1]
            if fine:
                ref[51] = a[5]
            assert torch.equal(b, ref)


def test_a_million_pages(q4):
    """Counts past a block's words, page numbers past 2^20: a few pages in use at the far end, and a few in between."""
    pages = (1 << 20) + 77
    k, v = (torch.zeros(pages, 1, 1, 64, dtype=torch.float16, device=DEV) for _ in "kv")
    k[:, 0, 0, 0] = torch.arange(pages, device=DEV) % 2039
    v[:, 0, 0, 1] = torch.arange(pages, device=DEV) % 2011
    pool = q4.PagePool([q4.PagedCache(k, v)])
    used = sorted(random.Random(11).sample(range(pages), 3000)) + [pages - 1]
    table = torch.tensor([used], dtype=torch.int32, device=DEV)
    lens = torch.tensor([len(used)], dtype=torch.int32, device=DEV)
    ids, count = pool.free(table, lens)
    mark = torch.ones(pages, dtype=torch.bool)
    mark[torch.tensor(used)] = False
    free = mark.nonzero().flatten().to(torch.int32)
    assert count.tolist() == [len(free)] and torch.equal(ids.cpu()[:len(free)], free) and (ids[len(free):] == -1).all()
    old = k[table[0].long(), 0, 0, 0].clone(), v[table[0].long(), 0, 0, 1].clone()
    n = len(set(used))
    assert pool.compact(table, lens).tolist() == [n] and int(table.max()) == n - 1
    assert torch.equal(k[table[0].long(), 0, 0, 0], old[0]) and torch.equal(v[table[0].long(), 0, 0, 1], old[1])
    pool.device_error()


def test_copy(q4):
    p = Pool(q4, 300, 16, 2, 40, layers=4, seed=6)
    before = p.snapshot()
    order = random.Random(7).sample(range(300), 300)
    src, dst = order[:120] + [-1, 5, 7], order[120:240] + [3, -1, 7]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)       # noqa: E731
    p.pool.copy(ints(src), ints(dst))
    p.pool.device_error()
    for a, b in zip(before, p.snapshot()):
        ref = a.clone()
        ref[dst[:120]] = a[src[:120]]
        assert torch.equal(b, ref)
    now = p.snapshot()
    p.pool.copy(ints([300, 1]), ints([2, 10 ** 9]))
    assert refused(q4, p.pool.device_error)
    assert all(torch.equal(a, b) for a, b in zip(now, p.snapshot()))
    p.pool.copy(ints([]), ints([]))
    p.pool.device_error()


def test_pages_past_32_bit_offsets(q4):
    """Pages that begin more than 2^32 bytes into a buffer."""
    n, shape, stride = 12, (2, 16, 160), 1 << 29
    far = torch.empty((n - 1) * stride + 2 * 16 * 160, dtype=torch.uint8, device=DEV).as_strided((n, *shape), (stride, 16 * 160, 160, 1))
    want = torch.randint(0, 256, (n, *shape), dtype=torch.uint8, generator=torch.Generator().manual_seed(12))
    far.copy_(want)
    pool = q4.PagePool([q4.PagedCache4(far, 128)])
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)       # noqa: E731
    pool.copy(ints(0, 11), ints(10, 1))
    want[10], want[1] = want[0].clone(), want[11].clone()
    assert torch.equal(far.cpu(), want)
    table, lens = ints(9, 2, -1).view(1, 3).repeat(2, 1), ints(20, 0)
    pool.fork(table, lens, ints(0), ints(1), ints(11))
    want[11] = want[2]
    assert torch.equal(far.cpu(), want) and table.tolist() == [[9, 2, -1], [9, 11, -1]] and lens.tolist() == [20, 20]
    assert pool.compact(table, lens).tolist() == [3] and table.tolist() == [[0, 2, -1], [0, 1, -1]]
    want[0], want[1] = want[9].clone(), want[11].clone()
    assert torch.equal(far.cpu(), want)
    pool.device_error()


def test_entries_past_the_last_page_are_reported(q4):
    p = Pool(q4, 64, 16, 3, 60, seed=8)
    p.kv[0] = 40
    p.lens[0] = 40
    p.table[0, 0], p.table[0, 1], p.table[0, 2] = 64, -9, 3
    used = {3} | {x for b in (1, 2) for x in p.rows[b]}
    ids, count = p.pool.free(p.table, p.lens)
    assert ids.tolist()[:count.item()] == [i for i in range(64) if i not in used]
    assert refused(q4, p.pool.device_error)
    p.pool.device_error()
    out = p.table.clone()
    assert p.pool.compact(p.table, p.lens, out).tolist() == [len(used)]
    assert out[0, :2].tolist() == [-1, -1] and out[0, 2] >= 0
    assert refused(q4, p.pool.device_error)


def test_empty_batch_and_captured_graph(q4):
    """No rows: every page is free.  In a graph, replays follow the table's contents."""
    p = Pool(q4, 500, 16, 8, 200, seed=9)
    ids, count = p.pool.free(p.table[:0], p.lens[:0])
    assert count.tolist() == [500] and ids.tolist() == list(range(500))
    assert p.pool.compact(p.table[:0], p.lens[:0]).tolist() == [0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(p.table)
    gc.collect()
    with torch.cuda.stream(side):
        p.pool.free(p.table, p.lens)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            ids, count = p.pool.free(p.table, p.lens)
            n = p.pool.compact(p.table, p.lens, out)
        for b in (3, 5):
            p.lens[b] = 0
            p.kv[b] = 0
            graph.replay()
            torch.cuda.synchronize()
            used = p.used()
            assert n.tolist() == [len(used)] and ids.tolist()[:count.item()] == [i for i in range(500) if i not in set(used)]
    p.pool.device_error()


@pytest.mark.parametrize("bits", [4, 16])
def test_beams_share_a_prefix(q4, bits):
    """Prompt, fork, a different token each, attention, one beam ends, compaction, attention: as if each beam had a
    cache of its own."""
    Hq, Hkv, D, page, dtype, n = 8, 2, 128, 16, torch.float16, 37
    g = torch.Generator().manual_seed(10)
    kv4 = lambda m: q4.PagedCache4.empty(m, Hkv, page, D, 32, dtype, DEV)                  # noqa: E731
    kv16 = lambda m: q4.PagedCache(*(torch.zeros(m, Hkv, page, D, dtype=dtype, device=DEV) for _ in "kv"))    # noqa: E731
    make = kv4 if bits == 4 else kv16
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    att.set_rope(D, 256)
    width = 4
    x = torch.randn(n, (Hq + 2 * Hkv) * D, generator=g).to(dtype).to(DEV)
    y = torch.randn(3, (Hq + 2 * Hkv) * D, generator=g).to(dtype).to(DEV)
    z = torch.randn(2, (Hq + 2 * Hkv) * D, generator=g).to(dtype).to(DEV)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)                       # noqa: E731

    def batch(table, kv, rows):
        return q4.PagedBatch(torch.tensor([0, *rows], device=DEV).cumsum(0).to(torch.int32), kv, table, tokens=sum(rows), max_q=max(rows))
    # each beam by itself
    alone = make(3 * width)
    table = torch.arange(3 * width, dtype=torch.int32, device=DEV).view(3, width)
    for b in range(3):
        att.append(x, alone, batch(table[b:b + 1], ints(n), [n]))
    kv = ints(n + 1, n + 1, n + 1)
    first = att.attend(att.append(y, alone, batch(table, kv, [1, 1, 1])), alone, batch(table, kv, [1, 1, 1]))
    keep = table[[0, 2]].contiguous()
    last = ints(n + 2, n + 2)
    second = att.attend(att.append(z, alone, batch(keep, last, [1, 1])), alone, batch(keep, last, [1, 1]))
    # sharing
    cache = make(20)
    pool = q4.PagePool([cache])
    table = torch.full((3, width), -1, dtype=torch.int32, device=DEV)
    table[0, :3] = ints(17, 5, 11)
    kv = ints(n, 0, 0)
    att.append(x, cache, batch(table[:1], ints(n), [n]))
    free, _ = pool.free(table, kv)
    pool.fork(table, kv, ints(0, 0), ints(1, 2), free[:2])
    assert kv.tolist() == [n] * 3 and table[:, :2].tolist() == [[17, 5]] * 3
    kv.add_(1)
    assert torch.equal(att.attend(att.append(y, cache, batch(table, kv, [1, 1, 1])), cache, batch(table, kv, [1, 1, 1])), first)
    kv[1] = 0
    assert pool.compact(table, kv).tolist() == [4]
    assert int(table.max()) == 3 and (table[1] == -1).all()
    keep, last = table[[0, 2]].contiguous(), ints(n + 2, n + 2)
    assert torch.equal(att.attend(att.append(z, cache, batch(keep, last, [1, 1])), cache, batch(keep, last, [1, 1])), second)
    att.device_error()
    pool.device_error()
