"""What the 4-bit cache, windows with sinks and the pages refuse: on the CPU, before any device call; with a handle,
on a GPU, before any launch."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from paged4 import no_handles_left  # noqa: E402, F401

DEV = "cuda:0"


@pytest.fixture(scope="module")
def q4():
    import __graft_entry__
    import os
    b = __graft_entry__._cuda_build_module()
    if not os.path.exists(b.LIB):
        b.build()
    import gptq_bit_weight_gb300 as q4mod
    return q4mod


def test_null_handles(q4):
    lib, bad = q4._lib, q4.GPTQ_Q4_INVALID_ARGUMENT
    assert lib.gptq_q4_attn_append4(None, None, 0, None, None, None, None, 0, None) == bad
    assert lib.gptq_q4_attn_attend4(None, None, 0, None, None, 1.0, 0, 0, None, 0, None) == bad
    assert lib.gptq_q4_attn_attend_sinks(None, None, 0, None, None, 1.0, 0, 0, None, 0, None) == bad
    assert lib.gptq_q4_attn_read(None, None, None, None, 0, None, 0, None) == bad
    assert lib.gptq_q4_attn_read4(None, None, None, None, 0, None, 0, None) == bad
    assert lib.gptq_q4_pages_free_list(None, None, 0, 0, None, None, None) == bad
    assert lib.gptq_q4_pages_fork(None, None, None, None, None, 1, None) == bad
    assert lib.gptq_q4_pages_copy(None, None, None, 1, None) == bad
    assert lib.gptq_q4_pages_compact(None, None, 0, 0, None, 0, None, None) == bad
    assert lib.gptq_q4_pages_device_error(None) == bad
    assert "NULL" in q4.gptq_q4_last_error()
    q4.gptq_q4_pages_free(None)


@pytest.mark.parametrize("change", [dict(data=0), dict(data=8), dict(bytes=0), dict(bytes=24), dict(bytes=-16), dict(stride=16),
                                    dict(stride=40), dict(stride=1 << 39), dict(pages=0), dict(pages=(1 << 22) + 1),
                                    dict(page_size=0), dict(bytes=(1 << 38) + 16, stride=1 << 38 | 16)], ids=str)
def test_pools_of_wrong_buffers(q4, change):
    a = dict(data=4096, bytes=32, stride=32, pages=4, page_size=16) | change
    buffer = (q4.gptq_q4_buffer * 1)(q4.gptq_q4_buffer(a["data"], a["bytes"], a["stride"]))
    assert not q4._lib.gptq_q4_pages_make(buffer, 1, a["pages"], a["page_size"])
    assert q4.gptq_q4_last_status() == q4.GPTQ_Q4_INVALID_ARGUMENT
    assert not q4._lib.gptq_q4_pages_make(None, 1, 4, 16) and not q4._lib.gptq_q4_pages_make(buffer, -1, 4, 16)


def test_caches_on_the_cpu_are_refused(q4):
    with pytest.raises(q4.GPTQ4Error):
        q4.PagedCache4(torch.zeros(4, 2, 16, 160, dtype=torch.uint8), 128)
    for group, dtype in ((48, torch.float16), (128, torch.float16), (32, torch.float64)):
        with pytest.raises(q4.GPTQ4Error):
            q4.PagedCache4(torch.zeros(4, 2, 16, 160, dtype=torch.uint8), 128, group, dtype)
    with pytest.raises(q4.GPTQ4Error):
        q4.PagePool([])
    assert [q4.PagedCache4.record(*a) for a in ((128, 32), (128, 64), (64, 32), (64, 64))] == [160, 144, 80, 72]


# ------------------------------------------------------------------ with a handle

@pytest.fixture(scope="module")
def made(q4):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    att = q4.PagedAttention(4, 2, 128, 16)
    kv = torch.zeros(6, 2, 16, 160, dtype=torch.uint8, device=DEV)
    batch = q4.PagedBatch(torch.tensor([0, 1], dtype=torch.int32, device=DEV), torch.tensor([5], dtype=torch.int32, device=DEV),
                          torch.zeros(1, 2, dtype=torch.int32, device=DEV), tokens=1)
    return att, kv, batch


@pytest.mark.gpu
def test_wrong_caches(q4, made):
    att, kv, batch = made
    lib, x = q4._lib, torch.zeros(1, 8 * 128, dtype=torch.float16, device=DEV)
    good = dict(kv=kv.data_ptr(), pages=6, page_stride=2 * 16 * 160, group=32)
    for change in (dict(kv=None), dict(kv=kv.data_ptr() + 8), dict(pages=0), dict(page_stride=2 * 16 * 160 - 16),
                   dict(page_stride=2 * 16 * 160 + 8), dict(page_stride=1 << 39), dict(group=16), dict(group=0)):
        c = ctypes.byref(q4.gptq_q4_cache4(*(good | change).values()))
        p, s = x.data_ptr(), 1024
        assert lib.gptq_q4_attn_append4(att.handle, p, s, c, batch.ref, None, p, s, None) == q4.GPTQ_Q4_INVALID_ARGUMENT
        assert lib.gptq_q4_attn_attend4(att.handle, p, s, c, batch.ref, 1.0, 0, 0, p, s, None) == q4.GPTQ_Q4_INVALID_ARGUMENT
        assert lib.gptq_q4_attn_read4(att.handle, c, batch.ref, p, s, p, s, None) == q4.GPTQ_Q4_INVALID_ARGUMENT
    q = torch.zeros(1, 4, 128, dtype=torch.float16, device=DEV)
    for cache in (q4.PagedCache4(kv, 128, 32, torch.bfloat16),                                   # another type, heads, page, width
                  q4.PagedCache4(kv[:, :1], 128), q4.PagedCache4(torch.zeros(6, 2, 8, 160, dtype=torch.uint8, device=DEV), 128),
                  q4.PagedCache4(torch.zeros(6, 2, 16, 80, dtype=torch.uint8, device=DEV), 64)):
        with pytest.raises(q4.GPTQ4Error):
            att.attend(q, cache, batch)
    for t in (kv[..., :144], kv.transpose(1, 2), kv[:, :, ::2], kv.half(), kv[0]):
        with pytest.raises(q4.GPTQ4Error):
            q4.PagedCache4(t, 128)
    att.device_error()


@pytest.mark.gpu
@pytest.mark.parametrize("group", [32, None])
def test_wrong_arguments(q4, made, group):
    att, kv, batch = made
    k = torch.zeros(6, 2, 16, 128, dtype=torch.float16, device=DEV)
    cache = q4.PagedCache4(kv, 128) if group else q4.PagedCache(k, k.clone())
    q = torch.zeros(1, 4, 128, dtype=torch.float16, device=DEV)
    for more in (dict(window=-1, sinks=1), dict(window=4, sinks=-1), dict(scale=float("nan"), sinks=1, window=2),
                 dict(out=q.float(), sinks=1), dict(out=q[:0])):
        with pytest.raises(q4.GPTQ4Error):
            att.attend(q, cache, batch, **more)
    out = torch.zeros(1, 2, 128, dtype=torch.float16, device=DEV)
    for more in (dict(k_out=q), dict(v_out=out.bfloat16()), dict(k_out=out[:0]), dict(v_out=out.cpu()),
                 dict(k_out=torch.zeros(1, 257, dtype=torch.float16, device=DEV)[:, 1:])):
        with pytest.raises(q4.GPTQ4Error):
            att.read(cache, batch, **more)
    with pytest.raises(q4.GPTQ4Error):
        att.append(q, cache, batch)
    att.device_error()


@pytest.mark.gpu
def test_wrong_rows_of_a_pool(q4, made):
    att, kv, _ = made
    cache = q4.PagedCache4(kv, 128)
    pool = q4.PagePool([cache])
    table = torch.zeros(3, 4, dtype=torch.int32, device=DEV)
    lens = torch.zeros(3, dtype=torch.int32, device=DEV)
    one = torch.zeros(1, dtype=torch.int32, device=DEV)
    for t, n in ((table.long(), lens), (table.t(), lens[:1].repeat(4)), (table, lens[:2]), (table.cpu(), lens), (table[0], lens),
                 (table, lens.long()), (table, torch.zeros(6, dtype=torch.int32, device=DEV)[::2]), (table[:1].expand(3, 4), lens)):
        with pytest.raises(q4.GPTQ4Error):
            pool.free(t, n)
        with pytest.raises(q4.GPTQ4Error):
            pool.compact(t, n)
        with pytest.raises(q4.GPTQ4Error):
            pool.fork(t, n, one, one, one)
    with pytest.raises(q4.GPTQ4Error):
        pool.free(table, lens, window=-1)
    with pytest.raises(q4.GPTQ4Error):
        pool.compact(table, lens, table[:2].contiguous())
    with pytest.raises(q4.GPTQ4Error):
        pool.fork(table, lens, one, one, one[:0])
    with pytest.raises(q4.GPTQ4Error):
        many = one.repeat(4097)
        pool.fork(table, lens, many, many, many)
    with pytest.raises(q4.GPTQ4Error):
        pool.copy(one, one.long())
    with pytest.raises(q4.GPTQ4Error):
        q4.PagePool([cache, q4.PagedCache4(kv[:3], 128)])
    with pytest.raises(q4.GPTQ4Error):
        q4.PagePool([q4.PagedCache4(kv[:0], 128)])
    pool.device_error()
