"""Handles given up in a thread that captures, or beside one that does, while the current stream is not captured: they
are freed at once, and the capture goes on."""
import gc
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from paged4 import no_handles_left  # noqa: E402, F401
from test_gpu_handles import DEV, MAKE, cache  # noqa: E402


@pytest.fixture(scope="module")
def q4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gptq_bit_weight_gb300 as q4mod
    return q4mod


def other_stream(give_up):
    with torch.cuda.stream(torch.cuda.Stream()):
        give_up()


def other_thread(give_up):
    failed = []

    def run():
        try:
            give_up()
        except Exception as e:                         # noqa: BLE001
            failed.append(e)
    t = threading.Thread(target=run)
    t.start()
    t.join()
    assert not failed


def use(q4, kind, handle):
    """Calls after which the handle has memory of all its sorts: made with it, grown by stream order, replaced."""
    if kind == "matrix":
        for m in (1, 40, 90):
            handle(torch.zeros(m, 256, dtype=torch.float16, device=DEV))
    elif kind == "adapters":
        handle.set(1, torch.zeros(8, 256, dtype=torch.float16, device=DEV), torch.zeros(128, 8, dtype=torch.float16, device=DEV))
        for m in (1, 300):
            handle.add(torch.zeros(m, 256, dtype=torch.float16, device=DEV), torch.ones(m, dtype=torch.int32, device=DEV),
                       torch.zeros(m, 128, dtype=torch.float16, device=DEV))
    elif kind == "attention":
        handle.set_rope(64, 100)
        handle.set_rope(64, 200)
    torch.cuda.synchronize()


@pytest.mark.parametrize("where", [other_stream, other_thread])
@pytest.mark.parametrize("given_up", ["closed", "dropped", "collected"])
@pytest.mark.parametrize("kind", MAKE)
def test_a_handle_given_up_beside_a_capture(q4, kind, given_up, where):
    pool, held = q4.PagePool([cache(q4)]), [MAKE[kind](q4)]
    use(q4, kind, held[0])
    table = torch.tensor([[3, 1]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([20], dtype=torch.int32, device=DEV)
    pool.free(table, lens)
    gc.collect()

    def give_up():
        if given_up == "closed":
            held[0].close()
        elif given_up == "dropped":
            held.clear()
        else:
            cycle = [held.pop()]
            cycle.append(cycle)
            del cycle
            gc.collect()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            _, count = pool.free(table, lens)
            where(give_up)
            assert not q4._kept
            ids, _ = pool.free(table, lens)
        graph.replay()
    torch.cuda.synchronize()
    assert count.tolist() == [2] and ids.tolist() == [0, 2, -1, -1]
    pool.device_error()


@pytest.mark.parametrize("kind", ["matrix", "adapters"])
def test_freeing_waits_for_calls_in_flight(q4, kind):
    """Calls on another stream, not waited for, whose handle is freed and whose memory is given to others at once."""
    K, N, M = 4096, 4096, 256
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(M, K, generator=g, device=DEV).half()
    side = torch.cuda.Stream()
    if kind == "matrix":
        import synthetic
        layer = synthetic.make_layer(K, N, 128, act_order=False, bias=False, key=(6, 1, 1))
        dev = lambda a: None if a is None else torch.from_numpy(a).to(DEV)             # noqa: E731
        parts = [dev(a) for a in (layer.qweight, layer.qzeros, layer.scales, layer.g_idx)]
        make = lambda: q4.Q4Matrix(*parts, None, 128)                                  # noqa: E731
        run = lambda h, out: h(x, out=out)                                             # noqa: E731
    else:
        a, b = torch.randn(64, K, generator=g, device=DEV).half(), torch.randn(N, 64, generator=g, device=DEV).half()
        y, slot = torch.randn(M, N, generator=g, device=DEV).half(), torch.zeros(M, dtype=torch.int32, device=DEV)

        def make():
            pool = q4.LoraPool(K, N, slots=1, max_rank=64)
            pool.set(0, a, b)
            return pool
        run = lambda h, out: h.add(x, slot, y, out=out)                                # noqa: E731
    want = torch.empty(M, N, dtype=torch.float16, device=DEV)
    run(make(), want)
    torch.cuda.synchronize()
    for _ in range(5):
        handle, outs = make(), [torch.zeros_like(want) for _ in range(40)]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for out in outs:
                run(handle, out)
            handle.close()
        others = [q4.LoraPool(K, N, slots=2, max_rank=64) for _ in range(3)]           # zeros in memory of these sizes
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for out in outs)
        for o in others:
            o.close()
