"""Handles closed, or dropped with the cycle that holds them, while a step is captured: the capture goes on, and they are
freed after it."""
import gc

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import synthetic  # noqa: E402

DEV = "cuda:0"


@pytest.fixture(scope="module")
def q4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gptq_bit_weight_gb300 as q4mod
    return q4mod


def matrix(q4):
    layer = synthetic.make_layer(256, 128, 64, act_order=False, bias=False, key=(5, 1, 1))
    dev = lambda a: None if a is None else torch.from_numpy(a).to(DEV)                 # noqa: E731
    return q4.Q4Matrix(dev(layer.qweight), dev(layer.qzeros), dev(layer.scales), dev(layer.g_idx), None, 64)


def cache(q4):
    return q4.PagedCache4(torch.zeros(4, 2, 16, 80, dtype=torch.uint8, device=DEV), 64)


MAKE = {"matrix": matrix, "adapters": lambda q4: q4.LoraPool(256, 128, slots=2, max_rank=8),
        "attention": lambda q4: q4.PagedAttention(4, 2, 64, 16, dtype=torch.bfloat16),
        "pages": lambda q4: q4.PagePool([cache(q4)])}


@pytest.mark.parametrize("given_up", ["closed", "dropped", "collected"])
@pytest.mark.parametrize("kind", MAKE)
def test_a_handle_given_up_in_a_capture(q4, kind, given_up):
    pool, other = q4.PagePool([cache(q4)]), MAKE[kind](q4)
    table = torch.tensor([[3, 1]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([20], dtype=torch.int32, device=DEV)
    pool.free(table, lens)
    gc.collect()
    held = [other]
    if given_up == "collected":
        held.append(held)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            _, count = pool.free(table, lens)
            if given_up == "closed":
                other.close()
            del other, held
            if given_up == "collected":
                gc.collect()
            assert len(q4._kept) == 1
            ids, _ = pool.free(table, lens)
        graph.replay()
    torch.cuda.synchronize()
    assert count.tolist() == [2] and ids.tolist() == [0, 2, -1, -1]
    assert len(q4._kept) == 1
    pool.close()
    assert not q4._kept
