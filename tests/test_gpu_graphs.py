"""Work buffers and captured graphs: a graph holds the addresses that its calls
were given, and goes on with them whatever the handle is used for since."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import synthetic  # noqa: E402

DEV = "cuda:0"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def q4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gptq_bit_weight_gb300 as q4mod
    return q4mod


def make(q4, K, N, gs, act_order, dtype, path):
    layer = synthetic.make_layer(K, N, gs, act_order=act_order, bias=True, key=(93, K, N))
    dev = lambda a: None if a is None else torch.from_numpy(a).to(DEV)                 # noqa: E731
    mat = q4.Q4Matrix(dev(layer.qweight), dev(layer.qzeros), dev(layer.scales), dev(layer.g_idx), dev(layer.bias), gs)
    mat.set_act_dtype(dtype)
    mat.set_path(path)
    return mat


CASES = [  # K, N, groupsize, act-order, type, path, rows of the captured call
    (1024, 448, 32, True, "fp16", "AUTO", 2),
    (1024, 448, 128, False, "bf16", "AUTO", 3),
    (1024, 448, 64, True, "fp32", "AUTO", 1),
    (4096, 4096, 128, True, "fp16", "DECODE_MMA", 16),
    (4096, 1024, 128, False, "bf16", "PREFILL", 40),
]


@pytest.mark.parametrize("grow", ["call", "reserve"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}x{c[1]}-{c[4]}-{c[5]}-{c[6]}")
def test_a_captured_step_outlives_a_larger_call(q4, case, grow):
    K, N, gs, act, kind, path, M = case
    dtype = TYPES[kind]
    mat = make(q4, K, N, gs, act, dtype, getattr(q4, "GPTQ_Q4_PATH_" + path))
    x = torch.randn(900, K, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
    want = mat(x[:M]).clone()
    y = torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            y.copy_(mat(x[:M]))
    torch.cuda.synchronize()
    if grow == "reserve":
        mat.reserve(300)
        mat.reserve(900)
    before = mat.info()["device_bytes"]
    for m in (M + 1, 48, 300, 900):
        mat(x[:m])
    if grow == "call":
        assert mat.info()["device_bytes"] > before       # the calls did need more
    others = [torch.full((n,), 77, dtype=torch.int8, device=DEV) for n in [1 << 16] * 40 + [1 << 21] * 4]
    torch.cuda.synchronize()
    for _ in range(2):
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    assert all((o == 77).all() for o in others)
    mat.device_error()
    mat.close()


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}x{c[1]}-{c[4]}-{c[5]}")
def test_buffers_grown_while_capturing(q4, case):
    """The captured call is the first that needs them; calls outside the graph use them too, before and after the
    graph has gone."""
    K, N, gs, act, kind, path, _ = case
    dtype, path, M = TYPES[kind], getattr(q4, "GPTQ_Q4_PATH_" + path), 48
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(2)).to(dtype).to(DEV)
    other = make(q4, K, N, gs, act, dtype, path)
    want = other(x).clone()
    mat = make(q4, K, N, gs, act, dtype, path)
    mat(x[:1])
    y, side, graph = torch.empty_like(want), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        y.copy_(mat(x))
    assert torch.equal(mat(x), want)
    graph.replay()
    assert torch.equal(y, want)
    y.zero_()
    graph.replay()
    assert torch.equal(y, want)
    del graph
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    assert torch.equal(mat(x), want)
    for m in (mat, other):
        m.device_error()
        m.close()


def test_a_captured_step_outlives_its_bias(q4):
    """Detached, the bias stays with the graph and with nobody else; another one, attached later, is the graph's too."""
    K, N, M = 1024, 448, 3
    mat = make(q4, K, N, 128, False, torch.float16, q4.GPTQ_Q4_PATH_AUTO)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(3)).half().to(DEV)
    want = mat(x).clone()
    y, side, graph = torch.empty_like(want), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        y.copy_(mat(x))
    q4.gptq_q4_set_bias(mat.handle, None)
    others = [torch.full((1024,), 77, dtype=torch.int8, device=DEV) for _ in range(4000)]
    plain = mat(x)
    assert not torch.equal(plain, want)
    graph.replay()
    assert torch.equal(y, want)
    other = torch.randn(N, generator=torch.Generator().manual_seed(4)).half().to(DEV)
    q4.gptq_q4_set_bias(mat.handle, other.data_ptr())
    want = mat(x)
    graph.replay()
    assert torch.equal(y, want) and not torch.equal(want, plain)
    assert all((o == 77).all() for o in others[::97])
    mat.device_error()
    mat.close()
