"""Chunks of tokens with 65 to 128 query heads for each key/value head: row tiles of one token, many of them over a
context of several key tiles, over both caches."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from paged4 import DEV, Step, attention, check, no_handles_left  # noqa: E402, F401


@pytest.fixture(scope="module")
def q4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gptq_bit_weight_gb300 as q4mod
    return q4mod


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 10)])
@pytest.mark.parametrize("shape", [(128, 1, 128, 256), (130, 2, 64, 16), (200, 2, 128, 32)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("group", [32, 64, None], ids=["4bit32", "4bit64", "16bit"])
def test_chunks_of_many_heads(q4, group, shape, window, sinks, dtype):
    Hq, Hkv, D, page = shape
    step = Step(q4, [(65, 700), (1, 300), (33, 513), (3, 2)], Hkv, D, page, dtype, group, seed=Hq, lead=1, tail=2, window=window, sinks=sinks)
    q = (torch.randn(step.tokens, Hq, D, generator=torch.Generator().manual_seed(1)) * 2).to(dtype)
    ref, tol = attention(step, q, D ** -0.5, window, sinks)
    att = q4.PagedAttention(Hq, Hkv, D, page, dtype=dtype)
    qd = q.to(DEV)
    for max_q in (65, 1):                              # the chunk kernel; the streaming one where a group is at most 16
        out = torch.full_like(qd, float("nan"))
        att.attend(qd, step.cache, step.make_batch(q4, max_q), out=out, window=window, sinks=sinks)
        check(out, ref, tol, f"max_q {max_q}")
        assert torch.isnan(out.cpu()[torch.isnan(ref)]).all()
    att.device_error()
