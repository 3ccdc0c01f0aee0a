"""The operators together, as examples/decoder_attention.py runs them, against
the whole computation in 64 bits on the dequantized weights.

Five stages round to fp16 (2^-11 each, of values no larger than a few times
the result's largest), the cached keys and weights p once more: 64 2^-11 of the
largest result leaves a factor of about eight."""
import importlib.util
import math
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("decoder_attention", os.path.join(ROOT, "examples", "decoder_attention.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_prompt_and_decode_match_the_whole_computation(example):
    q4 = example.q4
    Hq, Hkv, D, page, prompts, steps = 4, 2, 64, 8, (70, 5, 33), 6
    hidden, n = Hq * D, len(prompts)
    layer = example.DecoderAttention(Hq, Hkv, D, page, slots=3, max_rank=16, max_pos=256, groupsize=64, seed=3)
    g = torch.Generator().manual_seed(4)
    ads = {}
    for slot, rank in ((0, 16), (1, 5)):
        for name, pool in (("qkv", layer.qkv_adapters), ("o", layer.o_adapters)):
            a, b = (torch.randn(rank, pool.K, generator=g) * pool.K ** -0.5).half(), (torch.randn(pool.N, rank, generator=g) * 0.2).half()
            pool.set(slot, a.cuda(), b.cuda(), 1.5)
            ads[name, slot] = 1.5 * a.double().t() @ b.double().t()
    slots = [0, -1, 1]
    total = [p + steps for p in prompts]
    xs = [torch.randn(t, hidden, generator=g).half() for t in total]

    width = -(-max(total) // page)
    cache = q4.PagedCache(*(torch.full((n * width, Hkv, page, D), float("nan"), dtype=torch.float16, device="cuda") for _ in "kv"))
    table = torch.randperm(n * width, generator=g).to(torch.int32).view(n, width).cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")      # noqa: E731
    got = [[] for _ in prompts]
    done = [0] * n
    for count in [list(prompts)] + [[1] * n] * steps:
        cu = [0]
        for c in count:
            cu.append(cu[-1] + c)
        done = [d + c for d, c in zip(done, count)]
        x = torch.cat([xs[b][done[b] - count[b]:done[b]] for b in range(n)]).cuda()
        rows = i32([slots[b] for b in range(n) for _ in range(count[b])])
        y = layer.step(x, rows, cache, q4.PagedBatch(i32(cu), i32(done), table, tokens=cu[-1], max_q=max(count)))
        for b in range(n):
            got[b].append(y[cu[b]:cu[b + 1]].cpu())
    layer.check()

    w_qkv, w_o = layer.qkv.dequant().cpu().double(), layer.o.dequant().cpu().double()
    freqs, _ = q4.gptq_q4_rope_freqs(D, 500000.0, q4.GPTQ_Q4_ROPE_BANDS, 8.0, 1.0, 4.0, 8192)
    for b in range(n):
        x, T = xs[b].double(), total[b]
        add = lambda name: ads.get((name, slots[b]), 0.0)                  # noqa: E731
        qkv = (x @ (w_qkv + add("qkv"))).view(T, Hq + 2 * Hkv, D)
        angle = torch.arange(T, dtype=torch.float64)[:, None, None] * torch.tensor(freqs, dtype=torch.float64)
        u, v = qkv[:, :Hq + Hkv, :D // 2], qkv[:, :Hq + Hkv, D // 2:]
        turned = torch.cat([u * angle.cos() - v * angle.sin(), v * angle.cos() + u * angle.sin()], -1)
        q, k = turned[:, :Hq].view(T, Hkv, Hq // Hkv, D), turned[:, Hq:]
        s = torch.einsum("thgd,jhd->hgtj", q, k) / math.sqrt(D)
        s = s.masked_fill(torch.ones(T, T, dtype=torch.bool).triu(1), -math.inf)
        a = torch.einsum("hgtj,jhd->thgd", s.softmax(-1), qkv[:, Hq + Hkv:]).reshape(T, hidden)
        ref = a @ (w_o + add("o"))
        err = (torch.cat(got[b]).double() - ref).abs().max()
        assert float(err) <= 64 * 2.0 ** -11 * float(ref.abs().max()), (b, float(err), float(ref.abs().max()))


def test_the_example_runs(example, capsys):
    out = example.main(q_heads=8, kv_heads=2, head_dim=64, prompts=(40, 7, 130), decoded=5)
    assert out.shape == (3, 512) and "us a step" in capsys.readouterr().out
