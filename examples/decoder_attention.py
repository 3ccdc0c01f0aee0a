"""The attention half of a decoder layer over packed weights, as a server runs it.

    qkv = x . W_qkv (4 bits)  +  each request's low-rank adapter
    q   = rotary positions; keys and values go into the paged cache
    a   = attention over the cache
    y   = a . W_o (4 bits)    +  each request's low-rank adapter

Prompts of three requests go in together in one step, then tokens are decoded
one a step, in a captured CUDA graph; the lengths live on the GPU, so the graph
replays unchanged while they grow.  `python examples/decoder_attention.py`
prints how long a step takes.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gptq_bit_weight_gb300 as q4  # noqa: E402


def packed(K, N, groupsize, generator):
    """A random layer, packed to 4 bits: (qweight, qzeros, scales)."""
    w = torch.randn(K, N, device="cuda", generator=generator).mul_(K ** -0.5).half()
    scales = (w.view(K // groupsize, groupsize, N).abs().amax(1) / 7.0).half()
    qweight, qzeros = q4.pack(w, scales, groupsize=groupsize)
    return qweight, qzeros, scales


class DecoderAttention:
    """Projections, adapters and attention of one layer; hidden = q_heads * head_dim."""

    def __init__(self, q_heads, kv_heads, head_dim, page_size, slots, max_rank, max_pos, groupsize=128, dtype=torch.float16,
                 seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        hidden, kv = q_heads * head_dim, kv_heads * head_dim
        self.weights = [packed(hidden, n, groupsize, g) for n in (hidden, kv, kv)], packed(hidden, hidden, groupsize, g)
        self.qkv = q4.Q4Matrix.fused(self.weights[0], groupsize=groupsize)
        self.o = q4.Q4Matrix(*self.weights[1], groupsize=groupsize)
        for layer in (self.qkv, self.o):
            layer.set_act_dtype(dtype)
        self.qkv_adapters = q4.LoraPool(hidden, hidden + 2 * kv, slots, max_rank, dtype)
        self.o_adapters = q4.LoraPool(hidden, hidden, slots, max_rank, dtype)
        self.attention = q4.PagedAttention(q_heads, kv_heads, head_dim, page_size, dtype)
        self.attention.set_rope(head_dim, max_pos, base=500000.0, scaling="bands", factor=8.0, original=8192)

    def reserve(self, rows):
        """Size every workspace for steps of up to `rows` tokens, so that no step allocates."""
        for part in (self.qkv, self.o, self.qkv_adapters, self.o_adapters):
            part.reserve(rows)

    def step(self, x, row_slot, cache, batch):
        """x [tokens, hidden]: the step's tokens, request after request; row_slot: each token's adapter."""
        qkv = self.qkv(x)
        self.qkv_adapters.add(x, row_slot, qkv, out=qkv)
        q = self.attention.append(qkv, cache, batch)
        a = self.attention.attend(q, cache, batch).view(x.shape)
        y = self.o(a)
        return self.o_adapters.add(a, row_slot, y, out=y)

    def check(self):
        """Raise if a kernel has reported anything (synchronizes)."""
        for part in (self.qkv, self.o, self.qkv_adapters, self.o_adapters, self.attention):
            part.device_error()


def main(q_heads=64, kv_heads=8, head_dim=128, page_size=16, prompts=(1000, 37, 402), decoded=64):
    dtype, hidden, n = torch.bfloat16, q_heads * head_dim, len(prompts)
    layer = DecoderAttention(q_heads, kv_heads, head_dim, page_size, slots=4, max_rank=32, max_pos=8192, dtype=dtype)
    layer.reserve(sum(prompts))
    g = torch.Generator(device="cuda").manual_seed(1)
    normal = lambda *shape: torch.randn(*shape, device="cuda", generator=g)          # noqa: E731
    for slot, rank in ((0, 16), (2, 32)):                          # two adapters; the third request has none
        for pool in (layer.qkv_adapters, layer.o_adapters):
            pool.set(slot, (normal(rank, pool.K) * pool.K ** -0.5).to(dtype), (normal(pool.N, rank) * 0.1).to(dtype), 2.0)
    slots = torch.tensor([0, 2, -1], dtype=torch.int32, device="cuda")

    width = -(-(max(prompts) + decoded) // page_size)
    pages = n * width
    cache = q4.PagedCache(*(torch.empty(pages, kv_heads, page_size, head_dim, dtype=dtype, device="cuda") for _ in "kv"))
    table = torch.randperm(pages, device="cuda", generator=g).to(torch.int32).view(n, width)
    kv_len = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    lengths = torch.tensor(prompts)
    cu = torch.tensor([0, *lengths.cumsum(0)], dtype=torch.int32, device="cuda")
    prompt = q4.PagedBatch(cu, kv_len, table, tokens=sum(prompts), max_q=max(prompts))
    y = layer.step(normal(sum(prompts), hidden).to(dtype), slots.repeat_interleave(lengths.cuda()), cache, prompt)

    x = y[cu[1:].long() - 1].clone()                               # the last token of each prompt
    one = q4.PagedBatch(torch.arange(n + 1, dtype=torch.int32, device="cuda"), kv_len, table, tokens=n, max_q=1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                                  # one step outside, then capture the next
        kv_len.add_(1)
        layer.step(x, slots, cache, one)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            kv_len.add_(1)
            x.copy_(layer.step(x, slots, cache, one))
        a, b = (torch.cuda.Event(enable_timing=True) for _ in "ab")
        a.record()
        for _ in range(decoded - 1):
            graph.replay()
        b.record()
    torch.cuda.synchronize()
    layer.check()
    assert kv_len.tolist() == [p + decoded for p in prompts] and torch.isfinite(x).all()
    print(f"{sum(prompts)} prompt tokens of {n} requests, then {decoded} steps of {n} tokens: "
          f"{a.elapsed_time(b) / (decoded - 1) * 1e3:.1f} us a step ({q_heads} heads over {kv_heads} of {head_dim})")
    return x


if __name__ == "__main__":
    main()
