"""Operators that let one GPU hold more and longer contexts, as cases to be measured: the append to a paged
cache held in 4 bits, attention over such a cache, attention through a sliding window with a few first tokens
that stay visible, and the pages of a cache forked, freed and compacted.

`run` computes a case in plain torch operations, or with this package's operators where `own` is true.
`exact` computes it in 64 bits from the definitions.  Head layouts are those of the package's Llama-7B and
Llama-70B workloads (32 heads of 128; 64 query heads over 8 key/value heads of 128) and of smaller models.

The cache in 4 bits has a record of bytes for each token and key/value head, [pages, heads, page, record]:
codes of the key, codes of the value, parameters of the key, parameters of the value.  Eight codes share a
32-bit word, code e at bit 4 (e // 2) + 16 (e % 2); a group of 32 or 64 elements shares a step s and a least
value m, both of the cache's 16-bit type, and code c stands for m + s c, rounded to that type.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"float16": torch.float16, "bfloat16": torch.bfloat16}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a decode step of 64 requests: one token each, rotated, quantised, appended
        {"name": "append4_decode_64", "op": "append4", "B": 64, "q": 1, "kv": 2048, "Hq": 64, "Hkv": 8, "D": 128, "page": 16,
         "group": 32, "type": "bfloat16", "rotary": 128, "interleaved": False, "shape": 1},
        # prompts of three requests; interleaved pairs over half of the head
        {"name": "append4_prompts", "op": "append4", "B": 3, "q": 4096, "kv": 16384, "Hq": 32, "Hkv": 32, "D": 128, "page": 32,
         "group": 64, "type": "float16", "rotary": 64, "interleaved": True, "shape": 2},
        # one user at the start of an answer: latency
        {"name": "attend4_one_token", "op": "attend4", "B": 1, "q": 1, "kv": 777, "Hq": 32, "Hkv": 32, "D": 128, "page": 16,
         "group": 32, "type": "bfloat16", "window": 0, "sinks": 0, "shape": 3},
        # a decode step of 64 requests of very different lengths
        {"name": "attend4_decode_64", "op": "attend4", "B": 64, "q": 1, "kv": 8192, "Hq": 64, "Hkv": 8, "D": 128, "page": 16,
         "group": 32, "type": "float16", "window": 0, "sinks": 0, "shape": 4},
        # two requests with long contexts: the work has to be split along the context
        {"name": "attend4_decode_long", "op": "attend4", "B": 2, "q": 1, "kv": 131071, "Hq": 64, "Hkv": 8, "D": 128, "page": 64,
         "group": 64, "type": "bfloat16", "window": 0, "sinks": 0, "shape": 5},
        # a chunk of a long prompt over what the cache already holds
        {"name": "attend4_chunk_1024", "op": "attend4", "B": 1, "q": 1024, "kv": 16384, "Hq": 64, "Hkv": 8, "D": 128, "page": 16,
         "group": 32, "type": "bfloat16", "window": 0, "sinks": 0, "shape": 6},
        # a decode step of 32 long conversations that see their last 4096 tokens and the first four
        {"name": "sinks_decode_32", "op": "sinks", "B": 32, "q": 1, "kv": 65536, "Hq": 64, "Hkv": 8, "D": 128, "page": 16,
         "type": "bfloat16", "window": 4096, "sinks": 4, "shape": 7},
        # chunks of two documents, short heads, a window and an instruction of 100 tokens that stays visible
        {"name": "sinks_chunk_1500", "op": "sinks", "B": 2, "q": 1500, "kv": 16384, "Hq": 32, "Hkv": 8, "D": 64, "page": 32,
         "type": "float16", "window": 2048, "sinks": 100, "shape": 8},
        # one request branches into a second answer
        {"name": "fork_one", "op": "fork", "layers": 4, "bits": 4, "pages": 512, "B": 8, "forks": 1, "kv": 700, "Hkv": 8, "D": 128,
         "page": 16, "group": 32, "type": "bfloat16", "shape": 9},
        # a beam search step: 48 of 96 rows are replaced by copies of others
        {"name": "fork_beams_48", "op": "fork", "layers": 32, "bits": 16, "pages": 1536, "B": 96, "forks": 48, "kv": 400, "Hkv": 8,
         "D": 128, "page": 32, "group": 32, "type": "float16", "shape": 10},
        # a few requests are left in a small pool
        {"name": "compact_small", "op": "compact", "layers": 8, "bits": 16, "pages": 600, "B": 12, "kv": 800, "Hkv": 8, "D": 64,
         "page": 32, "group": 32, "type": "bfloat16", "window": 0, "sinks": 0, "shape": 11},
        # a pool of 16384 pages, a third of it in use after many requests have ended, others windowed
        {"name": "compact_large", "op": "compact", "layers": 32, "bits": 4, "pages": 16384, "B": 160, "kv": 2500, "Hkv": 8, "D": 128,
         "page": 16, "group": 32, "type": "float16", "window": 1024, "sinks": 4, "shape": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append4", "append4", "attend4", "attend4", "attend4", "attend4", "sinks", "sinks", "fork", "compact"])
    case = {"op": op, "type": rng.choice(list(TYPES)), "shape": rng.randrange(1 << 30)}
    if op in ("fork", "compact"):
        case |= {"layers": _log(rng, 1, 32), "bits": rng.choice([4, 16]), "Hkv": rng.choice([1, 8]), "D": rng.choice([64, 128]),
                 "page": rng.choice([16, 32, 64]), "group": rng.choice([32, 64])}
        if op == "fork":
            B = _log(rng, 2, 96)
            kv = _log(rng, 16, 400)
            return case | {"B": B, "forks": rng.randint(1, B // 2), "kv": kv, "pages": B * (kv // case["page"] + 2)}
        B = _log(rng, 1, 64)
        kv = _log(rng, 100, 2000)
        return case | {"B": B, "kv": kv, "pages": B * (kv // case["page"] + 1) + _log(rng, 10, 2000),
                       "window": rng.choice([0, 0, 500]), "sinks": rng.choice([0, 4, 40])}
    Hq, Hkv, D = rng.choice([(32, 32, 128), (64, 8, 128), (32, 8, 64), (40, 8, 128), (24, 8, 64), (16, 1, 128)])
    case |= {"Hq": Hq, "Hkv": Hkv, "D": D, "page": rng.choice([16, 32, 64])}
    if op != "sinks":
        case["group"] = rng.choice([32, 64])
    if op == "append4":
        decode = rng.random() < 0.5
        return case | {"B": _log(rng, 1, 256) if decode else rng.randint(1, 3), "q": 1 if decode else _log(rng, 2, 4096),
                       "kv": _log(rng, 4096, 16384) if not decode else 1024, "rotary": rng.choice([D, D, D // 2]),
                       "interleaved": rng.random() < 0.5}
    if op == "attend4":
        window, sinks = rng.choice([(0, 0), (0, 0), (1000, 0), (1000, 4)])
    else:
        window, sinks = _log(rng, 64, 4096), _log(rng, 1, 200)
    kind = rng.choice(["single", "single", "few", "chunk"])
    if kind == "single":
        B = _log(rng, 1, 128)
        return case | {"B": B, "q": 1, "kv": _log(rng, 1, min(131072, 524288 // B)), "window": window, "sinks": sinks}
    if kind == "few":
        return case | {"B": _log(rng, 1, 32), "q": rng.randint(2, 9), "kv": _log(rng, 32, 8192), "window": window, "sinks": sinks}
    return case | {"B": rng.randint(1, 2), "q": _log(rng, 16, 700), "kv": _log(rng, 1024, 8192), "window": window, "sinks": sinks}


def _lengths(case):
    """New tokens and cached tokens (the new ones among them) of each request: the largest as the case
    says, the others spread below it."""
    r = random.Random(case["shape"])
    B, q, kv = case["B"], case["q"], case["kv"]
    ql = [q] + [q if q < 16 else r.randint(max(1, q // 3), q) for _ in range(B - 1)]
    kl = [kv] + [_log(r, max(1, kv // 8), kv) for _ in range(B - 1)]
    return ql, [max(a, b) for a, b in zip(ql, kl)]


def _needed(case, n):
    """The pages that a request of n tokens still needs: all of its pages, or those of the first tokens and of the window."""
    page, w, s = case["page"], case.get("window", 0), case.get("sinks", 0)
    return [j for j in range(-(-n // page)) if not w or j * page < s or (j + 1) * page > n - w]


def _layout(case):
    """Of the cases about pages: lengths, the table's rows, and for forks the parents and children."""
    r = random.Random(case["shape"])
    B, page = case["B"], case["page"]
    kl = [case["kv"]] + [r.randint(case["kv"] // 2, case["kv"]) for _ in range(B - 1)]
    order = list(range(case["pages"]))
    r.shuffle(order)
    rows = []
    for b, n in enumerate(kl):
        row = [-1] * -(-n // page)
        shared = min(len(row), len(rows[-1])) // 2 if b % 2 else 0         # every other request shares a prefix with the last
        for j in _needed(case, n):
            row[j] = rows[-1][j] if j < shared and rows[-1][j] >= 0 else order.pop()
        rows.append(row)
    if case["op"] == "compact":
        return kl, rows, [], []
    who = r.sample(range(B), B)
    child = who[: case["forks"]]
    return kl, rows, [r.choice(who[case["forks"]:]) for _ in child], child


# ------------------------------------------------------------------ inputs

def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return torch.empty(shape, device=DEV, dtype=dtype).normal_(0.0, std, generator=g)


def _record(case):
    return case["D"] + 8 * case["D"] // case["group"]


def _quantise(x, group):
    """Codes, step and least value of groups along the last dimension of x, a 16-bit tensor."""
    y = x.float().unflatten(-1, (-1, group))
    least = y.amin(-1, keepdim=True)
    step = ((y.amax(-1, keepdim=True) - least) / 15).to(x.dtype).float()
    code = ((y - least) / step).round().nan_to_num(0.0, 0.0, 0.0).clamp(0, 15)
    return code.flatten(-2), step.squeeze(-1).to(x.dtype), least.squeeze(-1).to(x.dtype)


def _dequantise(code, step, least):
    group = code.shape[-1] // step.shape[-1]
    y = code.float().unflatten(-1, (-1, group)) * step.float()[..., None] + least.float()[..., None]
    return y.flatten(-2).to(step.dtype)


def _pack(k, v):
    """Records of bytes of (codes, step, least) of keys and values."""
    parts = []
    for code, _, _ in (k, v):
        c = code.to(torch.uint8).unflatten(-1, (-1, 8))
        parts.append((c[..., [0, 4, 1, 5]] | c[..., [2, 6, 3, 7]] << 4).flatten(-2))
    for _, step, least in (k, v):
        parts.append(torch.stack([step, least], -1).flatten(-2).view(torch.uint8))
    return torch.cat(parts, -1)


def _unpack(record, D, dtype):
    """(codes, step, least) of keys and of values, from records of bytes."""
    out = []
    params = record[..., D:].contiguous().view(dtype)
    for i in (0, 1):
        b = record[..., i * D // 2: (i + 1) * D // 2].unflatten(-1, (-1, 4))
        low, high = b & 15, b >> 4
        code = torch.stack([low[..., 0], low[..., 2], high[..., 0], high[..., 2],
                            low[..., 1], low[..., 3], high[..., 1], high[..., 3]], -1).flatten(-2)
        p = params.chunk(2, -1)[i].unflatten(-1, (-1, 2))
        out.append((code, p[..., 0], p[..., 1]))
    return out


def _inputs(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt, page, Hkv, D = TYPES[case["type"]], case["page"], case["Hkv"], case["D"]
    if case["op"] in ("fork", "compact"):
        kl, rows, parent, child = _layout(case)
        table = torch.full((case["B"], max(len(r) for r in rows) + 1), -1, dtype=torch.int32)
        for b, row in enumerate(rows):
            table[b, : len(row)] = torch.tensor(row, dtype=torch.int32)
        ints = {"table": table, "kv": torch.tensor(kl, dtype=torch.int32), "parent": torch.tensor(parent, dtype=torch.int32),
                "child": torch.tensor(child, dtype=torch.int32)}
        s = {n: t.to(DEV) for n, t in ints.items()}
        shape = (case["layers"], case["pages"], Hkv, page)
        if case["bits"] == 4:
            return s | {"kv4": torch.randint(0, 256, (*shape, _record(case)), dtype=torch.uint8, device=DEV, generator=g)}
        return s | {w: _normal(g, *shape, D, dtype=dt) for w in ("k", "v")}
    ql, kl = _lengths(case)
    need = [_needed(case | {"window": case["window"] + case["q"] if case.get("window") else 0}, n) for n in kl]
    pages, width = sum(len(n) for n in need) + 3, -(-max(kl) // page)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table, at = torch.full((case["B"], width), -1, dtype=torch.int32), 0
    for b, n in enumerate(need):                     # pages between the first tokens and the window have been freed
        table[b, n] = order[at:at + len(n)]
        at += len(n)
    cu = torch.tensor([0] + ql).cumsum(0).to(torch.int32)
    s = {"ql": ql, "kl": kl, "table": table.to(DEV), "cu": cu.to(DEV), "kv": torch.tensor(kl, dtype=torch.int32, device=DEV)}
    if case["op"] == "append4":
        s["kv4"] = torch.zeros((pages, Hkv, page, _record(case)), dtype=torch.uint8, device=DEV)
        s["qkv"] = _normal(g, sum(ql), (case["Hq"] + 2 * Hkv) * D, dtype=dt)
        return s
    s["q"] = _normal(g, sum(ql), case["Hq"], D, std=2.0, dtype=dt)
    # channels of keys have means of their own
    k = _normal(g, pages, Hkv, page, D, dtype=dt).add_(_normal(g, Hkv, 1, D, dtype=dt))
    v = _normal(g, pages, Hkv, page, D, dtype=dt)
    if case["op"] == "sinks":
        return s | {"k": k, "v": v}
    return s | {"kv4": _pack(_quantise(k, case["group"]), _quantise(v, case["group"]))}


def _frequencies(case):
    return 10000.0 ** (-2.0 * torch.arange(case["rotary"] // 2, dtype=torch.float64) / case["rotary"])


def prepare(case, seed):
    s = _inputs(case, seed) | {"case": case}
    dt = TYPES[case["type"]]
    if case["op"] == "append4":         # the table of cosines and sines, as a program keeps it
        angle = torch.arange(case["kv"], dtype=torch.float64, device=DEV)[:, None] * _frequencies(case).to(DEV)
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    if case["op"] == "compact":
        s["table_out"] = torch.empty_like(s["table"])
    if own:
        import gptq_bit_weight_gb300 as q4
        if case["op"] in ("fork", "compact"):
            s["pool"] = q4.PagePool([q4.PagedCache4(s["kv4"][i], case["D"], case["group"], dt) if case["bits"] == 4
                                     else q4.PagedCache(s["k"][i], s["v"][i]) for i in range(case["layers"])])
            s["dropped"] = s["child"].long()
            return s
        att = q4.PagedAttention(case["Hq"], case["Hkv"], case["D"], case["page"], dtype=dt)
        if case["op"] == "append4":
            att.set_rope(case["rotary"], case["kv"], base=10000.0, interleaved=case["interleaved"])
        s["attention"] = att
        s["cache"] = q4.PagedCache(s["k"], s["v"]) if case["op"] == "sinks" else \
            q4.PagedCache4(s["kv4"], case["D"], case["group"], dt)
        s["batch"] = q4.PagedBatch(s["cu"], s["kv"], s["table"], tokens=sum(s["ql"]), max_q=max(s["ql"]))
    return s


# ------------------------------------------------------------------ plain forms

def _append4(s):
    c = s["case"]
    Hq, Hkv, D, page, rot, dt = c["Hq"], c["Hkv"], c["D"], c["page"], c["rotary"], s["qkv"].dtype
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    req = torch.repeat_interleave(torch.arange(c["B"], device=DEV), n, output_size=sum(s["ql"]))
    pos = torch.arange(req.numel(), device=DEV) - s["cu"][1:].long()[req] + s["kv"].long()[req]
    at = s["table"].long()[req, pos // page]
    x = s["qkv"].view(-1, Hq + 2 * Hkv, D)
    first = slice(0, rot, 2) if c["interleaved"] else slice(0, rot // 2)
    second = slice(1, rot, 2) if c["interleaved"] else slice(rot // 2, rot)
    cos, sin = s["cos"][pos][:, None].double(), s["sin"][pos][:, None].double()      # 64 bits: codes have borders
    a, b = x[:, : Hq + Hkv, first].double(), x[:, : Hq + Hkv, second].double()
    qk = x[:, : Hq + Hkv].clone()
    qk[..., first], qk[..., second] = (a * cos - b * sin).to(dt), (b * cos + a * sin).to(dt)
    s["kv4"][at, :, pos % page] = _pack(_quantise(qk[:, Hq:], c["group"]), _quantise(x[:, Hq + Hkv:], c["group"]))
    k, v = _unpack(s["kv4"][at, :, pos % page], D, dt)
    return {"q": qk[:, :Hq].contiguous(), "k": _dequantise(*k), "v": _dequantise(*v)}


def _attend(s):
    """All requests at once, padded to the longest; of a windowed context only the first tokens and the last ones."""
    c = s["case"]
    B, Hq, Hkv, D, page, nq = c["B"], c["Hq"], c["Hkv"], c["D"], c["page"], max(s["ql"])
    cu, kv = s["cu"].long(), s["kv"].long()
    ql = cu[1:] - cu[:-1]
    window = c["window"] or 1 << 40
    head = c["sinks"] if c["window"] else 0
    span = min(max(s["kl"]), window + nq - 1)
    j = torch.cat([torch.arange(head, device=DEV).expand(B, -1),
                   kv[:, None] - span + torch.arange(span, device=DEV)], 1)                       # [B, keys]
    there = (j >= 0) & (j < kv[:, None])
    there[:, head:] &= j[:, head:] >= head
    i = (kv - ql)[:, None] + torch.arange(nq, device=DEV)                                         # [B, nq]
    seen = there[:, None] & (j[:, None] <= i[..., None]) & ((j[:, None] > i[..., None] - window) | (j[:, None] < head))
    jj = j.clamp(min=0)
    pg = s["table"].long().gather(1, (jj // page).clamp(max=s["table"].shape[1] - 1)).clamp(min=0)
    if c["op"] == "sinks":
        k, v = s["k"][pg, :, jj % page], s["v"][pg, :, jj % page]
    else:
        k, v = (_dequantise(*p) for p in _unpack(s["kv4"][pg, :, jj % page], D, s["q"].dtype))
    k, v = (t.transpose(1, 2).float() for t in (k, v))                                            # [B, Hkv, keys, D]
    row = (cu[:-1, None] + torch.arange(nq, device=DEV)).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().view(B, nq, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    scores = (q @ k.transpose(-1, -2)).view(B, Hkv, nq, Hq // Hkv, -1).mul_(D ** -0.5)
    scores.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    p = scores.sub_(scores.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, nq * (Hq // Hkv), -1) @ v).view(B, Hkv, nq, Hq // Hkv, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).permute(0, 2, 1, 3, 4).reshape(B, nq, Hq, D)
    good = torch.arange(nq, device=DEV) < ql[:, None]
    out = torch.empty_like(s["q"])
    out[row[good]] = o[good].to(out.dtype)
    return out


def _marks(s):
    """Which pages some request needs."""
    c, table, kv = s["case"], s["table"], s["kv"]
    page, pages, w, sinks = c["page"], c["pages"], c.get("window", 0), c.get("sinks", 0)
    j = torch.arange(table.shape[1], device=DEV) * page
    need = j < kv[:, None]
    if w:
        need = need & ((j < sinks) | (j + page > kv[:, None] - w))
    mark = torch.zeros(pages + 1, dtype=torch.bool, device=DEV)
    mark.scatter_(0, torch.where(need, table, pages).long().flatten(), True)
    return mark[:pages], need


def _caches(s):
    return {w: s[w] for w in ("kv4", "k", "v") if w in s}


def _fork(s):
    c, page = s["case"], s["case"]["page"]
    s["kv"].index_fill_(0, s["child"].long(), 0)                     # the beams that are dropped
    mark, _ = _marks(s)
    order = torch.argsort(mark.to(torch.int32), stable=True).to(torch.int32)
    free = torch.where(torch.arange(c["pages"], device=DEV) < (~mark).sum(), order, -1)
    fresh, parent, child = free[: c["forks"]], s["parent"].long(), s["child"].long()
    kv, rows = s["kv"][parent], s["table"][parent]
    j = torch.arange(rows.shape[1], device=DEV)
    rows = torch.where(j * page < kv[:, None], rows, -1)
    part = kv % page != 0
    last = (kv // page).clamp(max=rows.shape[1] - 1).long()
    src = rows.gather(1, last[:, None])[:, 0]
    rows = torch.where((j == last[:, None]) & part[:, None], fresh[:, None], rows)
    s["table"][child], s["kv"][child] = rows, kv
    src, dst = src[part].long(), fresh[part].long()
    for t in _caches(s).values():
        t[:, dst] = t[:, src]
    return {"table": s["table"], "kv": s["kv"], "free": free} | {"cache_" + n: t for n, t in _caches(s).items()}


def _compact(s):
    pages = s["case"]["pages"]
    mark, need = _marks(s)
    idx, count = torch.arange(pages, device=DEV), mark.sum()
    source, hole = mark & (idx >= count), ~mark & (idx < count)
    moved = int(source.sum())
    src = torch.argsort((~source).to(torch.int32), stable=True)[:moved]
    dst = torch.argsort((~hole).to(torch.int32), stable=True)[:moved]
    to = idx.to(torch.int32)
    to[src] = dst.to(torch.int32)
    s["table_out"].copy_(torch.where(need & (s["table"] >= 0), to[s["table"].clamp(min=0).long()], -1))
    for t in _caches(s).values():
        t[:, dst] = t[:, src]
    return {"table": s["table_out"], "count": count.to(torch.int32).view(1)} | {"cache_" + n: t for n, t in _caches(s).items()}


def run(state):
    c = state["case"]
    op = c["op"]
    if not own:
        return {"append4": _append4, "attend4": _attend, "sinks": _attend, "fork": _fork, "compact": _compact}[op](state)
    if op == "append4":
        q = state["attention"].append(state["qkv"], state["cache"], state["batch"])
        k, v = state["attention"].read(state["cache"], state["batch"])
        return {"q": q, "k": k, "v": v}
    if op in ("attend4", "sinks"):
        return state["attention"].attend(state["q"], state["cache"], state["batch"], window=c["window"], sinks=c["sinks"])
    caches = {"cache_" + n: t for n, t in _caches(state).items()}
    if op == "fork":
        state["kv"].index_fill_(0, state["dropped"], 0)
        free, _ = state["pool"].free(state["table"], state["kv"])
        state["pool"].fork(state["table"], state["kv"], state["parent"], state["child"], free[: c["forks"]])
        return {"table": state["table"], "kv": state["kv"], "free": free} | caches
    count = state["pool"].compact(state["table"], state["kv"], state["table_out"], window=c["window"], sinks=c["sinks"])
    return {"table": state["table_out"], "count": count} | caches


# ------------------------------------------------------------------ what a case cannot do without

def _seen(case, kv, i):
    """Keys that the token at index i of a context sees."""
    w = case["window"] or 1 << 60
    return min(i + 1, w) + (min(case["sinks"], max(0, i + 1 - w)) if case["window"] else 0)


def work(case):
    if case["op"] in ("fork", "compact"):
        kl, rows, parent, _ = _layout(case)
        page_bytes = case["layers"] * case["Hkv"] * case["page"] * (4 * case["D"] if case["bits"] == 16 else _record(case))
        entries = sum(len(r) for r in rows)
        if case["op"] == "fork":
            moved = sum(kl[p] % case["page"] != 0 for p in parent)
            return {"bytes": 2 * moved * page_bytes + 4 * (entries + case["pages"] + sum(len(rows[p]) for p in parent)), "flops": 0}
        used = {p for r in rows for p in r if p >= 0}
        return {"bytes": 2 * sum(p >= len(used) for p in used) * page_bytes + 8 * entries, "flops": 0}
    ql, kl = _lengths(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "append4":
        return {"bytes": sum(ql) * (4 * Hq * D + 4 * Hkv * D + 4 * case["rotary"] + Hkv * (2 * _record(case) + 4 * D)),
                "flops": sum(ql) * (3 * (Hq + Hkv) * case["rotary"] + 12 * Hkv * D)}
    token = 4 * D if case["op"] == "sinks" else _record(case)
    keys = sum(len([0] * min(k, _seen(case, k, k - 1) + q - 1)) for q, k in zip(ql, kl))
    pairs = sum(_seen(case, k, k - q + t) for q, k in zip(ql, kl) for t in range(q))
    return {"bytes": Hkv * token * keys + 4 * sum(ql) * Hq * D, "flops": 4 * Hq * D * pairs}


# ------------------------------------------------------------------ 64 bits

def _values64(codes, step, least, dtype):
    n = step.shape[-1]
    y = codes.double().reshape(*codes.shape[:-1], n, -1) * step.double().unsqueeze(-1) + least.double().unsqueeze(-1)
    return y.reshape(codes.shape).to(dtype).double()


def _rounded64(x, group, dtype):
    """The values that a quantised 16-bit tensor x stands for."""
    y = x.double().reshape(*x.shape[:-1], -1, group)
    lo, hi = y.min(-1).values, y.max(-1).values
    step = ((hi - lo) / 15).to(dtype)
    t = (y - lo[..., None]) / step.double()[..., None]
    c = torch.where(step.double()[..., None] > 0, torch.round(t), torch.zeros_like(t)).clamp(0, 15)
    return _values64(c.reshape(x.shape), step, lo, dtype)


def _words64(record, D, dtype):
    """Values of keys and values, from records: each code by its place in its 32-bit word."""
    words = record[..., :D].contiguous().view(torch.int32).long()
    codes = torch.stack([words >> (4 * (e // 2) + 16 * (e % 2)) & 15 for e in range(8)], -1).flatten(-2)
    params = record[..., D:].contiguous().view(dtype)
    half = params.shape[-1] // 2
    return [_values64(codes[..., i * D:(i + 1) * D], params[..., i * half:(i + 1) * half:2],
                      params[..., i * half + 1:(i + 1) * half:2], dtype) for i in (0, 1)]


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None                                                  # whole numbers and bytes
    s = _inputs(case, seed)
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    dt = TYPES[case["type"]]
    if case["op"] == "append4":
        z = s["qkv"].double().view(-1, Hq + 2 * Hkv, D)
        rot, f = case["rotary"], _frequencies(case).to(DEV)
        first, second = torch.arange(0, rot, 2, device=DEV), torch.arange(1, rot, 2, device=DEV)
        if not case["interleaved"]:
            first, second = torch.arange(rot // 2, device=DEV), torch.arange(rot // 2, rot, device=DEV)
        q, k, at = torch.empty_like(z[:, :Hq]), torch.empty_like(z[:, :Hkv]), 0
        for n, total in zip(s["ql"], s["kl"]):
            p = torch.arange(total - n, total, device=DEV)
            turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), p.double()[:, None] * f)[:, None, :]
            part = z[at:at + n, : Hq + Hkv].clone()
            u = torch.complex(part[:, :, first], part[:, :, second]) * turn
            part[:, :, first], part[:, :, second] = u.real, u.imag
            q[at:at + n], k[at:at + n] = part[:, :Hq], part[:, Hq:]
            at += n
        return {"q": q, "k": _rounded64(k.to(dt), case["group"], dt), "v": _rounded64(z[:, Hq + Hkv:].to(dt), case["group"], dt)}
    out, at, G = torch.empty_like(s["q"], dtype=torch.float64), 0, Hq // Hkv
    for b, (n, total) in enumerate(zip(s["ql"], s["kl"])):
        pages = s["table"][b, : -(-total // page)].long().clamp(min=0)
        i, j = torch.arange(total - n, total, device=DEV)[:, None], torch.arange(total, device=DEV)[None, :]
        hidden = j > i
        if case["window"]:
            hidden |= (j <= i - case["window"]) & (j >= case["sinks"])
        for h in range(Hkv):
            if case["op"] == "sinks":
                k, v = (s[w][pages, h].reshape(-1, D)[:total].double() for w in ("k", "v"))
            else:
                k, v = _words64(s["kv4"][pages, h].reshape(-1, _record(case))[:total], D, dt)
            q = s["q"][at:at + n, h * G:(h + 1) * G].double().transpose(0, 1)
            p = torch.softmax((q @ k.t() / math.sqrt(D)).masked_fill(hidden, -math.inf), -1)
            out[at:at + n, h * G:(h + 1) * G] = (p @ v).transpose(0, 1)
        at += n
    return out
