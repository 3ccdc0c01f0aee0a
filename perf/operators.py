"""Operators around the quantised projection, as cases to be measured: the low-rank adapters of a
batch's requests beside a projection, rotary positions with the append to the paged cache, and
attention of new tokens over that cache.

`run` computes a case in plain torch operations (32 bits, rounded once at the end), or with this
package's operators where `own` is true.  `exact` computes it in 64 bits from the definitions.
Sizes are those of the package's Llama-7B and Llama-70B workloads: hidden 4096 with 32 heads of 128,
hidden 8192 with 64 query heads and 8 key/value heads of 128, feed-forward 28672, fused QKV 10240.
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
        # one user, one token: the smallest call, all latency
        {"name": "lora_one_token", "op": "lora", "M": 1, "K": 4096, "N": 4096, "slots": 4, "rank": 16, "type": "float16",
         "segments": 1, "shape": 1},
        # a decode step of 64 requests over 32 adapters of mixed rank, beside the fused QKV projection
        {"name": "lora_decode_64", "op": "lora", "M": 64, "K": 8192, "N": 10240, "slots": 32, "rank": 64, "type": "bfloat16",
         "segments": 64, "shape": 2},
        # prompts of six requests in one pass, beside the gate/up projection
        {"name": "lora_prompts", "op": "lora", "M": 4099, "K": 8192, "N": 28672, "slots": 8, "rank": 64, "type": "float16",
         "segments": 6, "shape": 3},
        # a decode step of 64 requests: one token each, rotated and appended
        {"name": "append_decode_64", "op": "append", "B": 64, "q": 1, "kv": 2048, "Hq": 64, "Hkv": 8, "D": 128, "page": 16,
         "type": "bfloat16", "rotary": 128, "interleaved": False, "scaling": "none", "shape": 4},
        # prompts of three requests; interleaved pairs over half of the head, scaled for a longer context
        {"name": "append_prompts", "op": "append", "B": 3, "q": 4096, "kv": 16384, "Hq": 32, "Hkv": 32, "D": 128, "page": 32,
         "type": "float16", "rotary": 64, "interleaved": True, "scaling": "bands", "shape": 5},
        # one user at the start of an answer: latency
        {"name": "attend_one_token", "op": "attend", "B": 1, "q": 1, "kv": 777, "Hq": 32, "Hkv": 32, "D": 128, "page": 16,
         "type": "bfloat16", "window": 0, "mixed": False, "shape": 6},
        # a decode step of 64 requests of very different lengths
        {"name": "attend_decode_64", "op": "attend", "B": 64, "q": 1, "kv": 8192, "Hq": 64, "Hkv": 8, "D": 128, "page": 16,
         "type": "float16", "window": 0, "mixed": False, "shape": 7},
        # two requests with long contexts: the work has to be split along the context
        {"name": "attend_decode_long", "op": "attend", "B": 2, "q": 1, "kv": 131071, "Hq": 64, "Hkv": 8, "D": 128, "page": 64,
         "type": "bfloat16", "window": 0, "mixed": False, "shape": 8},
        # a chunk of a prompt over what the cache already holds
        {"name": "attend_chunk_512", "op": "attend", "B": 1, "q": 512, "kv": 8192, "Hq": 64, "Hkv": 8, "D": 128, "page": 16,
         "type": "bfloat16", "window": 0, "mixed": False, "shape": 9},
        # a chunk of one request together with the single tokens of 47 others
        {"name": "attend_mixed_48", "op": "attend", "B": 48, "q": 384, "kv": 4096, "Hq": 64, "Hkv": 8, "D": 128, "page": 16,
         "type": "float16", "window": 0, "mixed": True, "shape": 10},
        # a long prompt's last part: the largest call
        {"name": "attend_prompt_4096", "op": "attend", "B": 1, "q": 4096, "kv": 16384, "Hq": 64, "Hkv": 8, "D": 128, "page": 64,
         "type": "bfloat16", "window": 0, "mixed": False, "shape": 11},
        # short heads and a sliding window over several requests' chunks
        {"name": "attend_window_d64", "op": "attend", "B": 3, "q": 1500, "kv": 4096, "Hq": 32, "Hkv": 8, "D": 64, "page": 32,
         "type": "float16", "window": 1024, "mixed": False, "shape": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lora", "lora", "append", "attend", "attend", "attend"])
    case = {"op": op, "type": rng.choice(list(TYPES)), "shape": rng.randrange(1 << 30)}
    if op == "lora":
        K, N = rng.choice([(4096, 4096), (4096, 11008), (11008, 4096), (8192, 10240), (8192, 28672), (28672, 8192)])
        M = _log(rng, 1, 4099)
        return case | {"M": M, "K": K, "N": N, "slots": rng.randint(1, 32 if M <= 256 else 8),
                       "rank": rng.choice([8, 16, 24, 32, 64]), "segments": rng.randint(1, min(M, 64))}
    Hq, Hkv, D = rng.choice([(32, 32, 128), (64, 8, 128), (32, 8, 64), (40, 8, 128), (24, 8, 64)])
    case |= {"Hq": Hq, "Hkv": Hkv, "D": D, "page": rng.choice([16, 32, 64])}
    if op == "append":
        decode = rng.random() < 0.5
        return case | {"B": _log(rng, 1, 256) if decode else rng.randint(1, 4), "q": 1 if decode else _log(rng, 2, 4096),
                       "kv": _log(rng, 4096, 16384) if not decode else 1024, "rotary": rng.choice([D, D, D // 2]),
                       "interleaved": rng.random() < 0.5, "scaling": rng.choice(["none", "linear", "bands"])}
    kind = rng.choice(["single", "single", "few", "chunk", "mixed"])
    window = rng.choice([0, 0, 0, 1000])
    if kind == "single":
        B = _log(rng, 1, 128)
        return case | {"B": B, "q": 1, "kv": _log(rng, 1, min(131072, 786432 // B)), "window": window, "mixed": False}
    if kind == "few":
        B = _log(rng, 1, 32)
        q = rng.randint(2, 9)
        return case | {"B": B, "q": q, "kv": _log(rng, 32, 8192), "window": window, "mixed": False}
    q = _log(rng, 16, 2048)
    B = rng.randint(1, 3) if kind == "chunk" else rng.randint(2, 48)
    return case | {"B": B, "q": q, "kv": _log(rng, 2048, 8192), "window": window, "mixed": kind == "mixed"}


def _lengths(case):
    """New tokens and cached tokens (the new ones among them) of each request: the largest as the case
    says, the others spread below it."""
    r = random.Random(case["shape"])
    B, q, kv = case["B"], case["q"], case["kv"]
    ql = [q] + [1 if case.get("mixed") else (q if q < 16 else r.randint(max(1, q // 3), q)) for _ in range(B - 1)]
    kl = [kv] + [_log(r, max(1, kv // 8), kv) for _ in range(B - 1)]
    return ql, [max(a, b) for a, b in zip(ql, kl)]


def _row_slots(case):
    """The adapter of each row: runs of rows with the same one (single rows in a decode step), and some
    with none.  Returns the list and the adapters' ranks; the last adapter's slot stays empty if there
    are more than two."""
    r = random.Random(case["shape"])
    M, n = case["M"], case["slots"]
    cuts = sorted(r.sample(range(1, M), min(case["segments"], M) - 1)) if M > 1 else []
    rows = []
    for a, b in zip([0] + cuts, cuts + [M]):
        rows += [r.randrange(n) if a == 0 or r.random() < 0.9 else -1] * (b - a)
    ranks = [case["rank"]] + [max(1, case["rank"] >> r.randrange(4)) for _ in range(n - 1)]
    if n > 2:
        ranks[-1] = 0
        rows = [0 if s == n - 1 and m == 0 else s for m, s in enumerate(rows)]
    return rows, ranks


# ------------------------------------------------------------------ inputs

def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return torch.empty(shape, device=DEV, dtype=dtype).normal_(0.0, std, generator=g)


def _inputs(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = TYPES[case["type"]]
    if case["op"] == "lora":
        M, K, N, n, R = (case[k] for k in ("M", "K", "N", "slots", "rank"))
        rows, ranks = _row_slots(case)
        keep = torch.arange(R, device=DEV)[None, :] < torch.tensor(ranks, device=DEV)[:, None]
        a = _normal(g, n, R, K, std=K ** -0.5, dtype=dt) * keep[:, :, None]
        b = _normal(g, n, N, R, std=0.3, dtype=dt) * keep[:, None, :]
        return {"x": _normal(g, M, K, dtype=dt), "y": _normal(g, M, N, dtype=dt), "a": a, "b": b, "ranks": ranks,
                "scale": [2.0 / max(1, v) ** 0.5 for v in ranks],
                "rows": torch.tensor(rows, dtype=torch.int32, device=DEV)}
    ql, kl = _lengths(case)
    page, Hq, Hkv, D = (case[k] for k in ("page", "Hq", "Hkv", "D"))
    need = [-(-k // page) for k in kl]
    pages, width = sum(need) + 3, max(need)
    order = torch.randperm(pages, device=DEV, generator=g).to(torch.int32)
    table = torch.zeros((case["B"], width), dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cu = [0]
    for v in ql:
        cu.append(cu[-1] + v)
    s = {"ql": ql, "kl": kl, "table": table, "cu": torch.tensor(cu, dtype=torch.int32, device=DEV),
         "kv": torch.tensor(kl, dtype=torch.int32, device=DEV),
         "k": _normal(g, pages, Hkv, page, D, dtype=dt), "v": _normal(g, pages, Hkv, page, D, dtype=dt)}
    if case["op"] == "append":
        s["qkv"] = _normal(g, cu[-1], (Hq + 2 * Hkv) * D, dtype=dt)
    else:
        s["q"] = _normal(g, cu[-1], Hq, D, std=2.0, dtype=dt)
    return s


SCALING = {"none": {}, "linear": {"factor": 4.0},
           "bands": {"factor": 8.0, "low": 1.0, "high": 4.0, "original": 8192}}


def _frequencies(case):
    """The angle per position of each pair: base^(-2i/rotary), slowed by the factor over all pairs (linear), or over
    those whose wavelength is long against the original context, with a blend between (bands)."""
    i = torch.arange(case["rotary"] // 2, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / case["rotary"])
    p = SCALING[case["scaling"]]
    if case["scaling"] == "linear":
        f = f / p["factor"]
    if case["scaling"] == "bands":
        turns = p["original"] * f / (2 * math.pi)
        share = ((turns - p["low"]) / (p["high"] - p["low"])).clamp(0, 1)
        f = f * share + f / p["factor"] * (1 - share)
    return f


def prepare(case, seed):
    s = _inputs(case, seed) | {"case": case}
    if case["op"] == "append":          # the table of cosines and sines, as a program keeps it
        angle = torch.arange(case["kv"], dtype=torch.float64, device=DEV)[:, None] * _frequencies(case).to(DEV)
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    if own:
        import gptq_bit_weight_gb300 as q4
        dt = TYPES[case["type"]]
        if case["op"] == "lora":
            pool = q4.LoraPool(case["K"], case["N"], case["slots"], case["rank"], dtype=dt)
            for i, r in enumerate(s["ranks"]):
                if r:
                    pool.set(i, s["a"][i, :r], s["b"][i, :, :r], s["scale"][i])
            s["pool"] = pool
        else:
            att = q4.PagedAttention(case["Hq"], case["Hkv"], case["D"], case["page"], dtype=dt)
            if case["op"] == "append":
                att.set_rope(case["rotary"], case["kv"], base=10000.0, interleaved=case["interleaved"],
                             scaling=case["scaling"], **SCALING[case["scaling"]])
            s["attention"] = att
            s["cache"] = q4.PagedCache(s["k"], s["v"])
            s["batch"] = q4.PagedBatch(s["cu"], s["kv"], s["table"], tokens=sum(s["ql"]), max_q=max(s["ql"]))
    return s


# ------------------------------------------------------------------ plain forms

def _lora(s):
    n, R, K = s["a"].shape
    hot = s["rows"][:, None] == torch.arange(n, device=DEV)[None, :]
    weight = hot * torch.tensor(s["scale"], device=DEV)
    t = (s["x"].float() @ s["a"].reshape(n * R, K).float().t()).view(-1, n, R) * weight[:, :, None]
    delta = t.reshape(-1, n * R) @ s["b"].permute(0, 2, 1).reshape(n * R, -1).float()
    return (s["y"].float() + delta).to(s["y"].dtype)


def _rotate(x, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    y, r = x.float().clone(), x[..., :rot].float()
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = r[..., : rot // 2], r[..., rot // 2:]
        y[..., : rot // 2], y[..., rot // 2: rot] = a * cos - b * sin, b * cos + a * sin
    return y.to(x.dtype)


def _append(s):
    c = s["case"]
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    req = torch.repeat_interleave(torch.arange(c["B"], device=DEV), n, output_size=sum(s["ql"]))
    pos = torch.arange(req.numel(), device=DEV) - s["cu"][1:].long()[req] + s["kv"].long()[req]
    at = s["table"].long()[req, pos // page]
    x = s["qkv"].view(-1, Hq + 2 * Hkv, D)
    qk = _rotate(x[:, : Hq + Hkv], s["cos"][pos][:, None], s["sin"][pos][:, None], c["interleaved"])
    s["k"][at, :, pos % page] = qk[:, Hq:]
    s["v"][at, :, pos % page] = x[:, Hq + Hkv:]
    return {"q": qk[:, :Hq].contiguous(), "k": s["k"], "v": s["v"]}


def _padded(s, ids, out):
    """Attention of the requests `ids`, padded to their longest."""
    c = s["case"]
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    nq, nk = max(s["ql"][b] for b in ids), max(s["kl"][b] for b in ids)
    sel = torch.tensor(ids, device=DEV)
    ql, kl, first = (s["cu"][1:] - s["cu"][:-1]).long()[sel], s["kv"].long()[sel], s["cu"].long()[sel]
    width = -(-nk // page)
    k, v = (s[w][s["table"].long()[sel, :width]].float().permute(0, 2, 1, 3, 4).reshape(len(ids), Hkv, width * page, D)
            for w in ("k", "v"))
    t = torch.arange(nq, device=DEV)
    row = (first[:, None] + t).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().view(len(ids), nq, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(len(ids), Hkv, -1, D)
    scores = (q @ k.transpose(-1, -2)).view(len(ids), Hkv, nq, Hq // Hkv, -1).mul_(D ** -0.5)
    last = (kl - ql)[:, None] + t
    j = torch.arange(width * page, device=DEV)
    seen = j[None, None, :] <= last[:, :, None]
    if c["window"]:
        seen &= j[None, None, :] > last[:, :, None] - c["window"]
    scores.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(len(ids), Hkv, -1, width * page) @ v).view(len(ids), Hkv, nq, Hq // Hkv, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).permute(0, 2, 1, 3, 4).reshape(len(ids), nq, Hq, D)
    good = t < ql[:, None]
    out[row[good]] = o[good].to(out.dtype)


def _attend(s):
    out = torch.empty_like(s["q"])
    few = [b for b, n in enumerate(s["ql"]) if n < 16]
    for ids in [few] * bool(few) + [[b] for b, n in enumerate(s["ql"]) if n >= 16]:
        _padded(s, ids, out)
    return out


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"lora": _lora, "append": _append, "attend": _attend}[op](state)
    if op == "lora":
        return state["pool"].add(state["x"], state["rows"], state["y"])
    if op == "append":
        q = state["attention"].append(state["qkv"], state["cache"], state["batch"])
        return {"q": q, "k": state["k"], "v": state["v"]}
    return state["attention"].attend(state["q"], state["cache"], state["batch"], window=state["case"]["window"])


# ------------------------------------------------------------------ what a case cannot do without

def _visible(case):
    ql, kl = _lengths(case)
    w = case["window"] or 1 << 60
    return sum(sum(min(k - q + t + 1, w) for t in range(q)) for q, k in zip(ql, kl))


def work(case):
    if case["op"] == "lora":
        rows, ranks = _row_slots(case)
        M, K, N = case["M"], case["K"], case["N"]
        used = [r for r in rows if r >= 0 and ranks[r]]
        return {"bytes": 2 * (len(used) * K + 2 * M * N + sum(ranks[r] for r in set(used)) * (K + N)) + 4 * M,
                "flops": 2 * sum(ranks[r] for r in used) * (K + N)}
    ql, kl = _lengths(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "append":
        return {"bytes": sum(ql) * (4 * (Hq + 2 * Hkv) * D + 4 * case["rotary"]),
                "flops": 3 * sum(ql) * (Hq + Hkv) * case["rotary"]}
    w = case["window"] or 1 << 60
    seen = sum(min(k, q + w - 1) for q, k in zip(ql, kl))
    return {"bytes": 4 * Hkv * D * seen + 4 * sum(ql) * Hq * D, "flops": 4 * Hq * D * _visible(case)}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "lora":
        out, rows = s["y"].double(), s["rows"].tolist()
        for a in sorted(set(r for r in rows if r >= 0)):
            m = torch.tensor([i for i, r in enumerate(rows) if r == a], device=DEV)
            out[m] += s["scale"][a] * ((s["x"][m].double() @ s["a"][a].double().t()) @ s["b"][a].double().t())
        return out
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    if case["op"] == "append":
        z = s["qkv"].double().view(-1, Hq + 2 * Hkv, D)
        rot, f = case["rotary"], _frequencies(case).to(DEV)
        first, second = torch.arange(0, rot, 2, device=DEV), torch.arange(1, rot, 2, device=DEV)
        if not case["interleaved"]:
            first, second = torch.arange(rot // 2, device=DEV), torch.arange(rot // 2, rot, device=DEV)
        k, v, q, at = s["k"].double(), s["v"].double(), torch.empty_like(z[:, :Hq]), 0
        for b, (n, total) in enumerate(zip(s["ql"], s["kl"])):
            p = torch.arange(total - n, total, device=DEV)
            turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), p.double()[:, None] * f)[:, None, :]
            part = z[at:at + n].clone()
            u = torch.complex(part[:, : Hq + Hkv, first], part[:, : Hq + Hkv, second]) * turn
            part[:, : Hq + Hkv, first], part[:, : Hq + Hkv, second] = u.real, u.imag
            where = s["table"][b].long()[p // page]
            k[where, :, p % page], v[where, :, p % page] = part[:, Hq:Hq + Hkv], part[:, Hq + Hkv:]
            q[at:at + n] = part[:, :Hq]
            at += n
        return {"q": q, "k": k, "v": v}
    out, at, G = torch.empty_like(s["q"], dtype=torch.float64), 0, Hq // Hkv
    for b, (n, total) in enumerate(zip(s["ql"], s["kl"])):
        pages = s["table"][b, : -(-total // page)].long()
        i, j = torch.arange(total - n, total, device=DEV)[:, None], torch.arange(total, device=DEV)[None, :]
        hidden = (j > i) | (j <= i - (case["window"] or total + 1))
        for h in range(Hkv):
            k, v = (s[w][pages, h].reshape(-1, D)[:total].double() for w in ("k", "v"))
            q = s["q"][at:at + n, h * G:(h + 1) * G].double().transpose(0, 1)
            p = torch.softmax((q @ k.t() / math.sqrt(D)).masked_fill(hidden, -math.inf), -1)
            out[at:at + n, h * G:(h + 1) * G] = (p @ v).transpose(0, 1)
        at += n
    return out
