"""Steps and codes of the 4-bit cache where a difference of two 16-bit numbers does not fit fp32: the definition in
fractions, without any rounding but its own.  All of them have to be equal."""
import math
import random
from fractions import Fraction

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from paged4 import DEV, Step, no_handles_left  # noqa: E402, F401

BITS = {torch.float16: (11, -14), torch.bfloat16: (8, -126)}         # of the significand; least normal exponent


@pytest.fixture(scope="module")
def q4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gptq_bit_weight_gb300 as q4mod
    return q4mod


def unit(x, dtype):
    """The distance of the type's numbers at x."""
    bits, least = BITS[dtype]
    return Fraction(2) ** (max(math.frexp(float(abs(x)))[1] - 1 if x else least, least) - bits + 1)


def nearest(x, dtype):
    """x rounded to the type, ties to even."""
    u = unit(x, dtype)
    return round(x / u) * u


def definition(group, dtype):
    """(codes, step, least) of a group of fractions."""
    m = min(group)
    s = nearest((max(group) - m) / 15, dtype)
    return [min(round((x - m) / s), 15) if s else 0 for x in group], s, m


def in_fp32(group, dtype):
    """As `definition`, but differences are rounded to fp32 first."""
    f32 = lambda x: Fraction(float(torch.tensor(float(x), dtype=torch.float32)))                # noqa: E731
    m = min(group)
    s = nearest(f32(f32(max(group) - m) / 15), dtype)
    return [min(round(f32(x - m) / s), 15) if s else 0 for x in group], s, m


def groups_of(dtype, n):
    """Groups of up to n elements, as fractions: elements that are tiny beside the least one, which is a half step and a
    whole number of steps below 0; a tiny least element under elements at half steps; a step next to a border of the
    type; differences that are a half step but for their last bits."""
    r = random.Random(7)
    two = lambda e: Fraction(2) ** e                                                            # noqa: E731
    tinies = [two(-24), two(-20) * 3, two(-22)] if dtype == torch.float16 else [two(-133), two(-60) * 3, two(-26), two(-20)]
    out = []
    for s in (Fraction(1), Fraction(4), Fraction(3, 2)) + ((two(-100),) if dtype == torch.bfloat16 else ()):
        for k in range(14):
            for t in tinies:
                lo = -(k + Fraction(1, 2)) * s
                out.append([lo, lo + 15 * s, t, -t, Fraction(0)])
        halves = [(k + Fraction(1, 2)) * s for k in range(15)]
        for t in tinies:
            out += [[t, 15 * s, *halves], [-t, 15 * s, *halves]]
    for h in range(1028, 1920, 15):
        for sign in (1, -1):
            for last in (2047, 2046, 1025, 1024):
                out.append([sign * last * two(-16), Fraction(h)])
    for _ in range(300):
        s = nearest(Fraction(r.uniform(1, 2)), dtype) * 2 ** r.randint(0, 6)
        d = (r.randint(0, 14) + Fraction(1, 2)) * s
        lo = -nearest(d, dtype)
        x = nearest(d + lo, dtype)                     # what is left, of few bits
        near = [x + j * unit(x, dtype) for j in (-2, -1, 0, 1, 2)]
        out.append([lo, lo + 15 * s, *near, Fraction(0), *(-y for y in near)])
    kept = []
    for g in out:
        g = [x for x in (nearest(x, dtype) for x in g) if x >= g[0]]
        kept.append((g + [g[0]] * n)[:n])
    return kept


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("group", [32, 64])
def test_differences_that_do_not_fit_fp32(q4, group, dtype):
    D, page = 128, 16
    groups = groups_of(dtype, group)
    want = [definition(g, dtype) for g in groups]
    far = [a != in_fp32(g, dtype) for a, g in zip(want, groups)]
    assert sum(far) >= 40                              # such groups are among them
    per = D // group
    T = -(-len(groups) // per)
    x = torch.zeros(T, 3, D, dtype=dtype)
    flat = torch.tensor([[float(v) for v in g] for g in groups], dtype=torch.float64).to(dtype)
    assert all(Fraction(float(a)) == b for g, row in zip(groups, flat.tolist()) for a, b in zip(row, g))
    order = torch.randperm(group, generator=torch.Generator().manual_seed(1))
    flat = torch.cat([flat, torch.zeros(T * per - len(groups), group, dtype=dtype)])
    x[:, 1], x[:, 2] = flat[:, order].view(T, D), flat[:, order.flip(0)].view(T, D)
    step = Step(q4, [(T, T)], 1, D, page, dtype, group, seed=1)
    att = q4.PagedAttention(1, 1, D, page, dtype=dtype)
    att.append(x.view(T, -1).to(DEV), step.cache, step.batch)
    att.device_error()
    rec = torch.stack([step.pool.cpu()[int(step.table[0, t // page]), 0, t % page] for t in range(T)])
    words = rec[:, :D].contiguous().view(torch.int32).long() & 0xffffffff                       # [T, D / 4]
    codes = torch.stack([words >> (4 * (e // 2) + 16 * (e % 2)) & 15 for e in range(8)], -1)
    params = rec[:, D:].contiguous().view(dtype).double().view(T, 2, per, 2)
    for side, way in ((0, order), (1, order.flip(0))):
        c = codes.view(T, 2, per, group)[:, side].reshape(-1, group)
        for i, (code, s, m) in enumerate(want):
            got = params[:, side].reshape(-1, 2)[i]
            assert (Fraction(float(got[0])), Fraction(float(got[1]))) == (s, m), (i, groups[i], got)
            assert c[i].tolist() == [code[j] for j in way.tolist()], (i, s, m)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("group", [32, 64])
def test_which_finite_groups_read_back_finite(q4, group, dtype):
    """Those whose greatest element and the step's rounding, u of the span at most, stay within the type; past it the
    greatest may be infinite, as zeros and the largest fp16 number are.  Spans that fp32 has."""
    D, page = 128, 16
    big, u = Fraction(torch.finfo(dtype).max), Fraction(1, 2 ** BITS[dtype][0])
    r = random.Random(3)
    groups = []
    for i in range(400):
        lo = nearest(big * Fraction(r.uniform(-0.99, 0.99)), dtype)
        hi = nearest((big + u * lo) / (1 + u), dtype)
        while hi + u * (hi - lo) > big or hi - lo > Fraction(torch.finfo(torch.float32).max):
            hi -= unit(hi, dtype)
        groups.append([lo, hi] + [max(lo, nearest(lo + (hi - lo) * Fraction(r.random()), dtype)) for _ in range(group - 2)])
    groups.append([Fraction(0), Fraction(65504)] * (group // 2))
    per = D // group
    T = -(-len(groups) // per)
    flat = torch.tensor([[float(v) for v in g] for g in groups], dtype=torch.float64).to(dtype)
    flat = torch.cat([flat, torch.zeros(T * per - len(groups), group, dtype=dtype)])
    x = torch.zeros(T, 3, D, dtype=dtype)
    x[:, 1] = x[:, 2] = flat.view(T, D)
    step = Step(q4, [(T, T)], 1, D, page, dtype, group, seed=2)
    att = q4.PagedAttention(1, 1, D, page, dtype=dtype)
    att.append(x.view(T, -1).to(DEV), step.cache, step.batch)
    for got in att.read(step.cache, step.batch):
        got = got.cpu().reshape(-1, group)[:len(groups)]
        assert torch.isfinite(got[:-1]).all()
        assert torch.isinf(got[-1]).any() == (dtype == torch.float16)
    att.device_error()
