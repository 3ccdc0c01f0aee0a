"""Rotary angles and the argument checks of the operators around the
projection that need no GPU."""
import ctypes
import math
import os

import pytest


@pytest.fixture(scope="module")
def q4():
    import __graft_entry__
    b = __graft_entry__._cuda_build_module()
    if not os.path.exists(b.LIB):
        b.build()
    import gptq_bit_weight_gb300 as q4mod
    return q4mod


@pytest.mark.parametrize("rot,base", [(2, 10000.0), (64, 10000.0), (128, 500000.0), (48, 1e6)])
def test_plain_and_linear(q4, rot, base):
    f, m = q4.gptq_q4_rope_freqs(rot, base, q4.GPTQ_Q4_ROPE_PLAIN)
    assert m == 1.0 and len(f) == rot // 2
    for i, x in enumerate(f):
        assert math.isclose(x, base ** (-2.0 * i / rot), rel_tol=1e-14)
    g, _ = q4.gptq_q4_rope_freqs(rot, base, q4.GPTQ_Q4_ROPE_LINEAR, 4.0)
    assert all(math.isclose(a, b / 4, rel_tol=1e-14) for a, b in zip(g, f))


def test_ntk_keeps_the_fastest_pair_and_slows_the_slowest_by_the_factor(q4):
    f, _ = q4.gptq_q4_rope_freqs(128, 10000.0, q4.GPTQ_Q4_ROPE_PLAIN)
    g, _ = q4.gptq_q4_rope_freqs(128, 10000.0, q4.GPTQ_Q4_ROPE_NTK, 8.0)
    assert g[0] == 1.0 and math.isclose(g[-1], f[-1] / 8, rel_tol=1e-12)


def test_bands(q4):
    args = (500000.0, q4.GPTQ_Q4_ROPE_BANDS, 8.0, 1.0, 4.0, 8192)
    f, _ = q4.gptq_q4_rope_freqs(128, 500000.0, q4.GPTQ_Q4_ROPE_PLAIN)
    g, m = q4.gptq_q4_rope_freqs(128, *args)
    assert m == 1.0
    kinds = set()
    for a, b in zip(f, g):
        turns = 8192 * a / (2 * math.pi)
        if turns > 4:
            want, kind = a, "fast"
        elif turns < 1:
            want, kind = a / 8, "slow"
        else:
            s = (turns - 1) / 3
            want, kind = s * a + (1 - s) * a / 8, "between"
        kinds.add(kind)
        assert math.isclose(b, want, rel_tol=1e-13)
    assert kinds == {"fast", "slow", "between"}


def test_yarn(q4):
    base, rot, factor, orig = 10000.0, 128, 16.0, 4096
    f, _ = q4.gptq_q4_rope_freqs(rot, base, q4.GPTQ_Q4_ROPE_PLAIN)
    g, m = q4.gptq_q4_rope_freqs(rot, base, q4.GPTQ_Q4_ROPE_YARN, factor, 1.0, 32.0, orig)
    assert math.isclose(m, 0.1 * math.log(factor) + 1)
    pair = lambda r: rot * math.log(orig / (2 * math.pi * r)) / (2 * math.log(base))      # noqa: E731
    lo, hi = math.floor(pair(32.0)), math.ceil(pair(1.0))
    assert 0 < lo < hi < rot // 2
    for i, (a, b) in enumerate(zip(f, g)):
        s = 1 - min(max((i - lo) / (hi - lo), 0), 1)
        assert math.isclose(b, s * a + (1 - s) * a / factor, rel_tol=1e-13)
    assert g[0] == f[0] and math.isclose(g[-1], f[-1] / factor)


def test_refusals_without_a_device(q4):
    bad = q4.GPTQ_Q4_INVALID_ARGUMENT
    lib = q4._lib
    out, scale = (ctypes.c_double * 64)(), ctypes.c_double()
    for args in ((0, 1e4, 0, 1.0, 1.0, 4.0, 1), (7, 1e4, 0, 1.0, 1.0, 4.0, 1), (64, 1.0, 0, 1.0, 1.0, 4.0, 1),
                 (64, float("nan"), 0, 1.0, 1.0, 4.0, 1), (64, 1e4, 9, 1.0, 1.0, 4.0, 1), (64, 1e4, 1, 0.5, 1.0, 4.0, 1),
                 (2, 1e4, 2, 2.0, 1.0, 4.0, 1), (64, 1e4, 3, 2.0, 4.0, 1.0, 1), (64, 1e4, 3, 2.0, 0.0, 1.0, 1),
                 (64, 1e4, 4, 2.0, 1.0, 32.0, 0)):
        assert lib.gptq_q4_rope_freqs(*args, out, ctypes.byref(scale)) == bad, args
        assert q4.gptq_q4_last_error()
    assert lib.gptq_q4_rope_freqs(64, 1e4, 0, 1.0, 1.0, 4.0, 1, None, None) == bad
    assert not lib.gptq_q4_lora_make(60, 64, 1, 8, 0) and q4.gptq_q4_last_status() == bad
    assert not lib.gptq_q4_lora_make(64, 64, 1, 8, q4.GPTQ_Q4_DTYPE_FP32)
    assert q4.gptq_q4_last_status() == q4.GPTQ_Q4_UNSUPPORTED
    assert not lib.gptq_q4_attn_make(6, 4, 64, 16, 0) and q4.gptq_q4_last_status() == bad
    assert not lib.gptq_q4_attn_make(4, 4, 80, 16, 0) and q4.gptq_q4_last_status() == q4.GPTQ_Q4_UNSUPPORTED
    for name, n in (("lora_add", 10), ("lora_set", 7), ("attn_append", 9), ("attn_attend", 10)):
        f = getattr(lib, "gptq_q4_" + name)
        zero = [0 if t in (ctypes.c_int, ctypes.c_int64) else 0.0 if t in (ctypes.c_float, ctypes.c_double) else None
                for t in f.argtypes]
        assert len(zero) == n and f(*zero) == bad and "NULL" in q4.gptq_q4_last_error()
    lib.gptq_q4_lora_free(None)
    lib.gptq_q4_attn_free(None)
