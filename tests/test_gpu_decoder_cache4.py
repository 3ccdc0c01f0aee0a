"""The example's decoder step over a cache of 4 bits and through a window with first tokens: it runs, in a captured
graph, and its lengths and outputs are there (the example checks them)."""
import gc
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("bits,window,sinks", [(4, 0, 0), (4, 100, 4), (16, 100, 4)])
def test_example(bits, window, sinks):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import decoder_attention
    gc.collect()                     # no handle of an earlier test is freed while the step is captured
    x = decoder_attention.main(q_heads=16, kv_heads=2, head_dim=64, page_size=16, prompts=(150, 7, 33), decoded=8, bits=bits,
                               window=window, sinks=sinks)
    assert x.shape == (3, 1024) and torch.isfinite(x).all()
