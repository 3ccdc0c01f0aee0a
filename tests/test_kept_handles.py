"""Handles that are kept for later, without a GPU: what is freed, and when another thread empties the list meanwhile."""
import pytest

pytest.importorskip("torch")


@pytest.fixture(scope="module")
def q4():
    import __graft_entry__
    import os
    b = __graft_entry__._cuda_build_module()
    if not os.path.exists(b.LIB):
        b.build()
    import gptq_bit_weight_gb300 as q4mod
    return q4mod


class Emptied(list):
    """A list that another thread empties after it was seen to hold something."""

    def __bool__(self):
        return True

    def __len__(self):
        return 1


def test_kept_handles_are_freed(q4, monkeypatch):
    freed = []
    monkeypatch.setattr(q4, "_kept", [(freed.append, 1), (freed.append, 2)])
    q4._release(freed.append, 3)
    assert sorted(freed) == [1, 2, 3] and not q4._kept
    q4._release()
    assert len(freed) == 3


def test_another_thread_frees_the_last(q4, monkeypatch):
    monkeypatch.setattr(q4, "_kept", Emptied())
    q4._release()
    freed = []
    q4._release(freed.append, 7)
    assert freed == [7]
