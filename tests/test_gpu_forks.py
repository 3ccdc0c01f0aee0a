"""Fresh pages of forks that do not use them: fresh[i] is not looked at where the parent's last page is full."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from paged4 import no_handles_left, refused  # noqa: E402, F401

DEV = "cuda:0"
PAGE = 16


@pytest.fixture(scope="module")
def q4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gptq_bit_weight_gb300 as q4mod
    return q4mod


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# rows' lengths, parents, children, fresh pages, which forks are done
CASES = {
    "full_then_part": ([32, 5, 20, 0, 0], [0, 2], [3, 4], [50, 50], [True, True]),
    "part_then_full": ([32, 5, 20, 0, 0], [2, 0], [3, 4], [50, 50], [True, True]),
    "empty_then_part": ([0, 5, 20, 0, 0], [0, 2], [3, 4], [50, 50], [True, True]),
    "full_part_part": ([32, 5, 20, 0, 0, 0], [0, 2, 1], [3, 4, 5], [50, 50, 50], [True, True, False]),
    "part_full_part": ([32, 5, 20, 0, 0, 0], [1, 0, 2], [3, 4, 5], [50, 50, 50], [True, True, False]),
    "all_full": ([32, 16, 0, 1, 1, 1], [0, 1, 2], [3, 4, 5], [7, 7, 7], [True, True, True]),
    "no_fork_then_part": ([32, 5, 20, 0, 0], [-1, 2], [3, 4], [50, 50], [True, True]),
    "no_row_then_part": ([32, 5, 20, 0, 0], [99, 2], [3, 4], [50, 50], [False, True]),
    "no_length_then_part": ([-3, 5, 20, 0, 0], [0, 2], [3, 4], [50, 50], [False, True]),
    "too_long_then_part": ([1000, 5, 20, 0, 0], [0, 2], [3, 4], [50, 50], [False, True]),
}


@pytest.mark.parametrize("case", list(CASES))
def test_a_fresh_page_that_an_earlier_fork_does_not_use(q4, case):
    lens, parent, child, fresh, done = CASES[case]
    kv = torch.randint(0, 256, (64, 2, PAGE, 160), dtype=torch.uint8, generator=torch.Generator().manual_seed(1))
    cache = q4.PagedCache4(kv.to(DEV), 128)
    pool = q4.PagePool([cache])
    table = torch.arange(2 * len(lens), dtype=torch.int32).view(-1, 2)
    on_gpu, lengths = table.to(DEV), ints(*lens)
    pool.fork(on_gpu, lengths, ints(*parent), ints(*child), ints(*fresh))
    want, contents, n = table.clone(), kv.clone(), list(lens)
    for p, c, f, ok in zip(parent, child, fresh, done):
        if not ok or p < 0:
            continue
        pages, part = -(-lens[p] // PAGE), lens[p] % PAGE
        row = table[p, :pages].tolist()
        if part:
            contents[f] = kv[row[-1]]
            row[-1] = f
        want[c] = -1
        want[c, :pages] = torch.tensor(row, dtype=torch.int32)
        n[c] = lens[p]
    assert torch.equal(on_gpu.cpu(), want) and lengths.tolist() == n
    assert torch.equal(cache.kv.cpu(), contents)
    if all(done):
        pool.device_error()
    else:
        assert refused(q4, pool.device_error, q4.GPTQ_Q4_DEVICE_FAULT)
