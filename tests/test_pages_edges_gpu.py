"""The page pool on the GPU: tables and lengths that break its rules."""
import pytest
import torch

pytestmark = pytest.mark.gpu

from mla_attention_prolog_gb300 import binding  # noqa: E402
from test_pages_gpu import FULL, PAGE, SEQ, i32  # noqa: E402

PAGES, SIZE, WIDTH = 40, 64, 4
# -1, the first page behind the pool, and one whose slot is 320 in 32 bits
BAD = [-1, PAGES, (1 << 26) + 5, -(1 << 31)]


def pool_of(rows, lens, taken):
    table = torch.full((len(rows), WIDTH), -1, dtype=torch.int32)
    for s, row in enumerate(rows):
        table[s, :len(row)] = torch.tensor(row, dtype=torch.int32)
    refs = torch.zeros(PAGES, dtype=torch.int32)
    refs[taken] = 1
    table, refs, lens, status = table.cuda(), refs.cuda(), i32(*lens), i32(0)
    return binding.PagePool(table, lens, refs, SIZE, status), table, lens, refs, status


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("count", [1, 59, 60, 1500])
def test_extend_behind_a_page_that_is_none(bad, count):
    """The tokens that would lie in it get no slot; those of new pages do."""
    width = 40
    table = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
    table[0, 0], table[1, 0] = bad, 7
    lens, refs, status = i32(5, 5), torch.zeros(PAGES, dtype=torch.int32, device="cuda"), i32(0)
    refs[7] = 1
    total = 2 * count
    slots, pos = torch.full((total,), 99, dtype=torch.int32, device="cuda"), torch.zeros(total, dtype=torch.int32, device="cuda")
    binding.PagePool(table, lens, refs, SIZE, status).extend(i32(0, 1), i32(count, count), slots, pos)
    need = -(-(5 + count) // SIZE) - 1
    fits = 2 * need <= PAGES - 1
    free = [p for p in range(PAGES) if p != 7]
    want = []
    for s in range(2):
        pages = [bad if s == 0 else 7] + free[s * need:(s + 1) * need]
        if s == 1 and not fits:
            want += [-1] * count
            continue
        want += [-1 if pages[j // SIZE] == bad else pages[j // SIZE] * SIZE + j % SIZE for j in range(5, 5 + count)]
    assert slots.tolist() == want
    assert int(status) == PAGE | (0 if fits else FULL)
    assert lens.tolist() == [5 + count, 5 + count if fits else 5]
    assert int(table[0, 0]) == bad


@pytest.mark.parametrize("bad", BAD)
def test_fork_of_a_last_page_that_is_none(bad):
    """The child gets a page of its own and no copy is due; the other child's is."""
    pool, table, lens, refs, status = pool_of([[3, bad], [4, 5], [], []], [70, 70, 0, 0], [3, 4, 5])
    src, dst = i32(9, 9), i32(9, 9)
    pool.fork(i32(0, 1), i32(2, 3), src, dst)
    assert int(status) == PAGE
    assert src.tolist() == [-1, 5] and dst.tolist() == [-1, 1]
    assert table.tolist() == [[3, bad, -1, -1], [4, 5, -1, -1], [3, 0, -1, -1], [4, 1, -1, -1]]
    assert lens.tolist() == [70, 70, 70, 70]
    assert refs[:6].tolist() == [1, 1, 0, 2, 2, 1]


@pytest.mark.parametrize("length,cut", [(-3, 0), (-(1 << 31), 0), (WIDTH * SIZE + 1, WIDTH * SIZE), ((1 << 31) - 1, WIDTH * SIZE)])
def test_lengths_outside_the_table_are_cut_and_reported(length, cut):
    row = [2, 3, 4, 5]
    pool, table, lens, refs, status = pool_of([row], [length], row)
    slots = i32(9)
    pool.extend(i32(0), i32(1), slots)
    if cut:
        assert int(status) == SEQ | FULL and slots.tolist() == [-1] and lens.tolist() == [length]
    else:
        assert int(status) == SEQ and slots.tolist() == [0] and lens.tolist() == [1] and table.tolist() == [[0, 3, 4, 5]]

    pool, table, lens, refs, status = pool_of([row, []], [length, 0], row)
    pool.fork(i32(0), i32(1), i32(9), i32(9))
    assert int(status) == SEQ and lens.tolist() == [length, cut]
    assert table[1].tolist() == (row if cut else [-1] * WIDTH)
    assert refs[2:6].tolist() == [2 if cut else 1] * 4

    pool, table, lens, refs, status = pool_of([row], [length], row)
    pool.release(i32(0, 0))
    assert int(status) == SEQ and lens.tolist() == [0] and table.tolist() == [[-1] * WIDTH]
    assert refs[2:6].tolist() == [0 if cut else 1] * 4
