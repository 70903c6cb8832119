"""gda_block_tables on launches of one, four and eight blocks, with refusals, in place and from a graph: every integer
equal to the plain sequential reference."""
import random

import pytest
import torch

import grouped_differential_attention_gb300 as gda
from oracle import ref_serving as R
from test_gpu_block_tables import case, i32, run

pytestmark = pytest.mark.gpu

# B, most pages of a sequence, page size, longest chunk, rows at least: the number of blocks goes by the rows
SIZES = [
    (64, 40, 16, 60, 1000),          # one block
    (64, 40, 16, 300, 9000),         # four
    (192, 2048, 16, 682, 40000),     # eight
    (7, 6000, 7, 9000, 17000),       # eight, few sequences
    (3000, 30, 1, 25, 17000),        # eight, pages of one row
]


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_differential_attention_gb300 import build
    build.build()


def rows_of(new, at_least):
    return max(sum(max(n, 0) for n in new) + 5, at_least)


@pytest.mark.parametrize("B,max_pages,page_size,chunk,at_least", SIZES)
def test_all_served(B, max_pages, page_size, chunk, at_least):
    lens, new, table, free, num = case(B, max_pages, page_size, chunk, seed=B)
    assert run(lens, new, table, free, len(free), page_size, num, rows_of(new, at_least)) == 0


@pytest.mark.parametrize("B,max_pages,page_size,chunk,at_least", SIZES)
def test_refusals(B, max_pages, page_size, chunk, at_least):
    """A short stack, lengths out of range, a page outside the pool in a table and in the stack, too few rows."""
    lens, new, table, free, num = case(B, max_pages, page_size, chunk, seed=B + 1, idle=0.0)
    rows = rows_of(new, at_least)
    need = sum(-(-(n + m) // page_size) - -(-n // page_size) for n, m in zip(lens, new))
    err = run(lens, new, table, free, max(need - need // 3 - 1, 0), page_size, num, rows)
    assert err & gda.GDA_DEVERR_NO_PAGES
    assert run(lens, new, table, free, len(free), page_size, num, max(1, sum(new) * 2 // 3)) == gda.GDA_DEVERR_BAD_LENGTH
    free[-1 - need // 2] = num                                  # a page off the stack that no pool has
    for b in [b for b, n in enumerate(lens) if n % page_size][:1]:   # the open page of a sequence, where there is one
        table[b][lens[b] // page_size] = num + 1
    assert run(lens, new, table, free, len(free), page_size, num, rows) == gda.GDA_DEVERR_BAD_PAGE
    lens[1], new[2] = -1, -3
    lens[B - 1], new[B - 1] = max_pages * page_size, 1
    err = run(lens, new, table, free, len(free), page_size, num, rows)
    assert err == gda.GDA_DEVERR_BAD_PAGE | gda.GDA_DEVERR_BAD_LENGTH


@pytest.mark.parametrize("B,max_pages,page_size,chunk,at_least", SIZES)
def test_lengths_and_count_in_place_over_replays(B, max_pages, page_size, chunk, at_least):
    """All blocks read the lengths and the count before one of them writes the new ones into the same memory; later
    replays run out of pages and of positions."""
    rnd = random.Random(B)
    lens, new = [rnd.randint(0, 3 * page_size) for _ in range(B)], [rnd.randint(0, chunk) for _ in range(B)]
    lens = [min(n, max_pages * page_size) for n in lens]
    rows = rows_of(new, at_least)
    held = [-(-n // page_size) for n in lens]
    need = sum(-(-(n + m) // page_size) - h for n, m, h in zip(lens, new, held))
    ids = list(range(sum(held) + need * 5 // 2))
    rnd.shuffle(ids)
    table = [[ids.pop() if j < h else -1 for j in range(max_pages)] for h in held]
    pages = len(ids) + sum(held)
    d_lens, d_new, d_table, d_free, d_count = i32(lens), i32(new), i32(table), i32(ids), i32([len(ids)])
    out = (i32([0] * rows), i32([0] * rows), i32([0] * (B + 1)), d_lens, d_count)
    gda.gda_device_error(clear=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gda.gda_block_tables(d_lens, d_new, d_table, d_free, d_count, page_size, pages, rows, out=out)
    count, cap, why = len(ids), max_pages * page_size, 0
    for step in range(4):
        graph.replay()
        before = lens
        slots, pos, starts, lens, count, table = R.block_tables(lens, new, table, ids, count, page_size, pages, rows)
        torch.cuda.synchronize()
        assert out[0].cpu().tolist() == slots and out[1].cpu().tolist() == pos, step
        assert out[2].cpu().tolist() == starts and d_lens.cpu().tolist() == lens and d_count.item() == count, step
        assert d_table.cpu().tolist() == table.tolist(), step
        for n, m, after in zip(before, new, lens):
            if n + m > cap:
                why |= gda.GDA_DEVERR_BAD_LENGTH
            elif after != n + m:
                why |= gda.GDA_DEVERR_NO_PAGES
    assert why and gda.gda_device_error(clear=True) == why
