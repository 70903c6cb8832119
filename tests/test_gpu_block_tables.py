"""gda_block_tables on the GPU against the plain sequential reference: every integer equal."""
import random

import pytest
import torch

import grouped_differential_attention_gb300 as gda
from oracle import ref_serving as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_differential_attention_gb300 import build
    build.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def case(B, max_pages, page_size, chunk, seed, spare=3, idle=0.2):
    rnd = random.Random(seed)
    cap = max_pages * page_size
    new = [0 if rnd.random() < idle else rnd.randint(1, min(chunk, cap)) for _ in range(B)]
    lens = [rnd.choice([0, cap - n, rnd.randint(0, cap - n)]) for n in new]
    num_pages = B * max_pages + spare
    ids = list(range(num_pages))
    rnd.shuffle(ids)
    table = [[ids[b * max_pages + j] if j * page_size < lens[b] else -7 for j in range(max_pages)] for b in range(B)]
    used = {p for row in table for p in row if p >= 0}
    free = [p for p in ids if p not in used]
    return lens, new, table, free, num_pages


def run(lens, new, table, free, count, page_size, num_pages, max_rows):
    t = i32(table)
    gda.gda_device_error(clear=True)
    out = gda.gda_block_tables(i32(lens), i32(new), t, i32(free), i32([count]), page_size, num_pages, max_rows)
    err = gda.gda_device_error(clear=True)
    ref = R.block_tables(lens, new, table, free, min(max(count, 0), len(free)), page_size, num_pages, max_rows)
    for name, a, b in zip(("slots", "positions", "starts", "lens", "left"), out, ref):
        assert a.cpu().tolist() == (b if isinstance(b, list) else [b]), name
    assert t.cpu().tolist() == ref[5].tolist()
    return err


@pytest.mark.parametrize("B,max_pages,page_size,chunk", [
    (1, 1, 1, 1), (1, 9, 16, 100), (3, 5, 7, 1), (64, 8, 64, 1), (33, 40, 16, 300), (1000, 3, 16, 1),
    (1025, 6, 1, 4), (5, 700, 3, 2000), (8192, 2, 4, 2),
])
def test_matches_the_sequential_reference(B, max_pages, page_size, chunk):
    lens, new, table, free, num = case(B, max_pages, page_size, chunk, seed=B + chunk)
    assert run(lens, new, table, free, len(free), page_size, num, sum(new) + 13) == 0
    assert run(lens, new, table, free, len(free), page_size, num, max(1, sum(new))) == 0


@pytest.mark.parametrize("count", [0, 1, 5, 17])
def test_a_short_stack_refuses_in_order(count):
    lens, new, table, free, num = case(40, 6, 8, 30, seed=count)
    err = run(lens, new, table, free, count, 8, num, sum(new))
    assert err & gda.GDA_DEVERR_NO_PAGES


def test_lengths_and_rows_out_of_range_are_refused():
    lens, new, table, free, num = case(12, 4, 8, 6, seed=2, idle=0.0)
    lens[3], new[5], lens[7], new[7] = -1, -4, 31, 2         # 33 of 32 positions
    assert run(lens, new, table, free, len(free), 8, num, 60) & gda.GDA_DEVERR_BAD_LENGTH
    lens, new, table, free, num = case(12, 4, 8, 6, seed=3, idle=0.0)
    assert run(lens, new, table, free, len(free), 8, num, sum(new) - 1) & gda.GDA_DEVERR_BAD_LENGTH


def test_bad_page_ids_and_counts_are_reported():
    lens, new, table, free, num = case(6, 4, 8, 6, seed=4, idle=0.0)
    lens[2] = 9
    table[2][1] = num
    assert run(lens, new, table, free, len(free), 8, num, sum(new)) == gda.GDA_DEVERR_BAD_PAGE
    lens, new, table, free, num = case(6, 4, 8, 6, seed=5, idle=0.0)
    assert run(lens, new, table, free, len(free) + 3, 8, num, sum(new)) == gda.GDA_DEVERR_BAD_PAGE


def test_long_sums_do_not_wrap():
    """Lengths whose sum passes 32 bits: all but the first refused, nothing written for them."""
    B = 6
    new = [5] + [2 ** 31 - 6] * (B - 1)
    gda.gda_device_error(clear=True)
    t = i32([[-1]] * B)
    out = gda.gda_block_tables(i32([0] * B), i32(new), t, i32([3, 2, 1, 0]), i32([4]), 16, 4, 16)
    assert gda.gda_device_error(clear=True) == gda.GDA_DEVERR_BAD_LENGTH
    assert out[0].cpu().tolist() == [0, 1, 2, 3, 4] + [-1] * 11
    assert out[3].cpu().tolist() == [5, 0, 0, 0, 0, 0] and out[4].item() == 3
    assert out[2].cpu().tolist()[:3] == [0, 5, 2 ** 31 - 1] and out[2].cpu().tolist()[-1] == 2 ** 31 - 1
    assert t.cpu().tolist() == [[0]] + [[-1]] * 5


@pytest.mark.parametrize("chunk,max_rows", [(1, 64), (400, 9000)])
def test_steps_in_place_and_replayed_from_a_graph(chunk, max_rows):
    """Lengths, table and stack updated in place: three replays equal three steps of the reference."""
    rnd = random.Random(chunk)
    B, max_pages, ps = 24, 80, 16
    lens, new = [rnd.randint(0, 50) for _ in range(B)], [rnd.randint(0, chunk) for _ in range(B)]
    ids = list(range(B * max_pages))
    rnd.shuffle(ids)
    table = [[ids.pop() if j * ps < lens[b] else -1 for j in range(max_pages)] for b in range(B)]
    d_lens, d_new, d_table, d_free, d_count = i32(lens), i32(new), i32(table), i32(ids), i32([len(ids)])
    out = (i32([0] * max_rows), i32([0] * max_rows), i32([0] * (B + 1)), d_lens, d_count)
    gda.gda_device_error(clear=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gda.gda_block_tables(d_lens, d_new, d_table, d_free, d_count, ps, B * max_pages, max_rows, out=out)
    count = len(ids)
    for _ in range(3):
        graph.replay()
        slots, pos, starts, lens, count, table = R.block_tables(lens, new, table, ids, count, ps, B * max_pages, max_rows)
        torch.cuda.synchronize()
        assert out[0].cpu().tolist() == slots and out[1].cpu().tolist() == pos
        assert d_lens.cpu().tolist() == lens and d_count.item() == count
        assert d_table.cpu().tolist() == table.tolist()
    assert gda.gda_device_error(clear=True) == 0


def test_binding_refuses():
    a = (i32([1, 2]), i32([1, 1]), i32([[0], [1]]), i32([2, 3]), i32([2]))
    for i in range(5):
        bad = list(a)
        bad[i] = bad[i].long()
        with pytest.raises((TypeError, ValueError)):
            gda.gda_block_tables(*bad, 16, 4, 8)
    with pytest.raises(gda.GDAError):
        gda.gda_block_tables(*a, 0, 4, 8)
    with pytest.raises(gda.GDAError):
        gda.gda_block_tables(*a, 1 << 30, 4, 8)                       # slots pass 31 bits
    for sizes in ((1 << 32) + 16, 4, 8), (16, (1 << 32) + 4, 8), (16, 4, (1 << 32) + 8):
        with pytest.raises(ValueError):                               # not their low 32 bits
            gda.gda_block_tables(*a, *sizes)
