"""Blocks chosen for each query on the GPU, exactly those of the reference in whole numbers and float32."""
import numpy as np
import pytest
import torch

import grouped_differential_attention_gb300 as gda
from oracle import ref_serving as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_differential_attention_gb300 import build
    build.build()


def make(B, most, hs, hn, d, block, lens, seed, page=0, coarse=False):
    """Bounds of `most` blocks a sequence; coarse: few distinct ones, so that scores tie."""
    g = torch.Generator().manual_seed(seed)
    per = page // block if page else most
    mp = -(-most // per)
    pages = B * mp + (2 if page else 0)
    bounds, scales = [], []
    for h in (hs, hn):
        shape = (pages, per, h, d)
        a = torch.randint(-1, 2, shape, generator=g) * 40 if coarse else torch.randint(-112, 113, shape, generator=g)
        b = a - (40 if coarse else torch.randint(0, 60, shape, generator=g))
        bounds.append(torch.stack((a, b.clamp(min=-128)), 3).to(torch.int8))
        scales.append(torch.exp2(torch.randint(-3, 3, (pages, per, h), generator=g).float()) if not coarse
                      else torch.ones(pages, per, h))
    if coarse:
        for t in bounds:                                   # whole blocks alike
            t[:, 1:] = t[:, :1]
    table = torch.randperm(pages, generator=g)[:B * mp].view(B, mp).to(torch.int32) if page else None
    return dict(q=[torch.randn(B, h, d, generator=g).bfloat16() for h in (hs, hn)], bounds=bounds, scales=scales,
                table=table, lens=torch.tensor(lens, dtype=torch.int32), block=block)


def run(c, keep, **kw):
    dev = lambda t: t.cuda() if t is not None else None
    return gda.gda_block_select(*map(dev, (*c["q"], *c["bounds"], *c["scales"], c["lens"])), c["block"], keep,
                                block_table=dev(c["table"]), **kw)


def check(c, keep, first=1, last=1):
    lists, counts = run(c, keep, first=first, last=last)
    want, n = R.block_select(*c["q"], [t.numpy() for t in c["bounds"]], [t.numpy() for t in c["scales"]],
                             None if c["table"] is None else c["table"].numpy(), c["lens"].tolist(), c["block"], keep, first,
                             last)
    assert counts.tolist() == n
    got = lists.tolist()
    for b, groups in enumerate(want):
        for g, ids in enumerate(groups):
            assert got[b][g] == ids + [-1] * (keep - len(ids)), (b, g, got[b][g], ids)


@pytest.mark.parametrize("page", [0, 1])
@pytest.mark.parametrize("hs,hn,d,block", [(1, 1, 64, 16), (3, 1, 64, 64), (12, 4, 64, 64), (16, 4, 128, 32), (7, 7, 128, 128),
                                           (40, 1, 64, 16)])
def test_shapes_and_lengths(hs, hn, d, block, page):
    lens = [1, 0, block - 1, block, block + 1, 9 * block, 39 * block + 3, 40 * block, 17 * block - 1]
    c = make(len(lens), 40, hs, hn, d, block, lens, seed=hs + d, page=page * 3 * block)
    gda.gda_device_error(clear=True)
    for keep, first, last in ((1, 0, 0), (1, 1, 0), (2, 0, 1), (7, 1, 1), (9, 4, 5), (39, 1, 2), (40, 0, 0), (64, 1, 1)):
        check(c, keep, first, last)
    assert gda.gda_device_error(clear=True) == 0


@pytest.mark.parametrize("keep", [1, 5, 130, 257])
def test_equal_scores_go_to_the_lowest(keep):
    check(make(3, 300, 6, 2, 64, 16, [300 * 16, 299 * 16, 280 * 16], seed=3, coarse=True), keep,
          first=min(1, keep - 1))


@pytest.mark.parametrize("amax", [1.0, 1.0546875, 1.2734375, 1.875, 1.8671875 * 2.0 ** -60, 1.4296875 * 2.0 ** 100])
def test_queries_between_two_whole_numbers(amax):
    """Elements that are odd multiples of amax / 254: q8 goes by the rounding of 127 * (1 / amax), in few blocks that
    differ in one unit of it."""
    c = make(1, 64, 3, 1, 64, 16, [64 * 16], seed=6, coarse=True)
    for i, q in enumerate(c["q"]):
        half = torch.tensor([amax, amax / 2, -amax / 2, amax / 4]).bfloat16().repeat(16)
        c["q"][i] = half.expand_as(q).clone()
        g = torch.Generator().manual_seed(i)
        c["bounds"][i] = torch.randint(-1, 2, c["bounds"][i].shape, generator=g).to(torch.int8)
    for keep in (5, 20):
        check(c, keep)


def test_many_blocks():
    c = make(2, 5000, 3, 1, 64, 16, [5000 * 16, 4097 * 16 - 5], seed=4)
    for keep in (3, 300, 4999):
        check(c, keep, 1, 2)


@pytest.mark.parametrize("hs,hn,d,most,lens", [
    (24, 1, 64, 3000, [48000, 16 * 2500 + 1]),     # x of all heads fits eight thread blocks
    (100, 1, 64, 4000, [16 * 3999 + 5]),           # and does not: two launches
    (6, 2, 128, 300, [4800, 4097, 16, 0, 4000]), (3, 1, 64, 1100, [16 * 1100, 16 * 9, 16 * 257, 16 * 256]),
    (6, 2, 64, 12, [192] * 90),
])
def test_every_way_through(hs, hn, d, most, lens):
    c = make(len(lens), most, hs, hn, d, 16, lens, seed=hs + most, page=48 if most < 1000 else 0)
    for keep in (1, 8, 200):
        check(c, keep, min(1, keep - 1), min(2, keep - 1) if keep > 2 else 0)


def test_the_most_blocks_of_a_sequence():
    """32768 blocks; keys chosen so that block j's share grows with a known order, above that of a flat noise head."""
    n = 32768
    c = make(1, n, 1, 1, 64, 16, [n * 16], seed=5)
    g = torch.Generator().manual_seed(6)
    order = torch.randperm(n, generator=g)
    c["bounds"][0].fill_(1)
    c["bounds"][1].fill_(0)
    c["scales"][0] = ((order.float() + 1) * 2.0 ** -20).view(1, n, 1)
    c["q"][0].fill_(1.0)
    lists, counts = run(c, 1000, first=0, last=0)
    assert counts.tolist() == [1000]
    assert lists[0, 0].tolist() == sorted(torch.argsort(order, descending=True)[:1000].tolist())


def test_heads_without_a_score():
    """Zero, tiny, infinite and NaN queries take no part; where none is left the lowest blocks stay."""
    c = make(4, 60, 3, 1, 64, 16, [60 * 16] * 4, seed=7)
    c["q"][0][0, 1] = 0
    c["q"][0][1, 2, 5] = float("nan")
    c["q"][1][1] = float("inf")
    c["q"][0][2] = 1e-38
    c["q"][0][3], c["q"][1][3] = 0, float("nan")
    check(c, 9)
    assert run(c, 4, first=0, last=1)[0][3, 0].tolist() == [0, 1, 2, 59]


def test_bounds_past_float32():
    """A head whose bounds on some block are infinite takes no part, one with blocks at minus infinity does."""
    c = make(2, 60, 3, 1, 64, 16, [60 * 16] * 2, seed=10)
    c["q"][0][0, 1] *= 2.0 ** 125
    c["q"][0][1, 2] = 2.0 ** 120
    c["bounds"][0][1, 5:, 2] = -100
    c["bounds"][0][1, :5, 2] = 0
    check(c, 9)
    check(c, 4, 0, 0)


def test_bad_lengths_and_pages_are_reported():
    c = make(3, 12, 3, 1, 64, 16, [12 * 16, 12 * 16 + 1, -4], seed=8, page=48)
    gda.gda_device_error(clear=True)
    lists, counts = run(c, 5)
    assert gda.gda_device_error(clear=True) == gda.GDA_DEVERR_BAD_LENGTH and counts.tolist() == [5, 5, 0]
    assert (lists[2] == -1).all()
    c["lens"][:] = 100
    c["table"][1, 1] = 99999
    run(c, 5)
    assert gda.gda_device_error(clear=True) == gda.GDA_DEVERR_BAD_PAGE
    c["table"][1, 3] = -1                                  # behind the seven blocks: not read
    c["table"][1, 1] = 0
    run(c, 5)
    assert gda.gda_device_error(clear=True) == 0


def test_outputs_of_the_caller_replayed_over_any_workspace():
    c = make(5, 50, 6, 2, 64, 32, [50 * 32, 3, 0, 49 * 32, 700], seed=9, page=64)
    dev = [t.cuda() for t in (*c["q"], *c["bounds"], *c["scales"], c["lens"], c["table"])]
    out = (torch.empty(5, 2, 8, dtype=torch.int32, device="cuda"), torch.empty(5, dtype=torch.int32, device="cuda"))
    ws = torch.full((5 * 50 * 8 * 4,), 0xFF, dtype=torch.uint8, device="cuda")
    want = [t.clone() for t in run(c, 8)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gda.gda_block_select(*dev[:7], 32, 8, block_table=dev[7], out=out, workspace=ws)
    for _ in range(2):
        for t in out:
            t.fill_(77)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_binding_refuses():
    c = make(2, 6, 4, 2, 64, 16, [90, 5], seed=1, page=32)
    good = [t.cuda() for t in (*c["q"], *c["bounds"], *c["scales"], c["lens"])]
    table = c["table"].cuda()
    for i, t in enumerate(good):
        for other in (t.cpu(), t.double(), t[:, :1] if t.dim() > 1 else t[:1]):
            bad = list(good)
            bad[i] = other
            with pytest.raises((TypeError, ValueError, gda.GDAError)):
                gda.gda_block_select(*bad, 16, 2, block_table=table)
    for kw in (dict(first=2, last=1), dict(first=-1), dict(last=-1), dict(block_table=table.long()),
               dict(block_table=table[:1]), dict(block_table=None)):
        with pytest.raises((TypeError, ValueError, gda.GDAError)):
            gda.gda_block_select(*good, 16, 2, **(dict(block_table=table) | kw))
    for block, keep in ((24, 2), (8, 2), (16, 0), (0, 2), (256, 2)):
        with pytest.raises((ValueError, gda.GDAError, RuntimeError)):
            gda.gda_block_select(*good, block, keep, block_table=table, first=0, last=0)
