"""The 8-bit block cache's calls inside graphs with other kinds of work, and at the most heads and sequences."""
import pytest
import torch

import grouped_differential_attention_gb300 as gda
from grouped_differential_attention_gb300 import workloads as W
from tests.test_gpu_block_select import check as check_select
from tests.test_gpu_block_select import make as make_select
from tests.test_gpu_decode_fp8_block import check, make, pick, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_differential_attention_gb300 import build
    build.build()


@pytest.mark.parametrize("T", [40, 1100])
def test_in_a_graph_behind_copies_fills_and_other_streams(T):
    """Each call captured right behind a copy, a fill, and the end of another stream's work that it depends on."""
    B, hs, hn, d, dv, Lcap, block, keep = 2, 6, 2, 64, 128, 1280, 64, 3
    g = torch.Generator(device="cuda").manual_seed(T)
    dims = ((hs, d), (hn, d), (hs, dv))
    source = [torch.randn(T, h, n, generator=g, device="cuda").bfloat16() for h, n in dims]
    rows = [torch.zeros_like(t) for t in source]
    slots = torch.cat((torch.arange(T - 20), Lcap + torch.arange(20))).to(torch.int32).cuda()
    q = [torch.randn(B, h, d, generator=g, device="cuda").bfloat16() for h in (hs, hn)]
    lens0 = torch.tensor([T - 20, 20], dtype=torch.int32, device="cuda")
    lam0 = torch.full((hs,), 0.5, device="cuda")
    cache, bounds = W.empty_fp8_block_cache(B, Lcap, block, hs, hn, d, dv, "cuda")
    lens, lam, slot = torch.zeros_like(lens0), torch.zeros_like(lam0), torch.full_like(slots, -1)
    side = torch.cuda.Stream()

    def work():
        main = torch.cuda.current_stream()
        for a, b in zip(rows, source):
            a.copy_(b)                                       # a copy of memory
        side.wait_stream(main)
        with torch.cuda.stream(side):
            slot.copy_(slots)
        main.wait_stream(side)                               # the other stream's end
        gda.gda_cache_append_fp8_block(*rows, slot, *cache, k_sig_bounds=bounds[0], k_noise_bounds=bounds[1])
        side.wait_stream(main)
        with torch.cuda.stream(side):
            back = gda.gda_cache_read_fp8_block(slot, *cache)
            lens.copy_(lens0)
        main.wait_stream(side)
        lists = gda.gda_block_select(*q, *bounds, *cache[3:5], lens, block, keep)
        lam.zero_()                                          # a fill of memory
        lam.copy_(lam0)
        some = gda.gda_attn_decode_sparse_fp8_block(*q, *cache, *lists, lens, lam, 0.8)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            whole = gda.gda_attn_decode_fp8_block(*q, *cache, lens, lam, 0.8)
        main.wait_stream(side)
        return (*back, *lists, some, whole)

    def forget():
        for t in (*rows, lens, lam, *cache, *bounds):
            t.view(torch.uint8).zero_()
        slot.fill_(-1)
        torch.cuda.synchronize()

    want = [t.clone() for t in work()]
    held = [t.clone() for t in (*cache, *bounds)]
    c = dict(q1=q[0], q2=q[1], pools=cache[:3], scales=cache[3:], table=None, lam=lam0, block=block, lens=lens0, lists=None)
    check(want[6], c)
    check(want[5], c | {"lists": (want[3], want[4])})
    graph = torch.cuda.CUDAGraph()
    forget()
    with torch.cuda.graph(graph):
        got = work()
    for _ in range(3):
        forget()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip((*cache, *bounds), held))


@pytest.mark.parametrize("hs,hn,d,dv", [(127, 1, 64, 128), (64, 64, 64, 64), (126, 2, 128, 256), (100, 25, 64, 128)])
def test_the_most_heads(hs, hn, d, dv):
    c = make(3, 160, hs, hn, d, dv, [160, 0, 77], seed=hs, page=80, block=16)
    check(run(c), c)
    c["lists"] = pick(c, 4, seed=hs)
    check(run(c), c)
    check_select(make_select(2, 12, hs, hn, d, 16, [12 * 16, 9 * 16 - 3], seed=hs, page=48), 4)


def test_the_most_sequences():
    """65535 sequences over the pages of a few; every 997th of them is checked."""
    B, hs, hn = 65535, 2, 1
    c = make(4, 96, hs, hn, 64, 64, [96] * 4, seed=3, page=32, block=16)
    g = torch.Generator(device="cuda").manual_seed(4)
    c["q1"], c["q2"] = (torch.randn(B, h, 64, generator=g, device="cuda").bfloat16() for h in (hs, hn))
    c["lens"] = (torch.arange(B, device="cuda") * 7 % 97).to(torch.int32)
    c["table"] = torch.randint(0, c["pools"][0].shape[0], (B, 3), generator=g, device="cuda", dtype=torch.int32)
    some = torch.arange(0, B, 997, device="cuda")
    few = {k: c[k][some].contiguous() for k in ("q1", "q2", "lens", "table")}
    check(run(c)[some], c | few)
    bounds = [torch.randint(-112, 113, (*c["scales"][i].shape, 2, 64), generator=g, device="cuda").to(torch.int8) for i in (0, 1)]
    lists = gda.gda_block_select(c["q1"], c["q2"], *bounds, *c["scales"][:2], c["lens"], 16, 2, block_table=c["table"])
    c["lists"] = lists
    check(run(c)[some], c | few | {"lists": tuple(t[some] for t in lists)})
    one = dict(q=[few["q1"].cpu(), few["q2"].cpu()], bounds=[t.cpu() for t in bounds], scales=[t.cpu() for t in c["scales"][:2]],
               table=few["table"].cpu(), lens=few["lens"].cpu(), block=16)
    check_select(one, 2)
    again = gda.gda_block_select(few["q1"], few["q2"], *bounds, *c["scales"][:2], few["lens"], 16, 2, block_table=few["table"])
    assert torch.equal(again[0], lists[0][some]) and torch.equal(again[1], lists[1][some])


@pytest.mark.parametrize("d,dv", [(64, 64), (64, 128), (64, 256), (128, 64), (128, 128), (128, 256)])
@pytest.mark.parametrize("hs,hn", [(1, 1), (3, 1), (4, 2), (12, 4), (5, 1), (7, 7), (16, 4)])
def test_short_lengths_in_caches_that_may_be_long(hs, hn, d, dv):
    """The same rows where the block table and the lists leave room for many more: what is chosen by the room alone."""
    lens = [1, 0, 15, 16, 17, 33, 64, 128, 200, 7]
    c = make(len(lens), 208, hs, hn, d, dv, lens, seed=hs + d + dv, page=48, powers=hs != 4)
    room = {"table": torch.cat((c["table"], torch.zeros(len(lens), 3000, dtype=torch.int32, device="cuda")), 1).contiguous()}
    check(run(c | room), c)
    ids, counts = pick(c, 5, seed=hs)
    wide = torch.cat((ids, torch.full((*ids.shape[:2], 9000), -1, dtype=torch.int32, device="cuda")), 2).contiguous()
    check(run(c | {"lists": (wide, counts)}), c | {"lists": (ids, counts)})
    check(run(c | {"lists": (ids, counts)}), c | {"lists": (ids, counts)})


@pytest.mark.parametrize("B,Lcap", [(1, 128), (1, 1100), (1, 3000), (3, 700), (5, 2100), (17, 600), (40, 1000), (130, 300), (300, 100)])
def test_lengths_up_to_the_room(B, Lcap):
    """Batches from one sequence to many, whole and over lists, as one launch or two would take them."""
    lens = [Lcap - (13 * b) % Lcap for b in range(B)]
    c = make(B, Lcap, 6, 2, 64, 128, lens, seed=B, block=16)
    check(run(c), c)
    c["lists"] = pick(c, -(-Lcap // 32), seed=B)
    check(run(c), c)


def with_room(c, listed=False):
    """The same call over a block table (or lists) with room for many more."""
    table = torch.cat((c["table"], torch.zeros(c["table"].shape[0], 3000, dtype=torch.int32, device="cuda")), 1).contiguous()
    if not listed:
        return c | {"table": table}
    ids, counts = c["lists"]
    return c | {"table": table, "lists": (torch.cat((ids, torch.full((*ids.shape[:2], 9000), -1, dtype=torch.int32,
                                                                     device="cuda")), 2).contiguous(), counts)}


@pytest.mark.parametrize("listed", [False, True])
def test_bad_rows_pages_and_workspaces_where_there_is_room(listed):
    lens = [1, 0, 15, 17, 96, 130, 47]
    c = make(len(lens), 160, 6, 2, 64, 128, lens, seed=5, page=32, block=16)
    if listed:
        c["lists"] = pick(c, 4, seed=5)
    ws = torch.full((gda.gda_attn_decode_fp8_block_workspace_size(7, 6, 2, 64, 128),), 0xFF, dtype=torch.uint8, device="cuda")
    want = run(with_room(c, listed), workspace=ws).clone()
    check(want, c)
    assert torch.equal(run(with_room(c, listed), workspace=ws), want) and torch.equal(run(with_room(c, listed)), want)
    used = torch.zeros(c["pools"][0].shape[:2], dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        for j in range(n):
            used[c["table"][b, j // 32].long(), j % 32] = True
    clean = [t.clone() for t in (*c["pools"], *c["scales"])]
    for p, s in zip(c["pools"], c["scales"]):
        p[~used] = 0x7F
        s[~used.view(used.shape[0], -1, 16).any(-1)] = float("nan")
    assert torch.equal(run(with_room(c, listed)), want)
    c["pools"], c["scales"] = clean[:3], clean[3:]
    gda.gda_device_error(clear=True)
    c["lens"][4] = -4
    out = run(with_room(c, listed))
    assert gda.gda_device_error(clear=True) == gda.GDA_DEVERR_BAD_LENGTH
    c["lens"][4] = 0
    check(out, c)
    c["lens"][4], c["table"][5, 1], c["table"][4, 0] = 96, 10 ** 9, -1
    if listed:                                               # the pages in question are among the chosen ones
        c["lists"][0][4:6] = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
        c["lists"][1][4:6] = 4
    out = run(with_room(c, listed))
    assert gda.gda_device_error(clear=True) == gda.GDA_DEVERR_BAD_PAGE
    pages = c["pools"][0].shape[0]
    check(out, c | {"table": torch.where((c["table"] >= 0) & (c["table"] < pages), c["table"], 0)})


@pytest.mark.parametrize("d,dv", [(64, 64), (64, 128), (64, 256), (128, 64), (128, 128), (128, 256)])
@pytest.mark.parametrize("hs,hn", [(1, 1), (2, 1), (3, 1), (5, 1), (8, 4)])
def test_one_sequence_of_each_shape(hs, hn, d, dv):
    """The largest clusters, with the most shared memory."""
    for n in (16 * 128, 1999):
        c = make(1, 2048, hs, hn, d, dv, [n], seed=n, block=32)
        check(run(c), c)
        c["lists"] = pick(c, 40, seed=n)
        check(run(c), c)
