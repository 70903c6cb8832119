"""Decodes over an 8-bit cache with block scales, contiguous, paged and over listed blocks, against float64.

Tolerance.  With S the sum of absolute terms of a row's largest score (in
units of the exponent of 2), a score is off by less than 2^-19 (1 + S): its
products are exact, and a score of 128 terms passes through at most 16 float32
sums and products.  exp2, the sums of weights and values and the norm add less
than 2^-19 together.  So a weight is off by 2^-18 (1 + S) of itself, and an
output element before the norm by as much of mag, the sum of its absolute
terms, and by 2^-39 for each position of its map's largest weight times the
largest value (weights kept in two f16 numbers, the steps of whose smallest are
2^-24 where the largest is 2^15); the norm's factor by the row's share of that,
and the bf16 result by half a step, 2^-8 of itself.
"""
import math

import pytest
import torch

import grouped_differential_attention_gb300 as gda

pytestmark = pytest.mark.gpu
LAM0 = 0.8


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_differential_attention_gb300 import build
    build.build()


def make(B, Lcap, hs, hn, d, dv, lens, seed, block=16, page=0, powers=True, spread=1.0):
    """Codes of normal values and scales that differ from block to block, powers of two or any."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    size = page or -(-Lcap // block) * block
    mp = -(-Lcap // size)
    pages = B * mp + (2 if page else 0)
    pools, scales = [], []
    for h, n in ((hs, d), (hn, d), (hs, dv)):
        x = torch.randn(pages, size, h, n, generator=g, device="cuda") * 60
        pools.append(x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
        e = 2 * torch.rand(pages, size // block, h, generator=g, device="cuda")
        scales.append(spread * torch.exp2((e.floor() if powers else e) - 7))
    table = torch.randperm(pages, generator=g, device="cuda")[:B * mp].view(B, mp).to(torch.int32).contiguous() if page else None
    q1, q2 = (torch.randn(B, h, d, generator=g, device="cuda").bfloat16() for h in (hs, hn))
    lam = 0.2 + 0.6 * torch.rand(hs, generator=g, device="cuda")
    return dict(q1=q1, q2=q2, pools=pools, scales=scales, table=table, lam=lam, block=block, lists=None,
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))


def run(c, **kw):
    head = (c["q1"], c["q2"], *c["pools"], *c["scales"])
    if c["lists"] is not None:
        return gda.gda_attn_decode_sparse_fp8_block(*head, *c["lists"], c["lens"], c["lam"], LAM0,
                                                    block_table=c["table"], **kw)
    if c["table"] is None:
        return gda.gda_attn_decode_fp8_block(*head, c["lens"], c["lam"], LAM0, **kw)
    return gda.gda_attn_decode_paged_fp8_block(*head, c["table"], c["lens"], c["lam"], LAM0, **kw)


def rms(t):
    return (t * t).mean(-1, keepdim=True).sqrt()


def check(got, c, eps=1e-5):
    """Every element of the output within the bound of the definition in float64, one sequence and head at a time."""
    hs, hn, d, dv = c["q1"].shape[1], c["q2"].shape[1], c["q1"].shape[2], c["pools"][2].shape[3]
    r, bl, size = hs // hn, c["block"], c["pools"][0].shape[1]
    rows = [p.view(torch.uint8).flatten(0, 1).view(torch.float8_e4m3fn).float().double() if p.numel() < 1 << 28 else None
            for p in c["pools"]]
    scales = [s.double().flatten(0, 1) for s in c["scales"]]

    def value(i, at, h):
        code = rows[i][at, h] if rows[i] is not None else \
            c["pools"][i].view(torch.uint8).flatten(0, 1)[at, h].view(torch.float8_e4m3fn).float().double()
        return code * scales[i][at // bl, h][:, None]

    worst = 0.0
    for b, n in enumerate(c["lens"].tolist()):
        for g in range(hn):
            pos = torch.arange(n, device="cuda")
            if c["lists"] is not None:
                ids = c["lists"][0][b, g, :int(c["lists"][1][b])].long()
                pos = (ids[ids >= 0][:, None] * bl + torch.arange(bl, device="cuda")).flatten()
                pos = pos[pos < n]
            if pos.numel() == 0:
                assert (got[b, g * r:g * r + r] == 0).all()
                continue
            page = c["table"][b].long()[pos // size] if c["table"] is not None else torch.full_like(pos, b)
            at = page * size + pos % size
            k2 = value(1, at, g)
            x2, s2 = k2 @ c["q2"][b, g].double() / d ** 0.5, (k2.abs() @ c["q2"][b, g].double().abs()).max() / d ** 0.5
            a2 = torch.softmax(x2, 0)
            for h in range(g * r, g * r + r):
                k1, v = value(0, at, h), value(2, at, h)
                x1, s1 = k1 @ c["q1"][b, h].double() / d ** 0.5, (k1.abs() @ c["q1"][b, h].double().abs()).max() / d ** 0.5
                a1, lam = torch.softmax(x1, 0), c["lam"][h].double()
                o = (a1 - lam * a2) @ v
                off = 0
                for a, w, s in ((a1, 1.0, s1), (a2, lam.abs(), s2)):
                    off = off + w * (2.0 ** -18 * (1 + s / math.log(2)) * (a @ v.abs())
                                     + pos.numel() * 2.0 ** -39 * a.max() * v.abs().max())
                f = (1 - LAM0) / torch.sqrt((o * o).mean() + eps)
                ref = f * o
                bound = 2.0 ** -8 * ref.abs() + f * off + ref.abs() * rms(off) / torch.sqrt((o * o).mean() + eps)
                err = (got[b, h].double() - ref).abs()
                worst = max(worst, float((err / bound.clamp(min=1e-300)).max()))
    assert worst <= 1.0, worst


SHAPES = [(64, 64), (64, 128), (64, 256), (128, 64), (128, 128), (128, 256)]


@pytest.mark.parametrize("page", [0, 48])
@pytest.mark.parametrize("d,dv", SHAPES)
@pytest.mark.parametrize("hs,hn", [(1, 1), (3, 1), (4, 2), (12, 4), (5, 1), (7, 7), (16, 4)])
def test_shapes_and_edge_lengths(hs, hn, d, dv, page):
    lens = [1, 0, 15, 16, 17, 33, 64, 128, 200, 7]
    c = make(len(lens), 208, hs, hn, d, dv, lens, seed=hs * 7 + d + dv, page=page, powers=hs != 4)
    gda.gda_device_error(clear=True)
    out = run(c)
    assert gda.gda_device_error(clear=True) == 0
    check(out, c)
    assert (out[1] == 0).all()


@pytest.mark.parametrize("B,lens,page,block", [
    (1, [1], 0, 16), (1, [5000], 64, 64), (1, [40000], 128, 128), (3, [0, 9001, 0], 96, 32), (70, None, 16, 16),
    (300, None, 32, 16), (2, [0, 0], 16, 16), (5, [0, 0, 3, 0, 4097], 0, 128),
])
def test_batches_long_short_and_empty(B, lens, page, block):
    if lens is None:
        lens = [(37 * b) % 90 for b in range(B)]
    c = make(B, max(max(lens), 1), 6, 2, 64, 128, lens, seed=B, page=page, block=block)
    check(run(c), c)


def pick(c, keep, seed, first=True):
    """Ascending lists of different blocks of each sequence, then -1, as the selection gives them."""
    g = torch.Generator().manual_seed(seed)
    B, hn = c["q2"].shape[:2]
    lists = torch.full((B, hn, keep), -1, dtype=torch.int32)
    counts = []
    for b, n in enumerate(c["lens"].tolist()):
        blocks = -(-n // c["block"])
        counts.append(min(keep, blocks))
        for i in range(hn):
            lists[b, i, :counts[-1]] = torch.randperm(blocks, generator=g)[:counts[-1]].sort().values.to(torch.int32)
    return lists.cuda(), torch.tensor(counts, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("page", [0, 192])
@pytest.mark.parametrize("hs,hn,d,dv,block,keep", [(3, 1, 64, 128, 64, 4), (12, 4, 64, 128, 16, 9), (16, 4, 128, 256, 32, 5),
                                                   (6, 6, 64, 64, 64, 3), (5, 1, 128, 128, 16, 40), (2, 2, 64, 256, 64, 1)])
def test_listed_blocks(hs, hn, d, dv, block, keep, page):
    lens = [1, 0, 15, 17, 64, 700, 768, 333, 641]
    c = make(len(lens), 768, hs, hn, d, dv, lens, seed=keep, page=page, block=block, powers=keep != 5)
    c["lists"] = pick(c, keep, seed=keep)
    gda.gda_device_error(clear=True)
    out = run(c)
    assert gda.gda_device_error(clear=True) == 0
    check(out, c)


def test_lists_of_the_callers_own():
    """Holes, blocks past the length, a block twice, descending order, counts that end a list early, and nothing at all."""
    c = make(8, 640, 6, 2, 64, 128, [640, 640, 640, 640, 100, 640, 640, 0], seed=2, page=64, block=64)
    lists = torch.tensor([[3, -1, 5, -1], [9, 8, 1, 0], [4, 4, 4, 2], [-1, -1, -1, -1], [1, 2, 7, 9], [2, 6, 7, 8],
                          [2 ** 31 - 1, -(2 ** 31), 3, 10], [0, 1, 2, 3]], dtype=torch.int32, device="cuda")
    lists = torch.stack((lists, lists.flip(1)), 1).contiguous()
    c["lists"] = (lists, torch.tensor([4, 4, 4, 4, 4, 2, 4, 4], dtype=torch.int32, device="cuda"))
    gda.gda_device_error(clear=True)
    out = run(c)
    assert gda.gda_device_error(clear=True) == 0
    check(out, c)
    c["lists"][1][5], c["lists"][1][3] = 5, -1
    again = run(c)
    assert gda.gda_device_error(clear=True) == gda.GDA_DEVERR_BAD_LENGTH
    c["lists"][1][5], c["lists"][1][3] = 4, 0
    check(again, c)


def test_all_blocks_listed_is_the_whole_decode():
    c = make(5, 700, 12, 4, 64, 128, [700, 1, 64, 0, 513], seed=6, page=64, block=64)
    whole = run(c)
    c["lists"] = pick(c, 11, seed=1)
    some = run(c)
    check(whole, dict(c, lists=None))
    check(some, c)


def test_repeats_bit_for_bit_and_ignores_the_workspace_before():
    c = make(9, 704, 12, 4, 64, 128, [700, 3, 0, 555, 64, 64, 1, 699, 17], seed=3, page=64, block=32)
    for lists in (None, pick(c, 6, seed=2)):
        c["lists"] = lists
        ws = torch.full((gda.gda_attn_decode_fp8_block_workspace_size(9, 12, 4, 64, 128),), 0xFF, dtype=torch.uint8,
                        device="cuda")
        a = run(c, workspace=ws).clone()
        assert torch.equal(a, run(c, workspace=ws)) and torch.equal(a, run(c))
        check(a, c)


def test_paged_equals_contiguous():
    c = make(6, 512, 6, 2, 128, 128, [512, 1, 300, 64, 0, 511], seed=4, page=64, block=32)
    flat = dict(c, table=None)
    for k in ("pools", "scales"):
        flat[k] = [t[c["table"].long()].flatten(1, 2).contiguous() for t in c[k]]
    assert torch.equal(run(c), run(flat))
    c["lists"] = flat["lists"] = pick(c, 5, seed=3)
    assert torch.equal(run(c), run(flat))


def test_rows_past_a_length_are_never_used():
    """NaN codes in every cache row past the lengths, NaN scales in every block past them and in pages no table names."""
    lens = [1, 0, 15, 17, 96, 130, 47]
    c = make(len(lens), 160, 6, 2, 64, 128, lens, seed=5, page=32, block=16)
    want = run(c).clone()
    c["lists"] = pick(c, 4, seed=5)
    listed = run(c).clone()
    used = torch.zeros(c["pools"][0].shape[:2], dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        for j in range(n):
            used[c["table"][b, j // 32].long(), j % 32] = True
    for p, s in zip(c["pools"], c["scales"]):
        p[~used] = 0x7F
        s[~used.view(used.shape[0], -1, 16).any(-1)] = float("nan")
    assert torch.equal(run(c), listed)
    c["lists"] = None
    assert torch.equal(run(c), want)


def test_scales_far_apart_and_zero():
    """Blocks whose values are 2^40 apart, and blocks that are zero: each output is of the weighted largest."""
    c = make(3, 256, 6, 2, 64, 128, [256, 200, 129], seed=7, block=32)
    v = c["scales"][2]
    for k in range(v.shape[1]):
        v[:, k] = 0.0 if k == 0 else 2.0 ** (10 * ((5 * k) % 4) - 20)
    c["scales"][0][:, 3] = 0.0
    check(run(c), c)


def test_scales_without_a_finite_inverse():
    """Scales below 2^-128, whose inverse is past float32: beside ordinary blocks, and alone."""
    c = make(3, 256, 6, 2, 64, 128, [256, 200, 129], seed=13, block=32)
    v = c["scales"][2]
    v[:2, ::2] = 2.0 ** -149
    v[2] = 2.0 ** -140
    c["scales"][0][:, 3] = 2.0 ** -145
    out = run(c)
    check(out[:2], {**c, **{k: c[k][:2] for k in ("q1", "q2", "lens")}})
    assert (out[2].abs() <= 2.0 ** -120).all()


def test_large_queries_and_scores():
    c = make(2, 512, 3, 1, 128, 128, [512, 300], seed=8, block=64)
    c["q1"] *= 3e4
    c["q2"] *= 1e-6
    for s in c["scales"][:1]:
        s *= 2.0 ** -12
    check(run(c), c)


def test_tiny_and_nan_queries():
    c = make(3, 64, 3, 1, 64, 64, [64, 40, 16], seed=9)
    c["q1"][0] = 2.0 ** -120
    c["q2"][0] = 0
    check(run(c), c)
    c["q1"][1, 1, 3] = float("nan")
    out = run(c)
    assert torch.isnan(out[1, 1]).all() and torch.isfinite(out[2]).all() and torch.isfinite(out[1, 0]).all()


def test_bad_lengths_and_pages_are_reported():
    c = make(3, 96, 6, 2, 64, 128, [96, 97, -4], seed=10, page=32)
    gda.gda_device_error(clear=True)
    out = run(c)
    assert gda.gda_device_error(clear=True) == gda.GDA_DEVERR_BAD_LENGTH
    c["lens"] = torch.tensor([96, 96, 0], dtype=torch.int32, device="cuda")
    check(out, c)
    c["table"][0, 1], c["table"][1, 2] = 10 ** 9, -1
    for lists in (None, pick(c, 6, seed=4)):
        c["lists"] = lists
        out = run(c)
        assert gda.gda_device_error(clear=True) == gda.GDA_DEVERR_BAD_PAGE
        check(out, c | {"table": torch.where((c["table"] >= 0) & (c["table"] < 11), c["table"], 0)})


def test_captured_replayed_and_on_another_stream():
    c = make(4, 256, 6, 2, 64, 128, [200, 1, 0, 77], seed=11, page=64, block=64)
    for lists in (None, pick(c, 3, seed=6)):
        c["lists"] = lists
        ws = torch.empty(gda.gda_attn_decode_fp8_block_workspace_size(4, 6, 2, 64, 128), dtype=torch.uint8, device="cuda")
        out = torch.empty(4, 6, 128, dtype=torch.bfloat16, device="cuda")
        run(c, out=out, workspace=ws)
        graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph):
            run(c, out=out, workspace=ws)
        for n in ([256, 3, 9, 77], [0, 1, 256, 64]):
            c["lens"].copy_(torch.tensor(n, dtype=torch.int32))
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                graph.replay()
                other = run(c)
            torch.cuda.current_stream().wait_stream(s)
            check(out, c)
            assert torch.equal(out, other)
        c["lens"].copy_(torch.tensor([200, 1, 0, 77], dtype=torch.int32))


def test_rows_past_2_to_the_32_bytes():
    """A pool of 5.2 GB of V codes; the pages of the sequence are its last ones."""
    hs, hn, d, dv, ps, pages = 64, 1, 64, 256, 64, 5000
    pools = [torch.zeros(pages, ps, h, n, dtype=torch.uint8, device="cuda") for h, n in ((hs, d), (hn, d), (hs, dv))]
    assert pools[2].numel() > 1 << 32
    small = make(1, 3 * ps, hs, hn, d, dv, [3 * ps - 5], seed=12, page=ps, block=32)
    scales = [torch.zeros(pages, ps // 32, h, device="cuda") for h in (hs, hn, hs)]
    at = torch.tensor([pages - 1, pages - 3, pages - 2], device="cuda")
    for i in range(3):
        pools[i][at] = small["pools"][i][small["table"][0].long()]
        scales[i][at] = small["scales"][i][small["table"][0].long()]
    c = small | {"pools": pools, "scales": scales, "table": at.to(torch.int32)[None].contiguous()}
    assert torch.equal(run(c), run(small))
    lists = (torch.tensor([[[1, 3, 5]]], dtype=torch.int32, device="cuda"), torch.tensor([3], dtype=torch.int32, device="cuda"))
    assert torch.equal(run(c | {"lists": lists}), run(small | {"lists": lists}))


def test_binding_refuses():
    c = make(2, 64, 6, 2, 64, 128, [64, 3], seed=1, page=32)
    lists = pick(c, 2, seed=1)
    good = [c["q1"], c["q2"], *c["pools"], *c["scales"], c["table"], c["lens"], c["lam"]]
    for i, t in enumerate(good):
        for other in (t.cpu(), t.double(), t[:, :1] if t.dim() > 1 else t[:1]):
            bad = list(good)
            bad[i] = other
            with pytest.raises((TypeError, ValueError, gda.GDAError)):
                gda.gda_attn_decode_paged_fp8_block(*bad, LAM0)
            with pytest.raises((TypeError, ValueError, gda.GDAError)):
                gda.gda_attn_decode_sparse_fp8_block(*bad[:8], *lists, *bad[9:], LAM0, block_table=bad[8])
    with pytest.raises((TypeError, ValueError)):
        gda.gda_attn_decode_fp8_block(*good[:8], *good[9:], LAM0)       # more pages than sequences
    with pytest.raises((TypeError, ValueError)):
        gda.gda_attn_decode_paged_fp8_block(*good[:8], None, *good[9:], LAM0)
    for bad in ((lists[0].long(), lists[1]), (lists[0][:, :1], lists[1]), (lists[0], lists[1][:1]), (lists[0].cpu(), lists[1])):
        with pytest.raises((TypeError, ValueError)):
            gda.gda_attn_decode_sparse_fp8_block(*good[:8], *bad, *good[9:], LAM0, block_table=good[8])
    with pytest.raises((TypeError, ValueError)):
        run(c, out=torch.empty(2, 6, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(gda.GDAError):
        run(c, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
