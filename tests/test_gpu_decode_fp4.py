"""Decode over a 4-bit cache, contiguous and paged, against the float64 dense decode of the values it holds.

Tolerance, with mag the sum of absolute terms behind an output element and
rms(.) over a head's row: the weights and the scores behind them are off by at
most 2^-10 of each weight (a weight rounded to 11 bits, 2^-11; a score of
magnitude up to 200 in float32, 2^-13 in the exponent; exp2 2^-22), so an
element moves by 2^-10 mag, the norm's factor by the row's share of that, and
the bf16 result by half a step: |err| <= 2^-8 |ref| + 2^-10 (mag + |ref|
rms(mag) / rms(ref)), the second term doubled to 2^-9 for the sum of both maps.
"""
import numpy as np
import pytest
import torch

import grouped_differential_attention_gb300 as gda
from oracle import ref_serving as R

pytestmark = pytest.mark.gpu
LAM0 = 0.8


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_differential_attention_gb300 import build
    build.build()


def make(B, Lcap, hs, hn, d, dv, lens, seed, page=0, spread=1.0):
    """Normal rows in 4 bits, written by the library itself (its bytes are tested elsewhere)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    size = page or Lcap
    mp = -(-Lcap // size)
    pages = B * mp + (2 if page else 0)
    dims = ((hs, d), (hn, d), (hs, dv))
    scales = [0.25 + torch.rand(h, generator=g, device="cuda") for h, _ in dims]
    pools = [torch.empty(pages, size, h, n // 2, dtype=torch.uint8, device="cuda") for h, n in dims]
    blocks = [torch.empty(pages, size, h, n // 16, dtype=torch.uint8, device="cuda") for h, n in dims]
    rows = [(spread * torch.randn(pages * size, h, n, generator=g, device="cuda")).bfloat16() for h, n in dims]
    gda.gda_cache_append_fp4(*rows, torch.arange(pages * size, dtype=torch.int32, device="cuda"), *pools, *blocks, *scales)
    table = None
    if page:
        table = torch.randperm(pages, generator=g, device="cuda")[:B * mp].view(B, mp).to(torch.int32).contiguous()
    q1, q2 = (torch.randn(B, h, d, generator=g, device="cuda").bfloat16() for h in (hs, hn))
    lam = 0.2 + 0.6 * torch.rand(hs, generator=g, device="cuda")
    return dict(q1=q1, q2=q2, pools=pools, blocks=blocks, scales=scales, table=table, lam=lam,
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))


def run(c, **kw):
    head = (c["q1"], c["q2"], *c["pools"], *c["blocks"], *c["scales"])
    if c["table"] is None:
        return gda.gda_attn_decode_fp4(*head, c["lens"], c["lam"], LAM0, **kw)
    return gda.gda_attn_decode_paged_fp4(*head, c["table"], c["lens"], c["lam"], LAM0, **kw)


def reference(c, eps=1e-5):
    """(output, mag) in float64 [B, hs, dv], one sequence at a time."""
    hs, hn, d = c["q1"].shape[1], c["q2"].shape[1], c["q1"].shape[2]
    outs, mags = [], []
    lam = c["lam"].double()[:, None]
    grid = torch.tensor(np.concatenate([R.E2M1, -R.E2M1]), device="cuda")
    for b, n in enumerate(c["lens"].tolist()):
        kv = []
        for code, block, s in zip(c["pools"], c["blocks"], c["scales"]):
            if c["table"] is None:
                code, block = code[b], block[b]
            else:
                used = c["table"][b, :-(-max(n, 1) // code.shape[1])].long()
                code, block = (t[used].flatten(0, 1) for t in (code, block))
            u = torch.stack((code[:n] & 15, code[:n] >> 4), -1).flatten(-2).long()
            kv.append(grid[u] * block[:n].view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
                      * s.double()[:, None])
        if n == 0:
            outs.append(torch.zeros(hs, kv[2].shape[-1], dtype=torch.float64, device="cuda"))
            mags.append(outs[-1])
            continue
        a1 = torch.softmax(torch.einsum("hd,jhd->hj", c["q1"][b].double(), kv[0]) / d ** 0.5, -1)
        a2 = torch.softmax(torch.einsum("hd,jhd->hj", c["q2"][b].double(), kv[1]) / d ** 0.5, -1)
        a2 = a2.repeat_interleave(hs // hn, 0)
        o = torch.einsum("hj,jhe->he", a1 - lam * a2, kv[2])
        f = (1 - LAM0) / torch.sqrt((o * o).mean(-1, keepdim=True) + eps)
        outs.append(f * o)
        mags.append(f * torch.einsum("hj,jhe->he", a1 + lam.abs() * a2, kv[2].abs()))
    return torch.stack(outs), torch.stack(mags)


def check(got, c):
    ref, mag = reference(c)
    got = got.double()
    rms = lambda t: (t * t).mean(-1, keepdim=True).sqrt()
    bound = 2.0 ** -8 * ref.abs() + 2.0 ** -9 * (mag + ref.abs() * rms(mag) / rms(ref).clamp(min=1e-30))
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), float(((got - ref).abs() / bound.clamp(min=1e-30)).max()))


SHAPES = [(64, 64), (64, 128), (64, 256), (128, 64), (128, 128), (128, 256)]


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("d,dv", SHAPES)
@pytest.mark.parametrize("hs,hn", [(1, 1), (3, 1), (4, 2), (12, 4), (5, 1), (7, 7), (16, 4)])
def test_shapes_and_edge_lengths(hs, hn, d, dv, page):
    lens = [1, 0, 15, 16, 17, 33, 64, 128, 200, 7]
    c = make(len(lens), 208, hs, hn, d, dv, lens, seed=hs * 7 + d + dv, page=page)
    gda.gda_device_error(clear=True)
    out = run(c)
    assert gda.gda_device_error(clear=True) == 0
    check(out, c)
    assert (out[1] == 0).all()


@pytest.mark.parametrize("B,lens,page", [
    (1, [1], 0), (1, [5000], 64), (1, [40000], 128), (3, [0, 9001, 0], 100), (70, None, 1), (300, None, 16),
    (2, [0, 0], 16), (5, [0, 0, 3, 0, 4097], 0),
])
def test_batches_long_short_and_empty(B, lens, page):
    if lens is None:
        lens = [(37 * b) % 90 for b in range(B)]
    c = make(B, max(max(lens), 1), 6, 2, 64, 128, lens, seed=B, page=page)
    check(run(c), c)


def test_repeats_bit_for_bit_and_ignores_the_workspace_before():
    c = make(9, 700, 12, 4, 64, 128, [700, 3, 0, 555, 64, 64, 1, 699, 17], seed=3, page=16)
    ws = torch.full((gda.gda_attn_decode_fp4_workspace_size(9, 12, 4, 64, 128),), 0xFF, dtype=torch.uint8, device="cuda")
    a = run(c, workspace=ws).clone()
    assert torch.equal(a, run(c, workspace=ws)) and torch.equal(a, run(c))
    check(a, c)


def test_paged_equals_contiguous():
    c = make(6, 512, 6, 2, 128, 128, [512, 1, 300, 64, 0, 511], seed=4, page=64)
    flat = dict(c, table=None)
    for k in ("pools", "blocks"):
        flat[k] = [t[c["table"].long()].flatten(1, 2).contiguous() for t in c[k]]
    assert torch.equal(run(c), run(flat))


def test_rows_past_a_length_are_never_used():
    """NaN block scales in every cache row past the lengths, and in every page that no table names."""
    c = make(4, 96, 6, 2, 64, 128, [33, 1, 95, 48], seed=5, page=32)
    ref = run(c).clone()
    rows = torch.zeros(c["pools"][0].shape[0], 32, dtype=torch.bool, device="cuda")
    for b, n in enumerate(c["lens"].tolist()):
        for pos in range(n):
            rows[int(c["table"][b, pos // 32]), pos % 32] = True
    for t in c["blocks"]:
        t[~rows] = 0x7F
    for t in c["pools"]:
        t[~rows] = 0xFF
    assert torch.equal(run(c), ref) and torch.isfinite(ref.float()).all()
    c["blocks"][2][int(c["table"][2, 0]), 3, 4, 2] = 0x7F            # a NaN among the rows of sequence 2, head 4
    out = run(c)
    assert torch.isnan(out[2, 4]).any() and torch.equal(out[[0, 1, 3]], ref[[0, 1, 3]])
    assert torch.equal(out[2, :4], ref[2, :4]) and torch.equal(out[2, 5], ref[2, 5])


@pytest.mark.parametrize("lam", [0.0, 1.0, -0.7, 1.9])
def test_lambda_outside_the_usual_range(lam):
    c = make(3, 300, 6, 2, 64, 128, [300, 17, 2], seed=6)
    c["lam"].fill_(lam)
    check(run(c), c)


def test_large_scores_and_small_scales():
    """Scores up to ~200 (a few keys take all the weight), then block scales down among the subnormal e4m3."""
    c = make(2, 400, 3, 1, 128, 128, [400, 399], seed=7, spread=6.0)
    c["q1"].mul_(4), c["q2"].mul_(4)
    check(run(c), c)
    c = make(2, 400, 3, 1, 128, 128, [400, 399], seed=8, spread=2.0 ** -6)
    c["q1"].mul_(1000), c["q2"].mul_(2.0 ** -20)
    check(run(c), c)


def test_bad_lengths_and_pages_are_clamped_and_reported():
    c = make(4, 64, 3, 1, 64, 128, [64, 10, 20, 30], seed=9, page=16)
    gda.gda_device_error(clear=True)
    c["lens"][1], c["lens"][0] = -5, 65                                # read as 0 and as 64
    out = run(c)
    assert gda.gda_device_error(clear=True) == gda.GDA_DEVERR_BAD_LENGTH
    fixed = dict(c, lens=torch.tensor([64, 0, 20, 30], dtype=torch.int32, device="cuda"))
    assert (out[1] == 0).all() and torch.equal(out, run(fixed))
    fixed["table"] = c["table"].clone()
    fixed["table"][3, 1] = c["pools"][0].shape[0]
    out = run(fixed)
    assert gda.gda_device_error(clear=True) == gda.GDA_DEVERR_BAD_PAGE
    fixed["table"][3, 1] = 0
    assert torch.equal(out, run(fixed))                                # the bad page was read as page 0
    assert gda.gda_device_error(clear=True) == 0


def test_two_graphs_and_another_stream():
    c = make(5, 900, 12, 4, 64, 128, [900, 0, 1, 450, 899], seed=10, page=64)
    ref = run(c).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = run(c)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(other, ref)
    graphs = []
    for _ in range(2):                                                  # a workspace of its own each
        ws = torch.empty(gda.gda_attn_decode_fp4_workspace_size(5, 12, 4, 64, 128), dtype=torch.uint8, device="cuda")
        out, g = torch.zeros_like(ref), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(c, out=out, workspace=ws)
        graphs.append((g, out, ws))
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graphs[0][0].replay()
    graphs[1][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1], ref) and torch.equal(graphs[1][1], ref)
    c["lens"].copy_(torch.tensor([3, 900, 0, 77, 78], dtype=torch.int32))   # replayed on other lengths
    graphs[0][0].replay()
    torch.cuda.synchronize()
    check(graphs[0][1], c)


@pytest.mark.parametrize("hs,hn,d,dv", [(120, 8, 64, 128), (96, 32, 128, 256), (64, 64, 64, 64), (127, 1, 64, 128),
                                        (21, 3, 128, 64)])
def test_many_heads(hs, hn, d, dv):
    c = make(3, 130, hs, hn, d, dv, [130, 0, 77], seed=hs, page=32)
    check(run(c), c)


def test_a_batch_of_many_more_sequences_than_ranges():
    c = make(3000, 20, 2, 1, 64, 64, [b % 21 for b in range(3000)], seed=15, page=10)
    check(run(c), c)


def test_sequences_that_share_pages():
    c = make(3, 96, 6, 2, 64, 128, [96, 70, 33], seed=13, page=32)
    c["table"][1, 0], c["table"][2] = c["table"][0, 0], c["table"][0]
    check(run(c), c)
    c["table"][0, 1:] = c["table"][0, 0]                               # one page three times in a sequence
    check(run(c), c)


def test_codes_and_scales_in_their_own_types():
    c = make(2, 64, 3, 1, 64, 128, [64, 9], seed=14)
    typed = dict(c, blocks=[t.view(torch.float8_e4m3fn) for t in c["blocks"]])
    if hasattr(torch, "float4_e2m1fn_x2"):
        typed["pools"] = [t.view(torch.float4_e2m1fn_x2) for t in c["pools"]]
    assert torch.equal(run(typed), run(c))


def test_a_nan_in_a_query_stays_with_its_heads():
    c = make(3, 100, 6, 2, 64, 128, [100, 50, 7], seed=16)
    ref = run(c)
    c["q1"][1, 2, 5] = float("nan")
    c["q2"][2, 1, 0] = float("inf")                                    # heads 3 .. 5 share it
    out = run(c)
    assert torch.isnan(out[1, 2]).all() and torch.isnan(out[2, 3:]).all()
    same = torch.ones(3, 6, dtype=torch.bool, device="cuda")
    same[1, 2], same[2, 3:] = False, False
    assert torch.equal(out[same], ref[same])


def test_calls_on_two_streams_at_once():
    cs = [make(5, 900, 6, 2, 64, 128, [900, 20 * i, 1, 333, 512], seed=17 + i, page=16) for i in range(2)]
    refs = [run(c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for c, s, o in zip(cs, streams, outs):
            with torch.cuda.stream(s):
                o.append(run(c))
    torch.cuda.synchronize()
    for ref, o in zip(refs, outs):
        assert all(torch.equal(x, ref) for x in o)


def test_the_serving_batch():
    c = make(64, 8192, 12, 4, 64, 128, [4096 + 65 * b for b in range(64)], seed=11)
    check(run(c), c)


def test_offsets_past_32_bits():
    """Two sequences whose pages lie at the two ends of a pool with more than 2^32 bytes of V codes."""
    B, hs, hn, d, dv, ps, pages = 2, 64, 64, 64, 256, 64, 8400
    V = torch.zeros(pages, ps, hs, dv // 2, dtype=torch.uint8, device="cuda")
    assert V.numel() > 1 << 32
    pools = [torch.zeros(pages, ps, h, d // 2, dtype=torch.uint8, device="cuda") for h in (hs, hn)] + [V]
    blocks = [torch.zeros(pages, ps, h, n // 16, dtype=torch.uint8, device="cuda") for h, n in ((hs, d), (hn, d), (hs, dv))]
    g = torch.Generator(device="cuda").manual_seed(12)
    scales = [torch.ones(h, device="cuda") for h in (hs, hn, hs)]
    table = torch.tensor([[pages - 1, 0], [1, pages - 2]], dtype=torch.int32, device="cuda")
    slots = (table.view(-1, 1) * ps + torch.arange(ps, device="cuda", dtype=torch.int32)).view(-1)
    rows = [torch.randn(slots.numel(), h, n, generator=g, device="cuda").bfloat16() for h, n in ((hs, d), (hn, d), (hs, dv))]
    gda.gda_cache_append_fp4(*rows, slots, *pools, *blocks, *scales)
    c = dict(q1=torch.randn(B, hs, d, generator=g, device="cuda").bfloat16(),
             q2=torch.randn(B, hn, d, generator=g, device="cuda").bfloat16(), pools=pools, blocks=blocks, scales=scales,
             table=table, lam=torch.full((hs,), 0.5, device="cuda"),
             lens=torch.tensor([100, 128], dtype=torch.int32, device="cuda"))
    check(run(c), c)


def test_binding_refuses():
    c = make(2, 32, 3, 1, 64, 128, [3, 4], seed=1, page=16)
    good = [c["q1"], c["q2"], *c["pools"], *c["blocks"], *c["scales"], c["table"], c["lens"], c["lam"]]
    for i, t in enumerate(good):
        bad = list(good)
        bad[i] = t.double()
        with pytest.raises((TypeError, ValueError)):
            gda.gda_attn_decode_paged_fp4(*bad, LAM0)
        bad[i] = t.cpu()
        with pytest.raises((TypeError, ValueError)):
            gda.gda_attn_decode_paged_fp4(*bad, LAM0)
    with pytest.raises(ValueError):                                    # pages of another number of sequences
        gda.gda_attn_decode_fp4(*good[:11], *good[12:], LAM0)
    with pytest.raises(gda.GDAError):
        gda.gda_attn_decode_paged_fp4(*good, LAM0, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(gda.GDAError):
        gda.gda_attn_decode_paged_fp4(*good, float("nan"))
