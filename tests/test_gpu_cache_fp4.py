"""4-bit cache rows on the GPU: written bytes equal the reference's, rows read back are its values rounded once."""
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


def make(T, hs, hn, d, dv, ps, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    dims = ((hs, d), (hn, d), (hs, dv))
    rows = [(torch.randn(T, h, n, generator=g) * spread * torch.exp(torch.randn(T, h, 1, generator=g))).bfloat16()
            for h, n in dims]
    scales = [0.25 + torch.rand(h, generator=g) for h, _ in dims]
    pages = -(-T // ps) + 2
    slots = torch.randperm(pages * ps, generator=g)[:T].to(torch.int32)
    pools = [torch.randint(0, 256, (pages, ps, h, n // 2), generator=g, dtype=torch.uint8) for h, n in dims]
    blocks = [torch.randint(0, 120, (pages, ps, h, n // 16), generator=g, dtype=torch.uint8) for h, n in dims]
    return rows, slots, pools, blocks, scales


CASES = [  # T, h_s, h_n, d, dv, page size
    (1, 1, 1, 64, 64, 1), (5, 3, 1, 64, 128, 16), (64, 12, 4, 64, 128, 64), (77, 16, 4, 128, 256, 7),
    (300, 6, 2, 128, 64, 100), (1000, 2, 2, 64, 256, 32),
]


def same(a, b):
    """Equal values (a NaN equals a NaN, -0 equals 0)."""
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(0.0), b.nan_to_num(0.0))


@pytest.mark.parametrize("case", CASES, ids=str)
def test_written_bytes_and_values_read_back(case):
    T, hs, hn, d, dv, ps = case
    rows, slots, pools, blocks, scales = make(*case, seed=T)
    slots[T // 2] = -1 if T > 1 else slots[0]
    dp, db = [t.cuda() for t in pools], [t.cuda() for t in blocks]
    sc, sl = [t.cuda() for t in scales], slots.cuda()
    gda.gda_device_error(clear=True)
    gda.gda_cache_append_fp4(*(t.cuda() for t in rows), sl, *dp, *db, *sc)
    back = gda.gda_cache_read_fp4(sl, *dp, *(t.view(torch.float8_e4m3fn) for t in db), *sc)
    torch.cuda.synchronize()
    assert gda.gda_device_error(clear=True) == 0
    live = slots.numpy() >= 0
    at = slots.numpy()[live]
    for x, p0, b0, p, b, s, y in zip(rows, pools, blocks, dp, db, scales, back):
        codes, s8 = R.quantise_fp4(x, s.numpy())
        want_p, want_b = p0.flatten(0, 1).numpy().copy(), b0.flatten(0, 1).numpy().copy()
        want_p[at], want_b[at] = R.pack(codes)[live], s8[live]
        assert np.array_equal(b.cpu().flatten(0, 1).numpy(), want_b)      # rows of other slots untouched
        assert np.array_equal(p.cpu().flatten(0, 1).numpy(), want_p)
        value = R.dequantise_fp4(codes, s8, s.numpy())
        value[~live] = 0
        assert same(y.cpu(), torch.from_numpy(value).float().bfloat16())


def test_special_values():
    x = torch.zeros(1, 4, 64).bfloat16()
    x[0, 0, 3], x[0, 0, 17], x[0, 1, 0], x[0, 1, 1] = 2.0 ** -12, float("nan"), float("inf"), 1.0
    x[0, 2, :16] = torch.tensor([6.0, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 0])
    x[0, 3, 5] = -3e38
    z = torch.zeros(1, 1, 64).bfloat16()
    one = [torch.ones(h) for h in (4, 1, 4)]
    codes, s8 = R.quantise_fp4(x, one[0].numpy())
    pools = [torch.zeros(1, 2, h, 32, dtype=torch.uint8, device="cuda") for h in (4, 1, 4)]
    blocks = [torch.zeros(1, 2, h, 4, dtype=torch.uint8, device="cuda") for h in (4, 1, 4)]
    slot = torch.tensor([1], dtype=torch.int32, device="cuda")
    sc = [t.cuda() for t in one]
    gda.gda_cache_append_fp4(x.cuda(), z.cuda(), x.cuda(), slot, *pools, *blocks, *sc)
    back = gda.gda_cache_read_fp4(slot, *pools, *blocks, *sc)
    value = torch.from_numpy(R.dequantise_fp4(codes, s8, one[0].numpy())).float().bfloat16()
    for y in (back[0].cpu(), back[2].cpu()):
        assert torch.isnan(y[0, 0, 16:32]).all() and same(y, value)
    assert (blocks[0][0, 0] == 0).all() and (pools[0][0, 0] == 0).all()


def test_slots_past_the_pool_are_left_out_and_reported():
    rows, slots, pools, blocks, scales = make(8, 3, 1, 64, 128, 4, seed=1)
    slots[3] = pools[0].shape[0] * 4
    dp, db, sc = [t.cuda() for t in pools], [t.cuda() for t in blocks], [t.cuda() for t in scales]
    gda.gda_device_error(clear=True)
    gda.gda_cache_append_fp4(*(t.cuda() for t in rows), slots.cuda(), *dp, *db, *sc)
    assert gda.gda_device_error(clear=True) == gda.GDA_DEVERR_BAD_PAGE
    back = gda.gda_cache_read_fp4(slots.cuda(), *dp, *db, *sc)
    assert gda.gda_device_error(clear=True) == gda.GDA_DEVERR_BAD_PAGE
    assert all((t[3] == 0).all() and (t[4] != 0).any() for t in back)


def test_a_slot_read_twice():
    rows, slots, pools, blocks, scales = make(6, 3, 1, 64, 128, 4, seed=2)
    cache = [t.cuda() for t in (*pools, *blocks, *scales)]
    gda.gda_cache_append_fp4(*(t.cuda() for t in rows), slots.cuda(), *cache)
    once = gda.gda_cache_read_fp4(slots.cuda(), *cache)
    order = [3, 3, 0, 5, 3]
    for a, b in zip(gda.gda_cache_read_fp4(slots[order].cuda(), *cache), once):
        assert torch.equal(a, b[order])


def test_rows_out_of_a_fused_projection_on_another_stream():
    hs, hn, d, dv, T = 6, 2, 64, 128, 50
    g = torch.Generator().manual_seed(2)
    proj = torch.randn(T, hs * (d + dv) + hn * d + 24, generator=g).bfloat16().cuda()
    k1, k2 = proj[:, :hs * d].unflatten(-1, (hs, d)), proj[:, hs * d:(hs + hn) * d].unflatten(-1, (hn, d))
    v = proj[:, (hs + hn) * d:(hs + hn) * d + hs * dv].unflatten(-1, (hs, dv))
    _, slots, pools, blocks, scales = make(T, hs, hn, d, dv, 16, seed=3)
    s = torch.cuda.Stream()
    outs = []
    for rows in ((k1, k2, v), tuple(t.contiguous() for t in (k1, k2, v))):
        dp, db, sc = [t.cuda() for t in pools], [t.cuda() for t in blocks], [t.cuda() for t in scales]
        sl = slots.cuda()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            gda.gda_cache_append_fp4(*rows, sl, *dp, *db, *sc)
        torch.cuda.current_stream().wait_stream(s)
        outs.append((dp, db))
    for a, b in zip(outs[0], outs[1]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_rows_far_into_a_large_pool():
    """Byte offsets beyond 2^32: the last slots of a pool of 4.7 GB of V codes."""
    hs, hn, d, dv, ps = 64, 1, 64, 256, 64
    pages = 9000
    V = torch.zeros(pages, ps, hs, dv // 2, dtype=torch.uint8, device="cuda")
    assert V.numel() > 1 << 32
    k1p, k2p = (torch.zeros(pages, ps, h, d // 2, dtype=torch.uint8, device="cuda") for h in (hs, hn))
    blocks = [torch.zeros(pages, ps, h, n // 16, dtype=torch.uint8, device="cuda") for h, n in ((hs, d), (hn, d), (hs, dv))]
    g = torch.Generator().manual_seed(4)
    rows = [torch.randn(2, h, n, generator=g).bfloat16() for h, n in ((hs, d), (hn, d), (hs, dv))]
    sc = [torch.ones(h, device="cuda") for h in (hs, hn, hs)]
    slots = torch.tensor([pages * ps - 1, pages * ps - 70], dtype=torch.int32, device="cuda")
    gda.gda_cache_append_fp4(*(t.cuda() for t in rows), slots, k1p, k2p, V, *blocks, *sc)
    back = gda.gda_cache_read_fp4(slots, k1p, k2p, V, *blocks, *sc)
    for x, y, h in zip(rows, back, (hs, hn, hs)):
        codes, s8 = R.quantise_fp4(x, np.ones(h, dtype=np.float32))
        assert same(y.cpu(), torch.from_numpy(R.dequantise_fp4(codes, s8, np.ones(h))).float().bfloat16())
    assert int(torch.count_nonzero(V)) == int(torch.count_nonzero(V.view(-1, hs, dv // 2)[slots.long()]))


def test_binding_refuses():
    rows, slots, pools, blocks, scales = make(8, 3, 1, 64, 128, 4, seed=1)
    good = [t.cuda() for t in (*rows, slots, *pools, *blocks, *scales)]
    for i, t in enumerate(good):
        bad = list(good)
        bad[i] = t.cpu()
        with pytest.raises((TypeError, ValueError)):
            gda.gda_cache_append_fp4(*bad)
        bad[i] = t.double()
        with pytest.raises((TypeError, ValueError)):
            gda.gda_cache_append_fp4(*bad)
    with pytest.raises((TypeError, ValueError)):
        gda.gda_cache_append_fp4(good[0].transpose(1, 2).contiguous().transpose(1, 2), *good[1:])
