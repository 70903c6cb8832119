"""The 8-bit block cache at scales of any size and form."""
import numpy as np
import pytest
import torch

import grouped_differential_attention_gb300 as gda
from oracle import ref_serving as R
from tests.test_gpu_cache_fp8_block import Cache
from tests.test_gpu_decode_fp8_block import check, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_differential_attention_gb300 import build
    build.build()


# ---- bounds ----

def with_bounds(scale, seed, block=32):
    """Two blocks of codes, with scales of the caller's own and exactly their bounds."""
    c = Cache(1, 2 * block, block, 3, 1, 64, 64, seed=seed)
    for i in range(3):
        c.ref[0][i] &= 0xF7                                           # no NaN codes (bit 3 of 0x7F and 0xFF)
        c.ref[1][i][:] = scale
        if i < 2:
            v = R.e4m3_value(c.ref[0][i]).reshape(2, block, *c.ref[0][i].shape[1:]) / 4
            c.ref[2][i][:] = np.stack((np.ceil(v.max(1)), np.floor(v.min(1))), 2)
        for k in range(3):
            if k < 2 or i < 2:
                c.dev[k][i].copy_(torch.from_numpy(c.ref[k][i]).view(c.dev[k][i].shape))
    return c


def assert_bounds_hold(c):
    for i in range(2):
        code = R.e4m3_value(c.dev[0][i].cpu().numpy()[0])             # [slots, heads, n]
        code = code.reshape(2, -1, *code.shape[1:])
        top, low = (c.dev[2][i].cpu().numpy()[0, :, :, k].astype(np.float64) for k in range(2))
        assert (code.max(1) <= 4 * top).all(), (i, float((code.max(1) - 4 * top).max()))
        assert (code.min(1) >= 4 * low).all(), (i, float((4 * low - code.min(1)).max()))


@pytest.mark.parametrize("alone", [True, False])
@pytest.mark.parametrize("scale", [1.366, 0.75, 3.0, 1.9999999, 1.0, 0.3 * 2.0 ** -126])
def test_bounds_stay_bounds_when_a_scale_of_the_callers_own_grows(scale, alone):
    """Codes that are brought to a new scale are rounded to e4m3, upwards too, by up to half a step of 32."""
    for seed in range(3):
        c = with_bounds(scale, seed)
        assert_bounds_hold(c)
        g = torch.Generator().manual_seed(seed)
        slots = torch.tensor([5, 40] if alone else [5, 40, 9, 3, 63, 33], dtype=torch.int32)
        for times in (448 * 1.01, 448 * 1.3, 448 * 2.9, 448 * 64.0, 448 * 5e4):   # of the scale: it grows each time
            rows = [(x.float().sign() * times * scale).bfloat16() for x in c.rows(slots.numel(), g)]
            for x in rows:
                x[:, :, ::2] *= 0.01
            c.append(rows, slots)
            assert_bounds_hold(c)
            c.check()


# ---- reading ----

def bf16_once(x):
    """float64 x to bf16, rounded once (torch goes through float32)."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(all="ignore"):
        e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126)))
        step = np.exp2(e - 7)
        y = np.rint(x / step) * step
    return torch.from_numpy(np.where(np.abs(y) >= 2.0 ** 128, np.copysign(np.inf, x), y)).float().bfloat16()


@pytest.mark.parametrize("low,high", [(0.0, 1.0), (-126.0, -118.0), (-149.0, -126.0), (116.0, 127.99)])
def test_rows_of_any_scale_are_rounded_once(low, high):
    c = Cache(64, 32, 16, 4, 2, 64, 128, seed=11)
    g = torch.Generator().manual_seed(int(high))
    for s in c.dev[1]:
        s.copy_(torch.exp2(low + (high - low) * torch.rand(s.shape, generator=g)))
    c.dev[1][0][0, 0, 0], c.dev[1][0][0, 0, 1], c.dev[1][2][5, 1, 2] = 1.2881944, 0.0, 1.5
    c.ref[1] = [s.flatten(0, 1).cpu().numpy() for s in c.dev[1]]
    slots = torch.arange(64 * 32, dtype=torch.int32)
    back = gda.gda_cache_read_fp8_block(slots.cuda(), *c.dev[0], *c.dev[1])
    for i, y in enumerate(back):
        want = bf16_once(c.value(i, slots.numpy()).numpy())
        y = y.cpu()
        assert torch.equal(torch.isnan(y), torch.isnan(want))
        diff = torch.nan_to_num(y.float(), nan=7.0) != torch.nan_to_num(want.float(), nan=7.0)
        assert not diff.any(), (i, int(diff.sum()))


# ---- values of any size ----

def check_numbers(got, c, eps=1e-5):
    """The bound of tests/test_gpu_decode_fp8_block.py, which NaN would pass."""
    assert torch.isfinite(got).all()
    check(got, c, eps)


@pytest.mark.parametrize("power", [100, 65, 64, 63, 50, -40, -75, -100, -118])
@pytest.mark.parametrize("B,L,hs,hn,d,dv,page", [(3, 200, 6, 2, 64, 128, 48), (1, 20000, 3, 1, 64, 64, 0),
                                                 (40, 2100, 4, 2, 128, 256, 0), (2, 300, 1, 1, 64, 256, 0)])
def test_values_of_any_size(B, L, hs, hn, d, dv, page, power):
    """V near both ends of float32: the norm's squares are past it."""
    lens = [max(1, L - 37 * b) for b in range(B)]
    c = make(B, L, hs, hn, d, dv, lens, seed=power + 200, page=page, powers=power % 2 == 0)
    c["scales"][2] *= 2.0 ** power
    for s in c["scales"][:2]:
        s *= 0.25                                                     # flat maps: sums of many weights near one
    eps = 1e-5 if power > 0 else 0.0
    check_numbers(run(c, eps=eps), c, eps)


@pytest.mark.parametrize("power", [110, 118, 125])
@pytest.mark.parametrize("B,L,hs,hn,d,dv,page", [(3, 200, 6, 2, 64, 128, 48), (1, 20000, 3, 1, 64, 64, 0),
                                                 (40, 2100, 4, 2, 128, 256, 0), (2, 300, 1, 1, 64, 256, 0)])
def test_sums_of_large_values(B, L, hs, hn, d, dv, page, power):
    """V up to the end of float32, whose sums over hundreds of equal weights are past it."""
    lens = [max(1, L - 37 * b) for b in range(B)]
    c = make(B, L, hs, hn, d, dv, lens, seed=power, page=page, powers=power % 2 == 0)
    c["scales"][2] *= 2.0 ** power
    c["pools"][2] &= 0x7F                                             # of one sign
    for s in c["scales"][:2]:
        s *= 0.25
    check_numbers(run(c), c)


def test_values_of_one_sequence_at_both_ends():
    """Parts of a sequence whose sums are held by different powers of two are joined."""
    c = make(1, 40000, 3, 1, 64, 128, [40000], seed=3, block=64)
    c["scales"][2] *= 2.0 ** 60
    c["scales"][2][:, ::7] *= 2.0 ** 12
    c["scales"][2][:, 300:] *= 2.0 ** 3
    check_numbers(run(c), c)
