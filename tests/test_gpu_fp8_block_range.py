"""The 8-bit block cache at scales of any size and form."""
import math

import numpy as np
import pytest
import torch

import grouped_differential_attention_gb300 as gda
from oracle import ref_serving as R
from tests.test_gpu_cache_fp8_block import Cache
from tests.test_gpu_decode_fp8_block import LAM0, check, make, run

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


# ---- scales far apart ----

def far_apart(order, gap, apart, RH, seed=0, noise_too=True, B=2):
    """Blocks of V scales 2^apart and 1 whose keys' scores lie `gap` powers of two below and at the top, in an order that
    repeats; several of them to a warp (eight noise heads share the warps of the GPU, 240 tiles to a sequence)."""
    block, hs, hn, d, dv = 16, 8 * RH, 8, 64, 128
    order = order * (240 // len(order))
    n = len(order) * block
    c = make(B, n, hs, hn, d, dv, [n] * B, seed=seed, block=block)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for q, p, s in ((c["q1"], c["pools"][0], c["scales"][0]), (c["q2"], c["pools"][1], c["scales"][1])):
        unit = q.float().abs().sum(-1) / d ** 0.5 / math.log(2)       # score of sign(q), in powers of two
        code = (q.float().sign() * 8)[:, None] * (1 + 0.125 * torch.randint(0, 2, (B, n, 1, 1), generator=g, device="cuda"))
        p.copy_(code.expand(p.shape).to(torch.float8_e4m3fn).view(torch.uint8))
        for i, big in enumerate(order):
            sign = -1.0 if big and (noise_too or q is c["q1"]) else 1.0
            p.view(torch.float8_e4m3fn)[:, i * block:(i + 1) * block] = \
                (sign * p.view(torch.float8_e4m3fn)[:, i * block:(i + 1) * block].float()).to(torch.float8_e4m3fn)
        s.copy_((gap / 2 / (8 * unit))[:, None].expand(s.shape))
    for i, big in enumerate(order):
        c["scales"][2][:, i] = 2.0 ** apart if big else 1.0
    return c


def check_far_apart(got, c):
    """Bound of tests/test_gpu_decode_fp8_block.py with the weights' steps taken of the largest product of a weight and a
    V scale: they are 2^-39 (f16's smallest, where the largest is 2^15) of a number that is at most 2^12 times that."""
    hs, d = c["q1"].shape[1:]
    bl, r = c["block"], hs // c["q2"].shape[1]
    assert torch.isfinite(got).all()
    worst = 0.0
    for b, n in enumerate(c["lens"].tolist()):
        pos = torch.arange(n, device="cuda")

        def value(i, h):
            code = c["pools"][i][b, :n, h].view(torch.float8_e4m3fn).float().double()
            return code, c["scales"][i][b].double()[pos // bl, h][:, None]

        def softmax(i, q, h):
            code, s = value(i, h)
            k = code * s
            return torch.softmax(k @ q.double() / d ** 0.5, 0), (k.abs() @ q.double().abs()).max() / d ** 0.5

        for h in range(hs):
            a2, s2 = softmax(1, c["q2"][b, h // r], h // r)
            a1, s1 = softmax(0, c["q1"][b, h], h)
            code, vs = value(2, h)
            v, lam = code * vs, c["lam"][h].double()
            o, off = (a1 - lam * a2) @ v, 0
            for a, w, s in ((a1, 1.0, s1), (a2, lam.abs(), s2)):
                off = off + w * (2.0 ** -18 * (1 + s / math.log(2)) * (a @ v.abs())
                                 + n * 2.0 ** -27 * (a[:, None] * vs).max() * code.abs().max())
            f = (1 - LAM0) / torch.sqrt((o * o).mean() + 1e-5)
            ref = f * o
            rms = torch.sqrt((off * off).mean())
            bound = 2.0 ** -8 * ref.abs() + f * off + ref.abs() * rms / torch.sqrt((o * o).mean() + 1e-5)
            worst = max(worst, float(((got[b, h].double() - ref).abs() / bound).max()))
    assert worst <= 1.0, worst


@pytest.mark.parametrize("RH", [1, 2, 3])
@pytest.mark.parametrize("gap,apart", [(20, 18), (20, 24), (45, 40), (60, 40), (60, 58), (100, 90), (3, 30)])
@pytest.mark.parametrize("order", [(1, 0), (0, 1), (0, 1, 0, 1, 1, 0), (1, 1, 1, 0, 0, 1)])
def test_scales_far_apart_with_the_weight_on_the_small(order, gap, apart, RH):
    c = far_apart(order, gap, apart, RH)
    check_far_apart(run(c), c)


@pytest.mark.parametrize("order", [(1, 0), (0, 1), (0, 1, 0, 1, 1, 0)])
def test_scales_far_apart_in_one_map_only(order):
    c = far_apart(order, 60, 40, 3, noise_too=False)
    check_far_apart(run(c), c)


@pytest.mark.parametrize("step,apart", [(0.9, 30), (1.6, 40), (2.5, 90)])
def test_scales_far_apart_with_scores_that_rise_slowly(step, apart):
    """Saw teeth of 40 tiles: the first four have the large V scale, and the scores rise by `step` powers of two a tile."""
    tiles, block, hn, d, dv = 6400, 16, 8, 64, 64
    n = tiles * block
    c = make(1, n, hn, hn, d, dv, [n], seed=1, block=block)
    tooth = torch.arange(tiles, device="cuda") % 40
    for q, p, s in ((c["q1"], c["pools"][0], c["scales"][0]), (c["q2"], c["pools"][1], c["scales"][1])):
        unit = 8 * q.float().abs().sum(-1) / d ** 0.5 / math.log(2)   # score of 8 sign(q), in powers of two
        p.copy_((q.float().sign() * 8)[:, None].expand(p.shape).to(torch.float8_e4m3fn).view(torch.uint8))
        s.copy_(step * tooth[None, :, None] / unit[:, None])
    c["scales"][2].copy_(torch.where(tooth < 4, 2.0 ** apart, 1.0)[None, :, None].expand(c["scales"][2].shape))
    check_far_apart(run(c), c)


# ---- slices ----

@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("at", [1, 2, 3])
def test_lengths_and_lambda_from_longer_tensors(page, at):
    """The lengths and scales that one call of a step takes, the others take: 4-byte aligned slices."""
    c = make(3, 192, 6, 2, 64, 128, [192, 5, 130], seed=at, page=page, block=64)
    want = run(c).clone()

    def slice_of(t):
        longer = torch.zeros(t.numel() + 8, dtype=t.dtype, device="cuda")
        longer[at:at + t.numel()] = t.flatten()
        return longer[at:at + t.numel()].view(t.shape)

    bounds = [torch.randint(-112, 113, (*p.shape[:1], p.shape[1] // 64, p.shape[2], 2, 64), device="cuda").to(torch.int8)
              for p in c["pools"][:2]]
    choose = lambda c: gda.gda_block_select(c["q1"], c["q2"], *bounds, *c["scales"][:2], c["lens"], 64, 2, block_table=c["table"])
    lists = choose(c)
    some = run(c | {"lists": lists}).clone()
    cut = c | {"lens": slice_of(c["lens"]), "lam": slice_of(c["lam"]), "scales": [slice_of(s) for s in c["scales"]],
               "table": None if c["table"] is None else slice_of(c["table"])}
    assert cut["lens"].data_ptr() % 16 == 4 * at
    assert torch.equal(run(cut), want)
    assert all(torch.equal(a, b) for a, b in zip(choose(cut), lists))
    assert torch.equal(run(cut | {"lists": tuple(map(slice_of, lists))}), some)
