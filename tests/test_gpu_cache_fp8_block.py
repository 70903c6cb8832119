"""8-bit cache with block scales on the GPU: bytes, scales and bounds equal the reference's, values read back are exact."""
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


class Cache:
    """The same cache twice: on the device, and as numpy arrays that the reference writes."""

    def __init__(self, pages, ps, block, hs, hn, d, dv, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.dims, self.block, self.ps, self.pages = ((hs, d), (hn, d), (hs, dv)), block, ps, pages
        # what is not written yet is whatever was there
        codes = [torch.randint(0, 256, (pages, ps, h, n), generator=g, dtype=torch.uint8) for h, n in self.dims]
        scale = [torch.rand(pages, ps // block, h, generator=g) for h, _ in self.dims]
        bounds = [torch.randint(-128, 128, (pages, ps // block, h, 2, n), generator=g, dtype=torch.int8)
                  for h, n in self.dims[:2]]
        self.dev = [[t.cuda() for t in x] for x in (codes, scale, bounds)]
        self.ref = [[t.flatten(0, 1).numpy().copy() for t in x] for x in (codes, scale, bounds)]

    def append(self, rows, slots, bounds=True, workspace=None, given=None):
        b = dict(k_sig_bounds=self.dev[2][0], k_noise_bounds=self.dev[2][1]) if bounds else {}
        gda.gda_cache_append_fp8_block(*(given or [t.cuda() for t in rows]), slots.cuda(), *self.dev[0], *self.dev[1],
                                       workspace=workspace, **b)
        for i, x in enumerate(rows):
            R.append_fp8_block(x, slots.numpy(), self.ref[0][i], self.ref[1][i],
                               self.ref[2][i] if bounds and i < 2 else None)

    def check(self):
        torch.cuda.synchronize()
        for i in range(3):
            got, want = self.dev[0][i].flatten(0, 1).cpu().numpy(), self.ref[0][i]
            nan = ((got & 127) == 127) & ((want & 127) == 127)
            assert np.array_equal(got[~nan], want[~nan]), (i, int((got != want)[~nan].sum()))
            assert np.array_equal(self.dev[1][i].flatten(0, 1).cpu().numpy(), self.ref[1][i]), i
            if i < 2:
                assert np.array_equal(self.dev[2][i].flatten(0, 1).cpu().numpy(), self.ref[2][i]), i

    def rows(self, T, g, spread=1.0):
        return [(spread * torch.randn(T, h, n, generator=g) * torch.exp(torch.randn(T, h, 1, generator=g))).bfloat16()
                for h, n in self.dims]

    def value(self, i, slots):
        v = R.e4m3_value(self.ref[0][i][slots]) * self.ref[1][i][np.asarray(slots) // self.block][..., None].astype(np.float64)
        return torch.from_numpy(v)


CASES = [  # T, pages, page size, block, h_s, h_n, d, dv
    (1, 1, 16, 16, 1, 1, 64, 64), (5, 2, 32, 16, 3, 1, 64, 128), (64, 4, 64, 64, 12, 4, 64, 128),
    (77, 3, 96, 32, 16, 4, 128, 256), (300, 2, 256, 128, 6, 2, 128, 64), (1000, 11, 112, 16, 2, 2, 64, 256),
    (333, 3, 128, 128, 5, 1, 64, 128), (1500, 20, 112, 16, 3, 1, 64, 128), (2500, 20, 128, 128, 5, 1, 128, 256),
    (1100, 10, 128, 64, 6, 2, 64, 64), (2049, 70, 32, 32, 9, 3, 128, 128),
]


@pytest.mark.parametrize("order", ["ascending", "shuffled"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_rows_anywhere_in_several_calls(case, order):
    """Four calls with slots anywhere: blocks begin, go on, and begin again over what was there."""
    T, pages, ps, block, hs, hn, d, dv = case
    c = Cache(pages, ps, block, hs, hn, d, dv, seed=T)
    g = torch.Generator().manual_seed(T)
    begin = torch.arange(0, pages * ps, block, dtype=torch.int32)     # every block begun, so that all bytes are defined
    c.append(c.rows(begin.numel(), g, 0.02), begin)
    gda.gda_device_error(clear=True)
    for step, spread in enumerate((0.1, 1.0, 30.0, 1e-3)):
        n = min(T, pages * ps)
        slots = torch.randperm(pages * ps, generator=g)[:n].to(torch.int32)
        if order == "ascending":
            slots = slots.sort().values
        if step % 2:
            slots[slots % block == 0] = -1                            # no block begins: all go on
        rows = c.rows(n, g, spread)
        c.append(rows, slots, bounds=step != 2)
        c.check()
        some = torch.randperm(pages * ps, generator=g)[:min(200, pages * ps)].to(torch.int32)
        some[0] = -7
        back = gda.gda_cache_read_fp8_block(some.cuda(), *c.dev[0], *c.dev[1])
        for i, y in enumerate(back):
            assert (y[0] == 0).all()
            want = c.value(i, some[1:].numpy()).bfloat16()
            y = y[1:].cpu()
            assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.equal(y.nan_to_num(7.0), want.nan_to_num(7.0))
    assert gda.gda_device_error(clear=True) == 0


def test_one_token_a_call_matches_the_values_to_a_growing_scale():
    """A sequence written token by token: values differ from those written at once only by e4m3's subnormals."""
    hs, hn, d, dv, block, n = 3, 1, 64, 128, 32, 80
    one, all_ = (Cache(1, 96, block, hs, hn, d, dv) for _ in range(2))
    g = torch.Generator().manual_seed(5)
    rows = [(t.float() * torch.linspace(0.1, 30, n)[:, None, None]).bfloat16() for t in one.rows(n, g)]
    slots = torch.arange(n, dtype=torch.int32)
    all_.append(rows, slots)
    for t in range(n):
        one.append([x[t:t + 1] for x in rows], slots[t:t + 1])
    one.check()
    for i in range(3):
        assert np.array_equal(one.ref[1][i][:3], all_.ref[1][i][:3])
        a, b = one.value(i, slots.numpy()), all_.value(i, slots.numpy())
        scale = torch.from_numpy(all_.ref[1][i][slots.numpy() // block]).double()[..., None]
        # two roundings to steps of 2^-9 scale, half a step each at most, and their difference is whole steps
        assert ((a - b).abs() <= 2.0 ** -9 * scale).all()


def test_special_values():
    c = Cache(1, 32, 16, 4, 1, 64, 64)
    x = torch.zeros(2, 4, 64).bfloat16()
    x[0, 0, :4] = torch.tensor([float("nan"), float("inf"), -float("inf"), 448.0])
    x[0, 1, :3] = torch.tensor([1e-40, -1e-39, 0.0])                  # below the smallest scale's steps, and zeros
    x[0, 2, :3] = torch.tensor([3.3e38, -3.38e38, 1.0])
    x[1, 3, :8] = torch.tensor([448.0, 1.0625, 1.1875, -1.0625, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10])   # ties
    z = torch.full((2, 1, 64), float("nan")).bfloat16()
    slots = torch.tensor([0, 1], dtype=torch.int32)
    c.append([x, z, x], slots)
    c.check()
    assert (c.dev[2][1][0, 0, 0, 0] == -128).all() and (c.dev[2][1][0, 0, 0, 1] == 127).all()
    back = gda.gda_cache_read_fp8_block(slots.cuda(), *c.dev[0], *c.dev[1])
    assert torch.isnan(back[0][0, 0, :3]).all() and back[0][0, 0, 3] == 448 and torch.isnan(back[1]).all()
    assert torch.isfinite(back[0][:, 1:]).all()
    more = torch.full((1, 4, 64), 2.0).bfloat16()                     # the blocks go on
    c.append([more, more[:, :1], more], torch.tensor([5], dtype=torch.int32))
    c.check()


def test_scales_of_the_callers_own():
    """A block whose scale was not written by the library, of no power of two, goes on."""
    c = Cache(2, 32, 32, 3, 1, 64, 128, seed=9)
    for i in range(3):
        c.ref[0][i] &= 0x77                                           # no NaN codes
        c.dev[0][i].copy_(torch.from_numpy(c.ref[0][i]).view(c.dev[0][i].shape))
    g = torch.Generator().manual_seed(9)
    for spread in (0.1, 500.0):
        c.append(c.rows(3, g, spread), torch.tensor([3, 40, 9], dtype=torch.int32), bounds=False)
        c.check()


def test_slots_past_the_pool_and_the_same_slot_twice():
    c = Cache(2, 16, 16, 3, 1, 64, 128)
    g = torch.Generator().manual_seed(1)
    rows = c.rows(6, g)
    gda.gda_device_error(clear=True)
    c.append(rows, torch.tensor([0, 32, 2, 2 ** 31 - 1, -(2 ** 31), 16], dtype=torch.int32))
    assert gda.gda_device_error(clear=True) == gda.GDA_DEVERR_BAD_PAGE
    c.check()
    back = gda.gda_cache_read_fp8_block(torch.tensor([0, 32, 0], dtype=torch.int32).cuda(), *c.dev[0], *c.dev[1])
    assert gda.gda_device_error(clear=True) == gda.GDA_DEVERR_BAD_PAGE
    assert all((y[1] == 0).all() and torch.equal(y[0], y[2]) for y in back)
    two = [x[:2] for x in c.rows(2, g)]                               # one of the two rows, whole
    slots = torch.tensor([0, 0], dtype=torch.int32)
    gda.gda_cache_append_fp8_block(*(t.cuda() for t in two), slots.cuda(), *c.dev[0], *c.dev[1])
    got = [t[0, 0].cpu().numpy() for t in c.dev[0]]
    wrote = []
    for k in range(2):
        codes = [r.copy() for r in c.ref[0]]
        for i, x in enumerate(two):
            R.append_fp8_block(x[k:k + 1], slots[:1].numpy(), codes[i], c.ref[1][i].copy())
        wrote.append(all(np.array_equal(a, b[0]) for a, b in zip(got, codes)))
    assert any(wrote)


def test_fused_projection_other_stream_and_any_workspace():
    hs, hn, d, dv, T = 6, 2, 64, 128, 1050
    g = torch.Generator().manual_seed(2)
    proj = torch.randn(T, hs * (d + dv) + hn * d + 24, generator=g).bfloat16()
    cuts = (0, hs * d, (hs + hn) * d, (hs + hn) * d + hs * dv)
    split = lambda p: [p[:, a:b].unflatten(-1, (-1, n)) for a, b, n in zip(cuts, cuts[1:], (d, d, dv))]
    c = Cache(25, 48, 16, hs, hn, d, dv)
    slots = torch.arange(40, 40 + T, dtype=torch.int32)
    slots[10] = 0
    s = torch.cuda.Stream()
    need = gda.gda_cache_append_fp8_block_workspace_size(T, 25, 48)
    assert need == 4 * 25 * 48
    with torch.cuda.stream(s):
        for fill in (0, 0xFF, 0x01):                                  # 0x01: rows that do not have the slot
            ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
            c.append(split(proj), slots, workspace=ws, given=split(proj.cuda()))
    c.check()


def test_rows_far_into_a_large_pool():
    """Byte offsets beyond 2^32: the last slots of a pool of 9.4 GB of V codes."""
    hs, hn, d, dv, ps, block = 64, 1, 64, 256, 64, 64
    pages = 9000
    V = torch.zeros(pages, ps, hs, dv, dtype=torch.uint8, device="cuda")
    assert V.numel() > 1 << 33
    pools = [torch.zeros(pages, ps, h, d, dtype=torch.uint8, device="cuda") for h in (hs, hn)] + [V]
    scales = [torch.zeros(pages, 1, h, device="cuda") for h in (hs, hn, hs)]
    g = torch.Generator().manual_seed(4)
    rows = [torch.randn(2, h, n, generator=g).bfloat16() for h, n in ((hs, d), (hn, d), (hs, dv))]
    slots = torch.tensor([pages * ps - 1, pages * ps - 64], dtype=torch.int32, device="cuda")
    gda.gda_cache_append_fp8_block(*(t.cuda() for t in rows), slots, *pools, *scales)
    back = gda.gda_cache_read_fp8_block(slots, *pools, *scales)
    for x, y in zip(rows, back):
        codes, scale = np.zeros((64, *x.shape[1:]), np.uint8), np.zeros((1, x.shape[1]), np.float32)
        R.append_fp8_block(x, [63, 0], codes, scale)
        want = torch.from_numpy(R.e4m3_value(codes[[63, 0]]) * scale[0][:, None])
        assert torch.equal(y.cpu().double(), want)
    assert int(torch.count_nonzero(V)) == int(torch.count_nonzero(V.view(-1, hs, dv)[slots.long()]))


def test_captured_and_replayed():
    c = Cache(2, 64, 64, 6, 2, 64, 128)
    g = torch.Generator().manual_seed(6)
    c.append(c.rows(2, g), torch.tensor([0, 64], dtype=torch.int32))
    rows, slots = [t.cuda() for t in c.rows(2, g)], torch.zeros(2, dtype=torch.int32, device="cuda")
    ws = torch.empty(16, dtype=torch.uint8, device="cuda")            # few rows: its size does not matter
    graph = torch.cuda.CUDAGraph()
    slots.fill_(-1)
    with torch.cuda.graph(graph):
        gda.gda_cache_append_fp8_block(*rows, slots, *c.dev[0], *c.dev[1], k_sig_bounds=c.dev[2][0],
                                       k_noise_bounds=c.dev[2][1], workspace=ws)
    for step in range(1, 5):
        new = c.rows(2, g, 2.0 ** step)
        at = torch.tensor([step, 64 + step], dtype=torch.int32)
        for a, b in zip(rows, new):
            a.copy_(b)
        slots.copy_(at)
        graph.replay()
        for i, x in enumerate(new):
            R.append_fp8_block(x, at.numpy(), c.ref[0][i], c.ref[1][i], c.ref[2][i] if i < 2 else None)
        c.check()


def test_binding_refuses():
    c = Cache(2, 32, 16, 4, 2, 64, 128)
    g = torch.Generator().manual_seed(1)
    good = [*(t.cuda() for t in c.rows(4, g)), torch.arange(4, dtype=torch.int32, device="cuda"), *c.dev[0], *c.dev[1]]
    for i, t in enumerate(good):
        for other in (t.cpu(), t.double(), t[:, :1] if t.dim() > 1 else t[:1]):
            bad = list(good)
            bad[i] = other
            with pytest.raises((TypeError, ValueError, gda.GDAError)):
                gda.gda_cache_append_fp8_block(*bad)
            if i > 2 and other.device.type == "cpu":
                with pytest.raises((TypeError, ValueError)):
                    gda.gda_cache_read_fp8_block(*bad[3:])
    with pytest.raises(ValueError):
        gda.gda_cache_append_fp8_block(*good, k_sig_bounds=c.dev[2][0])
    with pytest.raises((TypeError, ValueError)):
        gda.gda_cache_append_fp8_block(*good, k_sig_bounds=c.dev[2][1], k_noise_bounds=c.dev[2][0])
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    many = [t[:1].expand(1025, *t.shape[1:]).contiguous() for t in good[:4]]
    with pytest.raises(gda.GDAError):
        gda.gda_cache_append_fp8_block(*many, *good[4:], workspace=small)
