"""Pins of the 64-bit references in oracle/ref_serving.py (CPU)."""
import numpy as np
import pytest
import torch

from oracle import ref_serving as R


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [16, 48, 64])
def test_rotation_keeps_pair_lengths_and_undoes_itself(rot, interleaved):
    g = torch.Generator().manual_seed(rot)
    x = torch.randn(5, 3, 64, generator=g, dtype=torch.float64)
    w = torch.ones(64, dtype=torch.float64)
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    pos = torch.tensor([0, 1, 7, -3, 100000])
    y = R.norm_rope(x, w, pos, freq, 0.0, interleaved)
    n = x / x.square().mean(-1, keepdim=True).sqrt()
    assert torch.equal(y[0], n[0])                                   # position 0 turns nothing
    assert torch.equal(y[..., rot:], n[..., rot:])
    ia, ib = R._pair_index(rot, interleaved)
    assert torch.allclose(y[..., ia] ** 2 + y[..., ib] ** 2, n[..., ia] ** 2 + n[..., ib] ** 2, rtol=1e-12)
    z = torch.complex(n[..., ia], n[..., ib]) * torch.exp(1j * pos[:, None, None] * freq)
    assert torch.allclose(y[..., ia], z.real, atol=1e-11) and torch.allclose(y[..., ib], z.imag, atol=1e-11)


def test_gradients_match_central_differences():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(2, 2, 64, generator=g, dtype=torch.float64)
    w = 1 + 0.2 * torch.randn(64, generator=g, dtype=torch.float64)
    freq = 100.0 ** (-torch.arange(0, 32, 2, dtype=torch.float64) / 32)
    pos, dy = torch.tensor([3, 11]), torch.randn(2, 2, 64, generator=g, dtype=torch.float64)
    dx, dw = R.norm_rope_grads(x, w, pos, freq, dy)
    h = 1e-6
    for i in (0, 5, 31, 32, 63):
        e = torch.zeros(64, dtype=torch.float64)
        e[i] = h
        fd = ((R.norm_rope(x, w + e, pos, freq) - R.norm_rope(x, w - e, pos, freq)) * dy).sum() / (2 * h)
        assert abs(fd - dw[i]) <= 1e-7 * (1 + abs(dw[i]))
        up, dn = x.clone(), x.clone()
        up[1, 0, i] += h
        dn[1, 0, i] -= h
        fd = ((R.norm_rope(up, w, pos, freq) - R.norm_rope(dn, w, pos, freq)) * dy).sum() / (2 * h)
        assert abs(fd - dx[1, 0, i]) <= 1e-7 * (1 + abs(dx[1, 0, i]))


def test_every_code_and_scale_survives_a_round_trip():
    for s in (2.0 ** -6, 0.40625, 1.0, 448.0):
        v = np.concatenate([R.E2M1, -R.E2M1]) * s
        x = torch.tensor(v, dtype=torch.float32).bfloat16()[None, None]
        assert torch.equal(x.double(), torch.tensor(v)[None, None])
        codes, blocks = R.quantise_fp4(x, [1.0])
        assert np.array_equal(R.dequantise_fp4(codes, blocks, [1.0])[0, 0], v)
        assert np.array_equal(R.unpack(R.pack(codes)), codes)


def test_half_way_points_go_to_the_even_code():
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    x = torch.tensor([6.0] + ties + [-t for t in ties] + [0.0]).bfloat16()[None, None]
    codes, _ = R.quantise_fp4(x, [1.0])
    assert codes[0, 0].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 8, 10, 10, 12, 12, 14, 14, 0]


def test_zero_tiny_infinite_and_nan_blocks():
    x = torch.zeros(5, 1, 16)
    x[1, 0, 3] = 2.0 ** -12            # below half the smallest e4m3 step times 6: the block is zero
    x[2, 0, 0], x[2, 0, 1] = float("inf"), 1.0
    x[3, 0, 5] = float("nan")
    x[4, 0, 0] = 3e38                  # saturates
    codes, blocks = R.quantise_fp4(x.bfloat16(), [1.0])
    v = R.dequantise_fp4(codes, blocks, [1.0])
    assert (v[:2] == 0).all()
    assert v[2, 0, 0] == 2688 and v[2, 0, 1] == 0 and v[4, 0, 0] == 2688
    assert np.isnan(v[3]).all()


def test_block_tables_of_a_small_step():
    table = np.array([[5, -1], [7, 2], [-1, -1]])
    out = R.block_tables([3, 6, 0], [2, 1, 0], table, [9, 8, 4], 3, 4, 16, 5)
    slots, pos, starts, lens, left, t = out
    assert starts == [0, 2, 3, 3] and lens == [5, 7, 0] and left == 2
    assert slots == [5 * 4 + 3, 4 * 4 + 0, 2 * 4 + 2, -1, -1] and pos == [3, 4, 6, 0, 0]
    assert t.tolist() == [[5, 4], [7, 2], [-1, -1]]
