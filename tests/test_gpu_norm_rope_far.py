"""Angles of far positions: float32 accuracy at any int32 position.

Rows of +1 and -1 with weights of 1 and eps = 0 have a norm of 1, so an output
is +-cos +- sin.  An angle is reduced to turns and rounded to float32 once (at
most 2^-26 of a turn, 2^-23.3 rad, which moves cos +- sin by 2^-22.8 at most);
the sine and the cosine are off by 2^-24 each (one step below 1), the root and
the products by 2^-22.5, their sum by 2^-24: together below 2^-21.  Sines of
the reference: position = 2^16 a + b, both products with a float32 frequency
exact in float64, joined by the addition theorem (2^-51).
"""
import pytest
import torch

import grouped_differential_attention_gb300 as gda

pytestmark = pytest.mark.gpu
BOUND = 2.0 ** -21


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_differential_attention_gb300 import build
    build.build()


def far_positions(n, seed):
    g = torch.Generator().manual_seed(seed)
    pos = torch.randint(-2 ** 31, 2 ** 31, (n,), generator=g)
    edge = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 24, 2 ** 24 - 1, 2 ** 24 + 1, -2 ** 24, 0, 1, -1, 2 ** 30 + 1,
                         2 ** 22, 123456789])
    pos[:edge.numel()] = edge
    pos[100:200] = pos[100:200] >> 8        # below 2^23
    return pos


def cos_sin(pos, freq):
    """float64 cos and sin of pos * freq, [positions, frequencies]."""
    b = pos % 65536
    x, y = ((t.double()[:, None] * freq.double()) for t in (pos - b, b))
    return x.cos() * y.cos() - x.sin() * y.sin(), x.sin() * y.cos() + x.cos() * y.sin()


def frequencies(kind, rot):
    if kind == "theta":
        return (1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float()
    g = torch.Generator().manual_seed(1)
    return (torch.rand(rot // 2, generator=g) * {"near 1": 1.0, "above 1": 2000.0}[kind] + 0.2).float()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", ["theta", "near 1", "above 1"])
def test_forward(kind, interleaved):
    d = rot = 128
    pos, freq = far_positions(3000, 2), frequencies(kind, rot)
    g = torch.Generator().manual_seed(3)
    x = [(torch.randint(0, 2, (pos.numel(), h, d), generator=g) * 2 - 1).float() for h in (2, 2, 1, 1)]
    out = gda.gda_qk_norm_rope(*(t.cuda() for t in x), torch.ones(4, d, device="cuda"), pos.to(torch.int32).cuda(),
                               freq.cuda(), eps=0.0, interleaved=interleaved)
    c, s = (t[:, None] for t in cos_sin(pos, freq))
    i = torch.arange(rot // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    for t, y in zip(x, out):
        a, b, y = t[..., ia].double(), t[..., ib].double(), y.cpu().double()
        off = torch.maximum((y[..., ia] - (a * c - b * s)).abs(), (y[..., ib] - (b * c + a * s)).abs())
        assert off.max() <= BOUND, float(off.max())


@pytest.mark.parametrize("pos", [2 ** 31 - 1, -2 ** 31, 2 ** 29 + 12345, 1 << 24, 777])
def test_gradient_turns_back_by_the_same_angle(pos):
    """One token and one head: dweight is the turned gradient times the row of ones."""
    d, freq = 64, frequencies("near 1", 64)
    one = torch.ones(1, 1, d, device="cuda")
    dw = gda.gda_qk_norm_rope_bwd(*[one] * 4, torch.ones(4, d, device="cuda"),
                                  torch.tensor([pos], dtype=torch.int32, device="cuda"), freq.cuda(), *[one] * 4,
                                  eps=0.0)[4].cpu().double()
    c, s = cos_sin(torch.tensor([pos]), freq)
    assert (dw - torch.cat((c + s, c - s), -1)).abs().max() <= BOUND
