"""Decode steps of large batches over the 8-bit block cache, and that no shape's outputs hold a NaN."""
import pytest
import torch

import grouped_differential_attention_gb300 as gda
from tests.test_gpu_cache_fp8_block import Cache
from tests.test_gpu_decode_fp8_block import SHAPES, make, pick, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_differential_attention_gb300 import build
    build.build()


@pytest.mark.parametrize("T", [1000, 1500])
@pytest.mark.parametrize("hs,hn,d,dv", [(3, 1, 64, 128), (2, 1, 128, 256)])
def test_one_row_to_each_of_many_blocks(T, hs, hn, d, dv):
    """As many sequences, each with a row of its own in a block of its own, step after step: blocks go on and begin."""
    block = 16
    c = Cache(T, 2 * block, block, hs, hn, d, dv, seed=T)
    g = torch.Generator().manual_seed(T)
    page = torch.randperm(T, generator=g)
    at = torch.randint(0, 8, (T,), generator=g)
    begin = (page * 2 * block).to(torch.int32)
    c.append(c.rows(T, g, 0.05), begin)                                   # the first rows of all sequences
    gda.gda_device_error(clear=True)
    for step, spread in enumerate((0.1, 4.0, 0.01)):
        place = torch.where(torch.arange(T) % 5 == step, block, at + 1 + step)   # some begin their second block
        slots = (page * 2 * block + place).to(torch.int32)
        slots[step::97] = -1                                              # and some have no token
        c.append(c.rows(T, g, spread), slots)
    c.check()
    assert gda.gda_device_error(clear=True) == 0


@pytest.mark.parametrize("d,dv", SHAPES)
def test_outputs_are_numbers(d, dv):
    """(The bound that the decodes' other tests hold outputs to would let a NaN pass.)"""
    lens = [1, 0, 15, 16, 17, 33, 64, 128, 200, 7]
    for hs, hn in ((1, 1), (3, 1), (4, 2), (12, 4), (5, 1), (7, 7), (16, 4)):
        for page in (0, 48):
            c = make(len(lens), 208, hs, hn, d, dv, lens, seed=hs * 7 + d + dv, page=page, powers=hs != 4)
            assert torch.isfinite(run(c)).all()
            c["lists"] = pick(c, 5, seed=hs)
            assert torch.isfinite(run(c)).all()
    for B, L in ((1, 40000), (70, 90), (3, 9001)):
        c = make(B, L, 6, 2, d, dv, [L - 7 * (b % 10) for b in range(B)], seed=B, block=32)
        assert torch.isfinite(run(c)).all()
        c["lists"] = pick(c, 9, seed=B)
        assert torch.isfinite(run(c)).all()
