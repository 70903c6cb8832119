"""Rows of the 4-bit decode near both ends of float32: the norm's squares are past it, the rows are not."""
import pytest
import torch

from tests.test_gpu_decode_fp4 import make, reference, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_differential_attention_gb300 import build
    build.build()


@pytest.mark.parametrize("power", [90, 70, 64, 50, 40, -40, -63, -90])
@pytest.mark.parametrize("B,L,hs,hn,d,dv,page", [(3, 200, 6, 2, 64, 128, 48), (1, 9000, 3, 1, 64, 64, 0),
                                                 (20, 300, 4, 2, 128, 256, 0)])
def test_values_of_any_size(B, L, hs, hn, d, dv, page, power):
    """(The bound is that of tests/test_gpu_decode_fp4.py.)"""
    c = make(B, L, hs, hn, d, dv, [max(1, L - 37 * b) for b in range(B)], seed=power + 200, page=page)
    c["scales"][2] *= 2.0 ** power
    eps = 1e-5 if power > 0 else 0.0
    got = run(c, eps=eps).double()
    ref, mag = reference(c, eps)
    rms = lambda t: (t * t).mean(-1, keepdim=True).sqrt()
    assert torch.isfinite(got).all()
    assert ((got - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -9 * (mag + ref.abs() * rms(mag) / rms(ref))).all()
