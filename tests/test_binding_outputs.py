"""Outputs that the caller hands over come in the call's own number: one too many would shift the pointers and sizes
that follow them at the C entry.  Tensors without memory stand in for CUDA ones; nothing is launched."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import grouped_differential_attention_gb300 as gda

B, L, HS, HN, D, DV, T = 2, 4, 6, 2, 64, 128, 8


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_differential_attention_gb300 import build
    build.build()


def calls():
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    t = lambda *shape, dtype=bf: torch.empty(shape, dtype=dtype, device="cuda:0")
    heads = (HS, HS, HN, HN)
    x, w, pos, freq = [t(T, h, D) for h in heads], t(4, D, dtype=f32), t(T, dtype=i32), t(D // 2, dtype=f32)
    dy = [t(T, h, D, dtype=f32) for h in heads]
    ws = t(1 << 20, dtype=torch.uint8)
    yield "norm_rope", [t(T, h, D) for h in heads], lambda o: gda.gda_qk_norm_rope(*x, w, pos, freq, out=o)
    yield ("norm_rope_bwd", [*(t(T, h, D) for h in heads), t(4, D, dtype=f32)],
           lambda o: gda.gda_qk_norm_rope_bwd(*x, w, pos, freq, *dy, grads=o, workspace=ws))
    yield ("block_tables", [t(n, dtype=i32) for n in (T, T, B + 1, B, 1)],
           lambda o: gda.gda_block_tables(t(B, dtype=i32), t(B, dtype=i32), t(B, 3, dtype=i32), t(9, dtype=i32),
                                          t(1, dtype=i32), 16, 9, T, out=o))
    dims = ((HS, D), (HN, D), (HS, DV))
    cache = [t(3, 16, h, n // 2, dtype=torch.uint8) for h, n in dims] + [t(3, 16, h, n // 16, dtype=torch.uint8)
                                                                         for h, n in dims] + [t(h, dtype=f32) for h, _ in dims]
    yield "cache_read", [t(T, h, n) for h, n in dims], lambda o: gda.gda_cache_read_fp4(t(T, dtype=i32), *cache, out=o)
    for name, dt in (("gda_attn_bwd", f32), ("gda_attn_bwd_bf16", bf)):
        q = [t(B, L, h, D, dtype=dt) for h in heads]
        v, lam, g = t(B, L, HS, DV, dtype=dt), t(HS, dtype=f32), t(B, L, HS, DV, dtype=dt)
        yield (name, [*(t(B, L, h, D, dtype=f32) for h in heads), t(B, L, HS, DV, dtype=f32), t(HS, dtype=f32)],
               lambda o, f=getattr(gda, name), q=q, v=v, lam=lam, g=g: f(*q, v, lam, 0.8, g, grads=o, workspace=ws))


@pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")
def test_wrong_numbers_of_outputs_are_refused():
    with FakeTensorMode():
        for name, outs, call in calls():
            for bad in (outs + [outs[0]], outs + outs, outs[:-1], []):
                with pytest.raises(ValueError, match="tensors"):
                    call(bad)
                    pytest.fail(name)
