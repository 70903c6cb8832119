"""The operators together, as a model uses them: a serving run over a 4-bit paged cache, and a training step."""
import pytest
import torch

import grouped_differential_attention_gb300 as gda
from oracle import ref_serving as R
from oracle.ref_torch_grad import gda_backward, gda_grad_magnitudes
from parity import assert_grad_bf16_close
from test_gpu_decode_fp4 import check as check_decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def device_error_word_stays_clear():
    from grouped_differential_attention_gb300 import build
    build.build()
    gda.gda_device_error(clear=True)
    yield
    assert gda.gda_device_error(clear=True) == 0


def test_prompts_then_decode_steps_over_a_paged_cache():
    """A prompt step of ragged chunks and five decode steps: tables, norm and rotation out of the fused projection,
    rows into the cache, decode.  Each decode step is checked in float64 against the values the cache then holds,
    and the cache against the rows that went in."""
    B, hs, hn, d, dv, ps, max_pages = 5, 6, 2, 64, 128, 16, 12
    g = torch.Generator(device="cuda").manual_seed(0)
    width = 2 * (hs + hn) * d + hs * dv
    pages = B * max_pages
    dims = ((hs, d), (hn, d), (hs, dv))
    pools = [torch.zeros(pages, ps, h, n // 2, dtype=torch.uint8, device="cuda") for h, n in dims]
    blocks = [torch.zeros(pages, ps, h, n // 16, dtype=torch.uint8, device="cuda") for h, n in dims]
    scales = [torch.full((h,), 1 / 64, device="cuda") for h, _ in dims]
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    count = torch.tensor([pages], dtype=torch.int32, device="cuda")
    weight = 1 + 0.2 * torch.randn(4, d, generator=g, device="cuda")
    freq = (10000.0 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)).float()
    lam = 0.2 + 0.6 * torch.rand(hs, generator=g, device="cuda")
    held = [[] for _ in range(B)]
    new_lens = [[40, 1, 0, 100, 17]] + [[1, 1, step // 3, 1, step % 2] for step in range(5)]
    for step, new in enumerate(new_lens):
        rows = sum(new) + 3                                            # padded, as a fixed batch would be
        slot, pos, starts, _, _ = gda.gda_block_tables(
            lens, torch.tensor(new, dtype=torch.int32, device="cuda"), table, free, count, ps, pages, rows,
            out=(torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(rows, dtype=torch.int32, device="cuda"),
                 torch.empty(B + 1, dtype=torch.int32, device="cuda"), lens, count))
        proj = torch.randn(rows, width, generator=g, device="cuda").bfloat16()
        cuts = [0, hs * d, 2 * hs * d, (2 * hs + hn) * d, 2 * (hs + hn) * d]
        x = [proj[:, a:b].unflatten(-1, (-1, d)) for a, b in zip(cuts, cuts[1:])]
        v = proj[:, cuts[-1]:].unflatten(-1, (hs, dv))
        q1, k1, q2, k2 = gda.gda_qk_norm_rope(*x, weight, pos, freq)
        gda.gda_cache_append_fp4(k1, k2, v, slot, *pools, *blocks, *scales)
        st = starts.tolist()
        for b in range(B):
            held[b] += [(k1[r], k2[r], v[r]) for r in range(st[b], st[b + 1])]
        assert lens.tolist() == [len(h) for h in held]
        if step == 0:
            continue
        last = torch.tensor([max(st[b + 1] - 1, 0) for b in range(B)], device="cuda")
        c = dict(q1=q1[last].contiguous(), q2=q2[last].contiguous(), pools=pools, blocks=blocks, scales=scales,
                 table=table, lens=lens, lam=lam)
        out = gda.gda_attn_decode_paged_fp4(c["q1"], c["q2"], *pools, *blocks, *scales, table, lens, lam, 0.8)
        check_decode(out, c | {"table": table.clamp(min=0)})
    for b in range(B):                                                  # what the pages hold, read back in order
        n = len(held[b])
        if n == 0:
            continue
        at = torch.arange(n, device="cuda")
        slots = (table[b, at // ps] * ps + at % ps).to(torch.int32)
        for i, y in enumerate(gda.gda_cache_read_fp4(slots, *pools, *blocks, *scales)):
            x = torch.stack([h[i] for h in held[b]])
            codes, s8 = R.quantise_fp4(x.cpu(), scales[i].cpu().numpy())
            assert torch.equal(y.cpu(), torch.from_numpy(R.dequantise_fp4(codes, s8, scales[i].cpu().numpy())).float().bfloat16())


def test_chunk_continues_a_prefix_read_from_the_cache():
    """A prefix of 70 rows read back from 4 bits, then a chunk of 30 rows over prefix and chunk."""
    hs, hn, d, dv, Lp, L = 6, 2, 64, 128, 70, 30
    g = torch.Generator(device="cuda").manual_seed(1)
    dims = ((hs, d), (hn, d), (hs, dv))
    rows = [torch.randn(Lp, h, n, generator=g, device="cuda").bfloat16() for h, n in dims]
    pools = [torch.zeros(6, 16, h, n // 2, dtype=torch.uint8, device="cuda") for h, n in dims]
    blocks = [torch.zeros(6, 16, h, n // 16, dtype=torch.uint8, device="cuda") for h, n in dims]
    scales = [torch.ones(h, device="cuda") for h, _ in dims]
    slots = torch.randperm(96, generator=g, device="cuda")[:Lp].to(torch.int32)
    gda.gda_cache_append_fp4(*rows, slots, *pools, *blocks, *scales)
    prefix = gda.gda_cache_read_fp4(slots, *pools, *blocks, *scales)
    fresh = [torch.randn(L, h, n, generator=g, device="cuda").bfloat16() for h, n in dims]
    k1, k2, v = (torch.cat((a, b))[None].contiguous() for a, b in zip(prefix, fresh))
    q1, q2 = (torch.randn(1, L, h, d, generator=g, device="cuda").bfloat16() for h in (hs, hn))
    lam = torch.full((hs,), 0.5, device="cuda")
    out = gda.gda_attn_fwd_chunk(q1, k1, q2, k2, v, lam, 0.8)
    # the same rows as a decode over a bf16 cache, one query at a time; each is within 3e-3 + 2e-2 |ref| of the truth
    for i in (0, 13, L - 1):
        ref = gda.gda_attn_decode(q1[:, i].contiguous(), q2[:, i].contiguous(), k1, k2, v,
                                  torch.tensor([Lp + i + 1], dtype=torch.int32, device="cuda"), lam, 0.8)
        assert (out[:, i].float() - ref.float()).abs().max() <= 2 * (3e-3 + 2e-2 * ref.float().abs().max())


def test_training_step_gradients():
    """Norm and rotation, attention's gradients, and back through norm and rotation, link by link in float64.

    The chain rounds the rotated projections to bf16 before the attention, and the references take the same values,
    so the attention's gradients obey the bounds of their own test, and the last link those of its own."""
    B, L, hs, hn, d, dv = 2, 100, 6, 2, 64, 128
    g = torch.Generator().manual_seed(2)
    heads = (hs, hs, hn, hn)
    x = [torch.randn(B, L, h, d, generator=g).bfloat16() for h in heads]
    v = torch.randn(B, L, hs, dv, generator=g).bfloat16()
    w = 1 + 0.2 * torch.randn(4, d, generator=g)
    pos = torch.arange(L, dtype=torch.int32)[None].expand(B, L).contiguous()
    freq = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float()
    lam, dy = 0.2 + 0.6 * torch.rand(hs, generator=g), torch.randn(B, L, hs, dv, generator=g).bfloat16()
    dev = [t.cuda() for t in x]
    q1, k1, q2, k2 = gda.gda_qk_norm_rope(*dev, w.cuda(), pos.cuda(), freq.cuda())
    grads = gda.gda_attn_bwd_bf16(q1, k1, q2, k2, v.cuda(), lam.cuda(), 0.8, dy.cuda())
    out = gda.gda_qk_norm_rope_bwd(*dev, w.cuda(), pos.cuda(), freq.cuda(), *grads[:4])
    mid = [t.cpu().double() for t in (q1, k1, q2, k2)]
    args = (*mid, v.double(), lam.double(), 0.8, dy.double())
    ref, mag = gda_backward(*args), gda_grad_magnitudes(*args)
    for i in range(4):
        assert_grad_bf16_close(grads[i], ref[i].numpy(), mag[i].numpy(), "attention gradient %d" % i)
        dx, dw = R.norm_rope_grads(x[i], w[i], pos, freq, grads[i].cpu())
        sx, sw = R.norm_rope_grad_size(x[i], w[i], freq, grads[i].cpu())
        err = (out[i].cpu().double() - dx).abs()
        assert (err <= 2.0 ** -8 * dx.abs() + 2.0 ** -18 * sx).all()
        assert ((out[4][i].cpu().double() - dw).abs() <= 2.0 ** -18 * sw).all()
