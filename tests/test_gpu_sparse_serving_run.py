"""The operators of an 8-bit block cache together, as a serving loop runs them: prompts and decode steps over pages."""
import numpy as np
import pytest
import torch

import grouped_differential_attention_gb300 as gda
from grouped_differential_attention_gb300 import workloads as W
from oracle import ref_serving as R
from test_gpu_decode_fp8_block import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def device_error_word_stays_clear():
    from grouped_differential_attention_gb300 import build
    build.build()
    gda.gda_device_error(clear=True)
    yield
    assert gda.gda_device_error(clear=True) == 0


@pytest.mark.parametrize("hs,hn,d,dv,ps,block", [(6, 2, 64, 128, 32, 16), (4, 1, 128, 256, 64, 64)])
def test_prompts_then_steps_over_selected_blocks(hs, hn, d, dv, ps, block):
    """Tables, norm and rotation out of the fused projection, rows into the cache, selection, decode over the chosen blocks
    and over all.  The cache and its bounds equal the reference's, the lists the reference's choice from them, and the
    outputs the float64 decode of the values that the cache holds."""
    B, max_pages, keep = 5, 480 // ps, 4
    g = torch.Generator(device="cuda").manual_seed(0)
    pages = B * max_pages
    dims = ((hs, d), (hn, d), (hs, dv))
    cache, bounds = W.empty_fp8_block_cache(pages, ps, block, hs, hn, d, dv, "cuda")
    ref = [[np.zeros((pages * ps, h, n), np.uint8) for h, n in dims],
           [np.zeros((pages * ps // block, h), np.float32) for h, _ in dims],
           [np.zeros((pages * ps // block, h, 2, n), np.int8) for h, n in dims[:2]]]
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    count = torch.tensor([pages], dtype=torch.int32, device="cuda")
    weight = 1 + 0.2 * torch.randn(4, d, generator=g, device="cuda")
    freq = (10000.0 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)).float()
    lam = 0.2 + 0.6 * torch.rand(hs, generator=g, device="cuda")
    width = 2 * (hs + hn) * d + hs * dv
    new_lens = [[140, 1, 0, 400, 17]] + [[1, 1, step // 3, 1, step % 2] for step in range(5)]
    for step, new in enumerate(new_lens):
        rows = sum(new) + 3                                            # padded, as a fixed batch would be
        slot, pos, starts, _, _ = gda.gda_block_tables(
            lens, torch.tensor(new, dtype=torch.int32, device="cuda"), table, free, count, ps, pages, rows,
            out=(torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(rows, dtype=torch.int32, device="cuda"),
                 torch.empty(B + 1, dtype=torch.int32, device="cuda"), lens, count))
        proj = (torch.randn(rows, width, generator=g, device="cuda") * (1 + step)).bfloat16()   # V grows: scales follow
        cuts = [0, hs * d, 2 * hs * d, (2 * hs + hn) * d, 2 * (hs + hn) * d]
        x = [proj[:, a:b].unflatten(-1, (-1, d)) for a, b in zip(cuts, cuts[1:])]
        v = proj[:, cuts[-1]:].unflatten(-1, (hs, dv))
        q1, k1, q2, k2 = gda.gda_qk_norm_rope(*x, weight, pos, freq)
        gda.gda_cache_append_fp8_block(k1, k2, v, slot, *cache, k_sig_bounds=bounds[0], k_noise_bounds=bounds[1])
        for i, t in enumerate((k1, k2, v)):
            R.append_fp8_block(t.cpu(), slot.cpu().numpy(), ref[0][i], ref[1][i], ref[2][i] if i < 2 else None)
            assert np.array_equal(cache[i].view(torch.uint8).flatten(0, 1).cpu().numpy(), ref[0][i])
            assert np.array_equal(cache[3 + i].flatten(0, 1).cpu().numpy(), ref[1][i])
            assert i == 2 or np.array_equal(bounds[i].flatten(0, 1).cpu().numpy(), ref[2][i])
        if step == 0:
            continue
        st = starts.tolist()
        at = torch.tensor([max(st[b + 1] - 1, 0) for b in range(B)], device="cuda")
        a1, a2 = q1[at].contiguous(), q2[at].contiguous()
        lists, counts = gda.gda_block_select(a1, a2, *bounds, *cache[3:5], lens, block, keep, block_table=table)
        want, n = R.block_select(a1.cpu(), a2.cpu(), [t.cpu().numpy() for t in bounds], [t.cpu().numpy() for t in cache[3:5]],
                                 table.cpu().numpy(), lens.tolist(), block, keep, 1, 1)
        assert counts.tolist() == n
        assert lists.tolist() == [[ids + [-1] * (keep - len(ids)) for ids in groups] for groups in want]
        c = dict(q1=a1, q2=a2, pools=cache[:3], scales=cache[3:], table=table.clamp(min=0), lens=lens, lam=lam, block=block,
                 lists=(lists, counts))
        check(gda.gda_attn_decode_sparse_fp8_block(a1, a2, *cache, lists, counts, lens, lam, 0.8, block_table=table), c)
        check(gda.gda_attn_decode_paged_fp8_block(a1, a2, *cache, table, lens, lam, 0.8), c | {"lists": None})


def test_a_captured_step_replayed():
    """Append, selection and decode captured once and replayed for ten tokens, against the same calls one by one."""
    B, hs, hn, d, dv, ps, block, keep = 3, 6, 2, 64, 128, 64, 32, 3
    g = torch.Generator(device="cuda").manual_seed(1)
    runs = [W.empty_fp8_block_cache(B, ps * 3, block, hs, hn, d, dv, "cuda") for _ in range(2)]
    first = [torch.randn(B * 100, h, n, generator=g, device="cuda").bfloat16() for h, n in ((hs, d), (hn, d), (hs, dv))]
    slots = (torch.arange(B, device="cuda")[:, None] * ps * 3 + torch.arange(100, device="cuda")).flatten().to(torch.int32)
    for cache, bounds in runs:
        gda.gda_cache_append_fp8_block(*first, slots, *cache, k_sig_bounds=bounds[0], k_noise_bounds=bounds[1])
    lam = torch.full((hs,), 0.5, device="cuda")
    q1, q2, k1, k2, v = (torch.empty(B, h, n, dtype=torch.bfloat16, device="cuda")
                         for h, n in ((hs, d), (hn, d), (hs, d), (hn, d), (hs, dv)))
    slot, lens = torch.full((B,), -1, dtype=torch.int32, device="cuda"), torch.full((B,), 100, dtype=torch.int32, device="cuda")

    def step(cache, bounds):
        gda.gda_cache_append_fp8_block(k1, k2, v, slot, *cache, k_sig_bounds=bounds[0], k_noise_bounds=bounds[1])
        lists = gda.gda_block_select(q1, q2, *bounds, *cache[3:5], lens, block, keep)
        return gda.gda_attn_decode_sparse_fp8_block(q1, q2, *cache, *lists, lens, lam, 0.8)

    for t in (q1, q2, k1, k2, v):
        t.normal_(generator=g)
    step(*runs[0])                                          # nothing is appended: all slots are -1
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*runs[0])
    for i in range(10):
        for t in (q1, q2, k1, k2, v):
            t.normal_(generator=g)
        slot.copy_(torch.arange(B, device="cuda") * ps * 3 + 100 + i)
        lens.fill_(101 + i)
        graph.replay()
        assert torch.equal(out, step(*runs[1]))
    for a, b in zip((*runs[0][0], *runs[0][1]), (*runs[1][0], *runs[1][1])):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_two_streams_at_once():
    """Two batches, each its cache and stream, appended, selected and decoded side by side, many times."""
    B, hs, hn, d, dv, L, block = 4, 12, 4, 64, 128, 512, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    lam = torch.full((hs,), 0.4, device="cuda")
    lens = torch.tensor([512, 400, 77, 300], dtype=torch.int32, device="cuda")
    sides = []
    for _ in range(2):
        rows = [torch.randn(B * L, h, n, generator=g, device="cuda").bfloat16() for h, n in ((hs, d), (hn, d), (hs, dv))]
        q = [torch.randn(B, h, d, generator=g, device="cuda").bfloat16() for h in (hs, hn)]
        sides.append((rows, q, W.empty_fp8_block_cache(B, L, block, hs, hn, d, dv, "cuda"), torch.cuda.Stream()))
    slots = torch.arange(B * L, dtype=torch.int32, device="cuda")

    def work(rows, q, held):
        cache, bounds = held
        gda.gda_cache_append_fp8_block(*rows, slots, *cache, k_sig_bounds=bounds[0], k_noise_bounds=bounds[1])
        lists = gda.gda_block_select(*q, *bounds, *cache[3:5], lens, block, 3)
        return (gda.gda_attn_decode_sparse_fp8_block(*q, *cache, *lists, lens, lam, 0.8),
                gda.gda_attn_decode_fp8_block(*q, *cache, lens, lam, 0.8), *lists)

    want = [[t.clone() for t in work(*s[:3])] for s in sides]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(sides):
            with torch.cuda.stream(s[3]):
                got[i].append(work(*s[:3]))
    torch.cuda.synchronize()
    for i in range(2):
        for outs in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(outs, want[i]))


def test_chunk_continues_a_prefix_read_from_the_cache():
    """A prefix of 70 rows read back from 8 bits, then a chunk of 30 rows over prefix and chunk."""
    hs, hn, d, dv, Lp, L = 6, 2, 64, 128, 70, 30
    g = torch.Generator(device="cuda").manual_seed(1)
    dims = ((hs, d), (hn, d), (hs, dv))
    rows = [torch.randn(Lp, h, n, generator=g, device="cuda").bfloat16() for h, n in dims]
    cache, _ = W.empty_fp8_block_cache(6, 16, 16, hs, hn, d, dv, "cuda")
    slots = torch.cat([torch.arange(16, device="cuda") + 16 * p for p in (4, 0, 5, 2, 1)])[:Lp].to(torch.int32)
    gda.gda_cache_append_fp8_block(*rows, slots, *cache)
    prefix = gda.gda_cache_read_fp8_block(slots, *cache)
    for x, y in zip(rows, prefix):                          # within half a step of e4m3, 2^-4, or of its smallest, 2^-10 / 448
        amax = x.float().abs().amax((0, 2), keepdim=True)
        assert ((x.float() - y.float()).abs() <= 2.0 ** -4 * x.float().abs() + 2.0 ** -10 / 224 * amax).all()
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
