"""Run one named workload a few times through the public API (for profilers).

    python -m grouped_differential_attention_gb300.run_workload prefill \
        gda_3to1_prefill_bf16_B4_L2048_h12+4_d64_dv128 --launches 3
    python -m grouped_differential_attention_gb300.run_workload decode --launches 3
    python -m grouped_differential_attention_gb300.run_workload decode_fp8 --launches 3
    python -m grouped_differential_attention_gb300.run_workload decode_fp4 --launches 3
    python -m grouped_differential_attention_gb300.run_workload decode_fp8_block --launches 3
    python -m grouped_differential_attention_gb300.run_workload decode_sparse --launches 3
    python -m grouped_differential_attention_gb300.run_workload norm_rope --launches 3
    python -m grouped_differential_attention_gb300.run_workload norm_rope_backward --launches 3
    python -m grouped_differential_attention_gb300.run_workload serving_step --launches 3
    python -m grouped_differential_attention_gb300.run_workload sparse_serving_step --launches 3
    python -m grouped_differential_attention_gb300.run_workload backward --launches 1
    python -m grouped_differential_attention_gb300.run_workload backward_bf16 --launches 3
    python -m grouped_differential_attention_gb300.run_workload prefill2pass --launches 3

Inputs are the seeded synthetic tensors of ``workloads``; prints the mean
device time per launch measured with CUDA events (not meaningful under a
profiler).
"""
from __future__ import annotations

import argparse
import sys

import torch

import grouped_differential_attention_gb300 as gda
from grouped_differential_attention_gb300 import workloads as W


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("kind", choices=["prefill", "prefill2pass", "decode", "decode_fp8", "decode_fp4", "decode_fp8_block",
                                     "decode_sparse", "backward", "backward_bf16", "norm_rope", "norm_rope_backward",
                                     "serving_step", "sparse_serving_step"])
    ap.add_argument("workload", nargs="?", default=None)
    ap.add_argument("--launches", type=int, default=3)
    ap.add_argument("--flags", type=int, default=0, help="gda_attn_fwd_ex flags for the prefill kind")
    args = ap.parse_args(argv)
    dev = torch.device("cuda:0")
    if args.kind == "prefill":
        w = W.PREFILL_WORKLOADS[args.workload or W.GDA3_PREFILL_L2048.name]
        inp = [t.to(dev) for t in W.make_prefill_inputs(w)]
        fn = gda.gda_attn_fwd if w.dtype == "bf16" else gda.gda_attn_fwd_f32
        out = torch.empty((w.B, w.L, w.h_s, w.dv), dtype=inp[0].dtype, device=dev)

        def launch():
            fn(*inp, w.lambda_init, causal=w.causal, eps=w.eps, out=out, flags=args.flags)
    elif args.kind == "prefill2pass":
        w = W.PREFILL_WORKLOADS[args.workload or W.GDA3_PREFILL_L2048.name]
        inp = [t.to(dev) for t in W.make_prefill_inputs(w)]
        out = torch.empty((w.B, w.L, w.h_s, w.dv), dtype=torch.bfloat16, device=dev)
        ws = torch.empty(gda.gda_attn_fwd_2pass_workspace_size(w.B, w.L, w.h_s, w.h_n), dtype=torch.uint8,
                         device=dev)

        def launch():
            gda.gda_attn_fwd_2pass(*inp, w.lambda_init, causal=w.causal, eps=w.eps, out=out, workspace=ws)
    elif args.kind == "backward_bf16":
        w = W.PREFILL_WORKLOADS[args.workload or W.GDA3_PREFILL_L2048.name]
        inp = [t.to(dev) for t in W.make_backward_inputs(w)]
        ws = torch.empty(gda.gda_attn_bwd_bf16_workspace_size(w.B, w.L, w.h_s, w.h_n, w.dv), dtype=torch.uint8,
                         device=dev)
        grads = gda.gda_attn_bwd_bf16(*inp[:6], w.lambda_init, inp[6], causal=w.causal, eps=w.eps, workspace=ws)

        def launch():
            gda.gda_attn_bwd_bf16(*inp[:6], w.lambda_init, inp[6], causal=w.causal, eps=w.eps, workspace=ws,
                                  grads=grads)
    elif args.kind == "backward":
        # float32 gradients at a prefill workload's sizes (default: the 3:1 B=4 L=2048 one)
        w = W.PREFILL_WORKLOADS[args.workload or W.GDA3_PREFILL_L2048.name]
        inp = [t.to(dev) for t in W.make_backward_inputs(w, dtype="f32")]
        ws = torch.empty(gda.gda_attn_bwd_workspace_size(w.B, w.L, w.h_s, w.d, w.dv), dtype=torch.uint8,
                         device=dev)
        grads = gda.gda_attn_bwd(*inp[:6], w.lambda_init, inp[6], causal=w.causal, eps=w.eps, workspace=ws)

        def launch():
            gda.gda_attn_bwd(*inp[:6], w.lambda_init, inp[6], causal=w.causal, eps=w.eps, workspace=ws,
                             grads=grads)
    elif args.kind == "decode_fp8":
        w = W.GDA3_DECODE_B64
        inp = [t.to(dev) for t in W.make_decode_inputs_fp8(w)]
        out = torch.empty((w.B, w.h_s, w.dv), dtype=torch.bfloat16, device=dev)
        ws = torch.empty(gda.gda_attn_decode_workspace_size(w.B, w.Lcap, w.h_s, w.h_n, w.dv),
                         dtype=torch.uint8, device=dev)

        def launch():
            gda.gda_attn_decode_fp8(*inp, w.lambda_init, eps=w.eps, out=out, workspace=ws)
    elif args.kind == "decode_fp4":
        w = W.GDA3_DECODE_B64
        q1, q2, k1c, k2c, vc, lens, lam = [t.to(dev) for t in W.make_decode_inputs(w)]
        cache = W.empty_fp4_cache(w.B, w.Lcap, w.h_s, w.h_n, w.d, w.dv, dev)
        gda.gda_cache_append_fp4(*(t.flatten(0, 1) for t in (k1c, k2c, vc)),
                                 torch.arange(w.B * w.Lcap, dtype=torch.int32, device=dev), *cache)
        out = torch.empty((w.B, w.h_s, w.dv), dtype=torch.bfloat16, device=dev)
        ws = torch.empty(gda.gda_attn_decode_fp4_workspace_size(w.B, w.h_s, w.h_n, w.d, w.dv), dtype=torch.uint8,
                         device=dev)

        def launch():
            gda.gda_attn_decode_fp4(q1, q2, *cache, lens, lam, w.lambda_init, eps=w.eps, out=out, workspace=ws)
    elif args.kind in ("decode_fp8_block", "decode_sparse"):
        # 8-bit caches with a scale for 64 tokens; sparse: 16 blocks of each sequence, chosen in each launch
        w, block, keep = W.GDA3_DECODE_B64, 64, 16
        q1, q2, k1c, k2c, vc, lens, lam = [t.to(dev) for t in W.make_decode_inputs(w)]
        cache, bounds = W.empty_fp8_block_cache(w.B, w.Lcap, block, w.h_s, w.h_n, w.d, w.dv, dev)
        gda.gda_cache_append_fp8_block(*(t.flatten(0, 1) for t in (k1c, k2c, vc)),
                                       torch.arange(w.B * w.Lcap, dtype=torch.int32, device=dev), *cache,
                                       k_sig_bounds=bounds[0], k_noise_bounds=bounds[1])
        out = torch.empty((w.B, w.h_s, w.dv), dtype=torch.bfloat16, device=dev)
        ws = torch.empty(gda.gda_attn_decode_fp8_block_workspace_size(w.B, w.h_s, w.h_n, w.d, w.dv), dtype=torch.uint8,
                         device=dev)
        if args.kind == "decode_fp8_block":
            def launch():
                gda.gda_attn_decode_fp8_block(q1, q2, *cache, lens, lam, w.lambda_init, eps=w.eps, out=out, workspace=ws)
        else:
            def launch():
                lists = gda.gda_block_select(q1, q2, *bounds, *cache[3:5], lens, block, keep)
                gda.gda_attn_decode_sparse_fp8_block(q1, q2, *cache, *lists, lens, lam, w.lambda_init, eps=w.eps, out=out,
                                                     workspace=ws)
    elif args.kind in ("norm_rope", "norm_rope_backward"):
        # the projections of a prefill workload (default: the 3:1 B=4 L=2048 one) before its attention
        w = W.PREFILL_WORKLOADS[args.workload or W.GDA3_PREFILL_L2048.name]
        q1, k1, q2, k2 = [t.to(dev) for t in W.make_prefill_inputs(w)[:4]]
        weight = torch.ones((4, w.d), device=dev)
        pos = torch.arange(w.L, dtype=torch.int32, device=dev).expand(w.B, w.L).contiguous()
        freq = (10000.0 ** (-torch.arange(0, w.d, 2, dtype=torch.float64) / w.d)).float().to(dev)
        x = (q1, k1, q2, k2)
        if args.kind == "norm_rope":
            out = tuple(torch.empty_like(t) for t in x)

            def launch():
                gda.gda_qk_norm_rope(*x, weight, pos, freq, out=out)
        else:
            dy = [torch.randn_like(t, dtype=torch.float32) for t in x]
            ws = torch.empty(gda.gda_qk_norm_rope_bwd_workspace_size(w.B * w.L, w.h_s, w.h_n, w.d), dtype=torch.uint8,
                             device=dev)
            grads = gda.gda_qk_norm_rope_bwd(*x, weight, pos, freq, *dy, workspace=ws)

            def launch():
                gda.gda_qk_norm_rope_bwd(*x, weight, pos, freq, *dy, grads=grads, workspace=ws)
    elif args.kind in ("serving_step", "sparse_serving_step"):
        # one new token for each sequence of the decode workload: its page and slot, norm and rotation, the row into a
        # paged cache of 4 bits, and the decode over it; sparse: of 8 bits with a scale for a page, the choice of 16 pages
        # and the decode over those (the cache's values are whatever zeroed pages hold)
        w, page = W.GDA3_DECODE_B64, 64
        rows = [t.to(dev) for t in W.make_prefill_inputs(W.GDA3_PREFILL_L2048, B=w.B, L=1, h_s=w.h_s, h_n=w.h_n, d=w.d,
                                                         dv=w.dv)]
        q1, k1, q2, k2, v = [t.view(w.B, t.shape[2], t.shape[3]) for t in rows[:5]]
        lam = rows[5]
        lens = torch.randint(w.len_range[0], w.len_range[1] - args.launches, (w.B,),
                             generator=torch.Generator().manual_seed(w.seed)).to(torch.int32).to(dev)
        per = -(-w.Lcap // page)
        sparse = args.kind == "sparse_serving_step"
        if sparse:
            cache, bounds = W.empty_fp8_block_cache(w.B * per, page, page, w.h_s, w.h_n, w.d, w.dv, dev)
        else:
            cache = W.empty_fp4_cache(w.B * per, page, w.h_s, w.h_n, w.d, w.dv, dev)
        table = torch.arange(w.B * per, dtype=torch.int32, device=dev).view(w.B, per)
        held = (lens.cpu() + page - 1) // page
        free = torch.cat([table[b, n:].cpu() for b, n in enumerate(held.tolist())]).to(dev)
        count = torch.tensor([free.numel()], dtype=torch.int32, device=dev)
        ones = torch.ones(w.B, dtype=torch.int32, device=dev)
        step = [torch.empty(n, dtype=torch.int32, device=dev) for n in (w.B, w.B, w.B + 1)]
        weight = torch.ones((4, w.d), device=dev)
        freq = (10000.0 ** (-torch.arange(0, w.d, 2, dtype=torch.float64) / w.d)).float().to(dev)
        out = torch.empty((w.B, w.h_s, w.dv), dtype=torch.bfloat16, device=dev)
        size = gda.gda_attn_decode_fp8_block_workspace_size if sparse else gda.gda_attn_decode_fp4_workspace_size
        ws = torch.empty(size(w.B, w.h_s, w.h_n, w.d, w.dv), dtype=torch.uint8, device=dev)

        def launch():
            slot, pos, *_ = gda.gda_block_tables(lens, ones, table, free, count, page, w.B * per, w.B,
                                                 out=(*step, lens, count))
            a1, b1, a2, b2 = gda.gda_qk_norm_rope(q1, k1, q2, k2, weight, pos, freq, eps=w.eps)
            if sparse:
                gda.gda_cache_append_fp8_block(b1, b2, v, slot, *cache, k_sig_bounds=bounds[0], k_noise_bounds=bounds[1])
                lists = gda.gda_block_select(a1, a2, *bounds, *cache[3:5], lens, page, 16, block_table=table)
                gda.gda_attn_decode_sparse_fp8_block(a1, a2, *cache, *lists, lens, lam, w.lambda_init, block_table=table,
                                                     eps=w.eps, out=out, workspace=ws)
            else:
                gda.gda_cache_append_fp4(b1, b2, v, slot, *cache)
                gda.gda_attn_decode_paged_fp4(a1, a2, *cache, table, lens, lam, w.lambda_init, eps=w.eps, out=out,
                                              workspace=ws)
    else:
        w = W.GDA3_DECODE_B64
        inp = [t.to(dev) for t in W.make_decode_inputs(w)]
        out = torch.empty((w.B, w.h_s, w.dv), dtype=torch.bfloat16, device=dev)
        ws = torch.empty(gda.gda_attn_decode_workspace_size(w.B, w.Lcap, w.h_s, w.h_n, w.dv),
                         dtype=torch.uint8, device=dev)

        def launch():
            gda.gda_attn_decode(*inp, w.lambda_init, eps=w.eps, out=out, workspace=ws)

    launch()
    torch.cuda.synchronize()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    for _ in range(args.launches):
        launch()
    e1.record()
    torch.cuda.synchronize()
    err = gda.gda_device_error(clear=True)
    print(f"{w.name}: {e0.elapsed_time(e1) / args.launches:.4f} ms per launch, device error word {err}")
    return 0 if err == 0 else 1


if __name__ == "__main__":
    sys.exit(main())
