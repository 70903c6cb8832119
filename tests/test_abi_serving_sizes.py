"""Sizes at the C entries of the operators around the attention (host only)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from grouped_differential_attention_gb300 import build
    build.build()
    import grouped_differential_attention_gb300 as gda
    return gda._load()


UNSUPPORTED_DIMS = [(1, 1), (2, 2), (16, 16), (96, 128), (64, 96), (64, 4096), (4096, 64), (64, 512), (256, 256),
                    (10 ** 9, 10 ** 9), (2 ** 31 - 1, 2 ** 31 - 1), (64, 2 ** 31 - 1)]


def test_fp4_workspace_size_is_zero_for_head_dims_without_a_kernel(lib):
    """In a child process: a size that ends the process fails this test alone."""
    code = ("import grouped_differential_attention_gb300 as gda\n"
            f"for d, dv in {UNSUPPORTED_DIMS}:\n"
            "    for B, hs, hn in ((1, 1, 1), (1, 2, 1), (4, 6, 2), (65535, 127, 1)):\n"
            "        n = gda.gda_attn_decode_fp4_workspace_size(B, hs, hn, d, dv)\n"
            "        assert n == 0, (B, hs, hn, d, dv, n)\n")
    res = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert res.returncode == 0, (res.returncode, res.stderr[-500:])


def test_fp4_workspace_size_of_supported_head_dims(lib):
    for d in (64, 128):
        for dv in (64, 128, 256):
            assert lib.gda_attn_decode_fp4_workspace_size(1, 1, 1, d, dv) > 0
            assert lib.gda_attn_decode_fp4_workspace_size(65535, 127, 1, d, dv) > 0
            assert lib.gda_attn_decode_fp4_workspace_size(65536, 1, 1, d, dv) == 0
            assert lib.gda_attn_decode_fp4_workspace_size(1, 127, 2, d, dv) == 0


def test_head_counts_whose_sum_wraps_are_refused(lib):
    """h_s + h_n past 2^31: every entry refuses them before any device work."""
    from test_abi_serving_host import UNSUPPORTED, append, decode, paged, read, rope, rope_bwd
    big = 2 ** 31 - 1
    for hs, hn in ((big, 1), (big, big), (2 ** 30, 2 ** 30), (big - 128, 1)):
        assert lib.gda_attn_decode_fp4_workspace_size(1, hs, hn, 64, 128) == 0
        assert lib.gda_qk_norm_rope_bwd_workspace_size(1, hs, hn, 64) == 0
        for call in (rope, rope_bwd):
            assert call(lib, hs=hs, hn=hn, T=1) == UNSUPPORTED
        for call in (append, read):
            assert call(lib, hs=hs, hn=hn) == UNSUPPORTED
        for call in (decode, paged):
            assert call(lib, hs=hs, hn=hn, ws_bytes=1 << 60) == UNSUPPORTED


def test_decode_refuses_caches_of_more_than_32_bit_rows(lib):
    """The decode counts cache rows in 32 bits: 2^32 rows are the most, one more would be read as a low one."""
    from test_abi_serving_host import CUDA, UNSUPPORTED, decode, paged
    import torch
    assert decode(lib, B=33, Lcap=1 << 27) == UNSUPPORTED                    # 2^32 + 2^27 rows
    assert decode(lib, B=1025, Lcap=1 << 22) == UNSUPPORTED
    assert paged(lib, ps=16, pages=(1 << 28) + 1) == UNSUPPORTED
    assert paged(lib, ps=3, pages=(1 << 32) // 3 + 1) == UNSUPPORTED
    if not torch.cuda.is_available():
        assert decode(lib, B=32, Lcap=1 << 27) == CUDA                       # 2^32 rows
        assert paged(lib, ps=16, pages=1 << 28) == CUDA
        assert paged(lib, B=256, Lcap=1 << 27, ps=16) == CUDA                # tables may name a page more than once
