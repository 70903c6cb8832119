"""Host-side checks of the 8-bit cache with block scales, its decodes and the selection: bad arguments get their
documented status before any device work, and the binding refuses host tensors."""
import ctypes

import numpy as np
import pytest
import torch

INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE, CUDA = -1, -2, -3, -4, -5
A = 0x10000   # 16-byte aligned, never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    from grouped_differential_attention_gb300 import build
    build.build()
    import grouped_differential_attention_gb300 as gda
    return gda._load()


def ptrs(n, **change):
    p = [A + 4096 * i for i in range(n)]
    for k, v in change.items():
        p[int(k[1:])] = v
    return [ctypes.c_void_p(x) for x in p]


def append(lib, p=None, T=5, pages=4, ps=64, block=32, hs=6, hn=2, d=64, dv=128, s=None, ws=A, ws_bytes=None):
    s = s or [hs * d, hn * d, hs * dv]
    need = lib.gda_cache_append_fp8_block_workspace_size(T, pages, ps)
    return lib.gda_cache_append_fp8_block(*(p or ptrs(12)), T, pages, ps, block, hs, hn, d, dv, *s, ws,
                                          need if ws_bytes is None else ws_bytes, None)


def read(lib, p=None, T=5, pages=4, ps=64, block=32, hs=6, hn=2, d=64, dv=128):
    return lib.gda_cache_read_fp8_block(*(p or ptrs(10)), T, pages, ps, block, hs, hn, d, dv, None)


@pytest.mark.parametrize("call,n", [(append, 12), (read, 10)])
def test_cache_rows_refuse(lib, call, n):
    for i in range(n):
        assert call(lib, p=ptrs(n, **{f"p{i}": None})) == INVALID       # one of the two bounds alone, too
        assert call(lib, p=ptrs(n, **{f"p{i}": A + 2})) == MISALIGNED
    for bad in (dict(T=0), dict(pages=0), dict(ps=0), dict(block=0), dict(block=-16), dict(hs=6, hn=4), dict(ps=80),
                dict(pages=1 << 20, ps=1 << 11), dict(d=0), dict(dv=-1)):
        assert call(lib, **bad) == INVALID
    for bad in (dict(d=96), dict(dv=96), dict(hs=128, hn=1), dict(hs=2 ** 31 - 1, hn=1), dict(block=8), dict(block=64, ps=192, d=32),
                dict(ps=48, block=48), dict(ps=256, block=256)):
        args = dict(s=[1 << 39] * 3) | bad if call is append else bad
        assert call(lib, **args) == UNSUPPORTED
    if not torch.cuda.is_available():
        assert call(lib) == CUDA
        if call is append:
            assert append(lib, p=ptrs(12, p10=None, p11=None)) == CUDA  # no bounds kept


def test_append_strides_and_workspace(lib):
    assert append(lib, s=[383, 128, 768]) == INVALID and append(lib, s=[384, 132, 768]) == MISALIGNED
    assert append(lib, s=[384, 128, (1 << 40) + 8]) == INVALID
    assert append(lib, T=1025, ws=None) == WORKSPACE and append(lib, T=1025, ws=A + 8) == WORKSPACE
    assert append(lib, T=1025, ws_bytes=4 * 64 * 4 - 1) == WORKSPACE
    size = lib.gda_cache_append_fp8_block_workspace_size
    assert size(1025, 4, 64) == 1024 and size(1024, 4, 64) == 0 and size(0, 4, 64) == 0
    assert size(9999, 0, 64) == 0 and size(9999, 4, 0) == 0 and size(9999, 1 << 20, 1 << 11) == 0
    assert size(2 ** 31 - 1, 1, 2 ** 31 - 1) == 4 * (2 ** 31 - 1)
    if not torch.cuda.is_available():
        assert append(lib, ws=None) == CUDA                             # few rows: none is needed


def select(lib, p=None, B=3, mp=4, ps=64, pages=9, block=32, keep=5, first=1, last=1, hs=6, hn=2, d=64, ws=A,
           ws_bytes=None):
    need = lib.gda_block_select_workspace_size(B, mp * (ps // block) if block > 0 else 1, hs, hn)
    return lib.gda_block_select(*(p or ptrs(10)), B, mp, ps, pages, block, keep, first, last, hs, hn, d, ws,
                                need if ws_bytes is None else ws_bytes, None)


def test_select_refuses(lib):
    for i in range(10):
        assert select(lib, p=ptrs(10, **{f"p{i}": None})) == INVALID    # no table: pages for each sequence do not fit
        assert select(lib, p=ptrs(10, **{f"p{i}": A + 2})) == MISALIGNED
    for bad in (dict(B=0), dict(mp=0), dict(ps=0), dict(pages=0), dict(block=0), dict(ps=80), dict(keep=0),
                dict(first=-1), dict(last=-1), dict(first=3, last=3), dict(first=6, last=0), dict(hs=6, hn=4), dict(d=0),
                dict(mp=1 << 20, ps=1 << 11), dict(first=2 ** 31 - 1, last=2 ** 31 - 1)):
        assert select(lib, **bad) == INVALID
    for bad in (dict(d=96), dict(hs=128, hn=1), dict(B=65536), dict(block=8), dict(mp=32768, ps=32, block=16),
                dict(mp=32769, ps=32), dict(pages=2 ** 31 - 1)):
        assert select(lib, **bad) == UNSUPPORTED
    many = dict(mp=8192, ps=32, pages=1, hs=80)             # x of 40 heads of a group does not fit
    assert select(lib, ws=None, **many) == WORKSPACE and select(lib, ws=A + 8, **many) == WORKSPACE
    assert select(lib, ws_bytes=3 * 8192 * 82 * 4 - 1, **many) == WORKSPACE
    if not torch.cuda.is_available():
        assert select(lib) == CUDA and select(lib, p=ptrs(10, p6=None), mp=1, pages=3) == CUDA
        assert select(lib, mp=32768, ps=32, pages=1) == CUDA            # the most blocks
        assert select(lib, ws=None) == CUDA and select(lib, **many) == CUDA
    size = lib.gda_block_select_workspace_size
    assert size(3, 8, 6, 2) == 0 and size(3, 30000, 6, 2) == 0 and size(3, 10000, 24, 1) == 0
    assert size(3, 8192, 80, 2) == 3 * 8192 * 82 * 4 and size(1, 32768, 127, 1) == 32768 * 128 * 4
    assert size(0, 8192, 80, 2) == 0 and size(3, 32769, 80, 2) == 0 and size(3, 8192, 80, 3) == 0
    assert size(65536, 8192, 80, 2) == 0 and size(3, 8192, 127, 2) == 0


def decode(lib, p=None, kind="whole", B=4, Lcap=64, block=32, hs=6, hn=2, d=64, dv=128, lam0=0.8, eps=1e-5, ws=A,
           ws_bytes=None, ps=32, pages=9, keep=3, table=A, lists=(A, A)):
    p = p or ptrs(11)
    need = lib.gda_attn_decode_fp8_block_workspace_size(B, hs, hn, d, dv)
    tail = (hs, hn, d, dv, eps, ws, need if ws_bytes is None else ws_bytes, None)
    if kind == "whole":
        return lib.gda_attn_decode_fp8_block(*p[:10], lam0, p[10], B, Lcap, block, *tail)
    if kind == "paged":
        return lib.gda_attn_decode_paged_fp8_block(*p[:8], table, *p[8:10], lam0, p[10], B, Lcap // 32, ps, pages, block,
                                                   *tail)
    return lib.gda_attn_decode_sparse_fp8_block(*p[:8], table, *lists, *p[8:10], lam0, p[10], B, Lcap // 32, ps, pages,
                                                block, keep, *tail)


@pytest.mark.parametrize("kind", ["whole", "paged", "sparse"])
def test_decode_refuses(lib, kind):
    for i in range(11):
        assert decode(lib, kind=kind, p=ptrs(11, **{f"p{i}": None})) == INVALID
        assert decode(lib, kind=kind, p=ptrs(11, **{f"p{i}": A + 2})) == MISALIGNED
    for bad in (dict(B=0), dict(Lcap=0), dict(hs=6, hn=4), dict(eps=-1.0), dict(eps=float("nan")), dict(lam0=float("inf")),
                dict(block=0), dict(Lcap=80, ps=80), dict(d=0)):
        assert decode(lib, kind=kind, **bad) == INVALID
    for bad in (dict(d=96), dict(dv=96), dict(hs=128, hn=1), dict(hs=2 ** 31 - 1, hn=1), dict(B=65536), dict(block=8),
                dict(block=256, ps=256, Lcap=256)):
        assert decode(lib, kind=kind, **bad) == UNSUPPORTED
    assert decode(lib, kind=kind, ws=None) == WORKSPACE and decode(lib, kind=kind, ws=A + 8) == WORKSPACE
    need = lib.gda_attn_decode_fp8_block_workspace_size(4, 6, 2, 64, 128)
    assert need > 0 and decode(lib, kind=kind, ws_bytes=need - 1) == WORKSPACE
    if not torch.cuda.is_available():
        assert decode(lib, kind=kind) == CUDA


def test_decode_refuses_tables_lists_and_positions_past_32_bits(lib):
    assert decode(lib, kind="paged", table=None) == INVALID
    for kind in ("paged", "sparse"):
        assert decode(lib, kind=kind, table=A + 2) == MISALIGNED
        assert decode(lib, kind=kind, ps=0) == INVALID and decode(lib, kind=kind, pages=0) == INVALID
        assert decode(lib, kind=kind, ps=1 << 30, Lcap=64) == INVALID
        assert decode(lib, kind=kind, pages=2 ** 31 - 1) == UNSUPPORTED
    assert decode(lib, kind="sparse", table=None) == INVALID            # two pages a sequence need one
    if not torch.cuda.is_available():
        assert decode(lib, kind="sparse", table=None, Lcap=32, pages=4) == CUDA
    for lists in ((None, A), (A, None)):
        assert decode(lib, kind="sparse", lists=lists) == INVALID
    for lists in ((A + 2, A), (A, A + 2)):
        assert decode(lib, kind="sparse", lists=lists) == MISALIGNED
    assert decode(lib, kind="sparse", keep=0) == INVALID
    assert decode(lib, kind="sparse", keep=1 << 26) == UNSUPPORTED      # keep * block of 2^31
    assert decode(lib, kind="sparse", keep=(1 << 26) - 1, B=32) == UNSUPPORTED
    assert decode(lib, Lcap=(1 << 30) + 32, B=32, block=32) == UNSUPPORTED


def test_decode_workspace_sizes(lib):
    size = lib.gda_attn_decode_fp8_block_workspace_size
    for d, dv in [(1, 1), (16, 16), (96, 128), (64, 96), (64, 512), (2 ** 31 - 1, 64), (64, 2 ** 31 - 1)]:
        assert size(1, 1, 1, d, dv) == 0
    for d in (64, 128):
        for dv in (64, 128, 256):
            assert size(1, 1, 1, d, dv) > 0 and size(65535, 127, 1, d, dv) > 0
            assert size(65536, 1, 1, d, dv) == 0 and size(1, 127, 2, d, dv) == 0 and size(1, 6, 4, d, dv) == 0


def test_sizes_past_32_bits_are_refused_by_the_binding(lib):
    import grouped_differential_attention_gb300 as gda
    for big in (1 << 31, (1 << 32) + 4, -(1 << 32) + 4):
        with pytest.raises(ValueError):
            gda.gda_attn_decode_fp8_block_workspace_size(big, 6, 2, 64, 128)
        with pytest.raises(ValueError):
            gda.gda_block_select_workspace_size(1, big, 6, 2)
        with pytest.raises(ValueError):
            gda.gda_cache_append_fp8_block_workspace_size(2000, big, 16)


def test_binding_refuses_host_tensors():
    import grouped_differential_attention_gb300 as gda
    bf = torch.bfloat16
    x, v = torch.zeros(2, 2, 64, dtype=bf), torch.zeros(2, 2, 128, dtype=bf)
    pools = [torch.zeros(1, 32, 2, n, dtype=torch.uint8) for n in (64, 64, 128)]
    scales = [torch.ones(1, 2, 2) for _ in range(3)]
    bounds = [torch.zeros(1, 2, 2, 2, 64, dtype=torch.int8)] * 2
    i = lambda *a: torch.tensor(a, dtype=torch.int32)
    lam, table = torch.ones(2), i(0).view(1, 1)
    for call in (lambda: gda.gda_cache_append_fp8_block(x, x, v, i(0, 1), *pools, *scales),
                 lambda: gda.gda_cache_read_fp8_block(i(0, 1), *pools, *scales),
                 lambda: gda.gda_block_select(x[:1], x[:1], *bounds, *scales[:2], i(3), 16, 1, first=0),
                 lambda: gda.gda_attn_decode_fp8_block(x[:1], x[:1], *pools, *scales, i(3), lam, 0.8),
                 lambda: gda.gda_attn_decode_paged_fp8_block(x[:1], x[:1], *pools, *scales, table, i(3), lam, 0.8),
                 lambda: gda.gda_attn_decode_sparse_fp8_block(x[:1], x[:1], *pools, *scales, i(0, 0).view(1, 2, 1), i(1),
                                                              i(3), lam, 0.8)):
        with pytest.raises((TypeError, ValueError)):
            call()


def test_reference_of_the_format():
    """The reference's own rounding against torch's conversions, and a growing scale by hand."""
    from oracle import ref_serving as R
    x = np.concatenate([np.linspace(-448, 448, 4001), 2.0 ** np.linspace(-12, 8, 999)]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.round_e4m3(x), want)
    codes, scale = np.zeros((16, 1, 64), np.uint8), np.full((1, 1), 7, np.float32)
    bounds = np.zeros((1, 1, 2, 64), np.int8)
    rows = torch.zeros(2, 1, 64).bfloat16()
    rows[0, 0, 0], rows[1, 0, 0], rows[1, 0, 1] = 448.0, 449.0, -9.0   # bf16 449 is 448, so the scale stays 1
    R.append_fp8_block(rows, [0, 5], codes, scale, bounds)
    assert scale[0, 0] == 1.0 and R.e4m3_value(codes[[0, 5], 0, 0]).tolist() == [448.0, 448.0]
    assert bounds[0, 0, :, 0].tolist() == [112, 112] and bounds[0, 0, :, 1].tolist() == [0, -3]
    R.append_fp8_block(2 * rows[:1] + 8, [6], codes, scale, bounds)
    assert scale[0, 0] == 4.0 and R.e4m3_value(codes[[0, 6], 0, 0]).tolist() == [112.0, 224.0]
    assert bounds[0, 0, :, 0].tolist() == [56, 28] and bounds[0, 0, :, 1].tolist() == [1, -1]
