"""Host-side checks of the operators around the attention: bad arguments get their documented status before any
device work, and the binding refuses host tensors."""
import ctypes

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


def P(x):
    return ctypes.c_void_p(x) if x is not None else None


def ptrs(n, **change):
    p = [A + 4096 * i for i in range(n)]
    for k, v in change.items():
        p[int(k[1:])] = v
    return [P(x) for x in p]


def rope(lib, entry="gda_qk_norm_rope", p=None, T=5, hs=6, hn=2, d=64, rot=64, s=None, eps=1e-5, flags=0):
    s = s or [hs * d, hs * d, hn * d, hn * d]
    return getattr(lib, entry)(*(p or ptrs(11)), T, hs, hn, d, rot, *s, eps, flags, None)


def rope_bwd(lib, entry="gda_qk_norm_rope_bwd", p=None, T=5, hs=6, hn=2, d=64, rot=64, s=None, eps=1e-5, flags=0,
             ws=A, ws_bytes=None, strides=True):
    s = s or [hs * d, hs * d, hn * d, hn * d] * 2
    need = lib.gda_qk_norm_rope_bwd_workspace_size(T, hs, hn, d)
    return getattr(lib, entry)(*(p or ptrs(16)), T, hs, hn, d, rot, (ctypes.c_longlong * 8)(*s) if strides else None,
                               eps, flags, P(ws), need if ws_bytes is None else ws_bytes, None)


@pytest.mark.parametrize("call,n,f32", [(rope, 11, "gda_qk_norm_rope_f32"), (rope_bwd, 16, "gda_qk_norm_rope_bwd_f32")])
def test_norm_rope_refuses(lib, call, n, f32):
    for i in range(n):
        assert call(lib, p=ptrs(n, **{f"p{i}": None})) == INVALID
    for i in range(5):
        assert call(lib, p=ptrs(n, **{f"p{i}": A + 8})) == MISALIGNED
    assert call(lib, p=ptrs(n, p5=A + 2)) == MISALIGNED and call(lib, p=ptrs(n, p6=A + 2)) == MISALIGNED
    assert call(lib, T=0) == INVALID and call(lib, hs=6, hn=4) == INVALID and call(lib, rot=0) == INVALID
    assert call(lib, eps=-1.0) == INVALID and call(lib, eps=float("nan")) == INVALID and call(lib, flags=1) == INVALID
    assert call(lib, d=96) == UNSUPPORTED and call(lib, rot=80) == UNSUPPORTED and call(lib, rot=24) == UNSUPPORTED
    more = 1 if call is rope else 2
    assert call(lib, s=[383, 384, 128, 128] * more) == INVALID             # less than a row
    assert call(lib, s=[388, 384, 128, 128] * more) == MISALIGNED          # bf16: 8 bytes off
    assert call(lib, entry=f32, s=[386, 384, 128, 128] * more) == MISALIGNED
    if not torch.cuda.is_available():
        assert call(lib) == CUDA and call(lib, entry=f32, s=[388, 384, 128, 132] * more, flags=4) == CUDA


def test_norm_rope_bwd_workspace(lib):
    assert lib.gda_qk_norm_rope_bwd_workspace_size(0, 6, 2, 64) == 0
    assert rope_bwd(lib, ws=None) == WORKSPACE and rope_bwd(lib, ws=A + 8) == WORKSPACE
    need = lib.gda_qk_norm_rope_bwd_workspace_size(5, 6, 2, 64)
    assert rope_bwd(lib, ws_bytes=need - 1) == WORKSPACE
    assert rope_bwd(lib, strides=False) == INVALID


def tables(lib, p=None, B=4, mp=8, ps=16, pages=40, cap=8, rows=64):
    return lib.gda_block_tables(*(p or ptrs(10)), B, mp, ps, pages, cap, rows, None)


def test_block_tables_refuses(lib):
    for i in range(10):
        assert tables(lib, p=ptrs(10, **{f"p{i}": None})) == INVALID
        assert tables(lib, p=ptrs(10, **{f"p{i}": A + 2})) == MISALIGNED
    for bad in (dict(B=0), dict(mp=0), dict(ps=0), dict(pages=0), dict(cap=0), dict(rows=0),
                dict(mp=1 << 20, ps=1 << 11), dict(pages=1 << 20, ps=1 << 11)):
        assert tables(lib, **bad) == INVALID
    assert tables(lib, B=8193) == UNSUPPORTED


def append(lib, p=None, T=4, pages=5, ps=16, hs=6, hn=2, d=64, dv=128, s=None):
    return lib.gda_cache_append_fp4(*(p or ptrs(13)), T, pages, ps, hs, hn, d, dv, *(s or [hs * d, hn * d, hs * dv]), None)


def read(lib, p=None, T=4, pages=5, ps=16, hs=6, hn=2, d=64, dv=128):
    return lib.gda_cache_read_fp4(*(p or ptrs(13)), T, pages, ps, hs, hn, d, dv, None)


@pytest.mark.parametrize("call", [append, read])
def test_cache_rows_refuse(lib, call):
    for i in range(13):
        assert call(lib, p=ptrs(13, **{f"p{i}": None})) == INVALID
        assert call(lib, p=ptrs(13, **{f"p{i}": A + 2})) == MISALIGNED
    for bad in (dict(T=0), dict(pages=0), dict(ps=0), dict(hs=6, hn=4), dict(pages=1 << 20, ps=1 << 11)):
        assert call(lib, **bad) == INVALID
    for bad in (dict(d=96), dict(dv=96), dict(hs=128, hn=1)):
        assert call(lib, **bad) == UNSUPPORTED
    assert append(lib, s=[383, 128, 768]) == INVALID and append(lib, s=[384, 132, 768]) == MISALIGNED


def decode(lib, p=None, B=4, Lcap=64, hs=6, hn=2, d=64, dv=128, lam0=0.8, eps=1e-5, ws=A, ws_bytes=None):
    p = p or ptrs(14)
    need = lib.gda_attn_decode_fp4_workspace_size(B, hs, hn, d, dv)
    return lib.gda_attn_decode_fp4(*p[:13], lam0, p[13], B, Lcap, hs, hn, d, dv, eps, P(ws),
                                   need if ws_bytes is None else ws_bytes, None)


def paged(lib, p=None, B=4, Lcap=64, hs=6, hn=2, d=64, dv=128, lam0=0.8, eps=1e-5, ws=A, ws_bytes=None, ps=16, pages=9,
          table=A):
    p = p or ptrs(14)
    need = lib.gda_attn_decode_fp4_workspace_size(B, hs, hn, d, dv)
    return lib.gda_attn_decode_paged_fp4(*p[:11], P(table), *p[11:13], lam0, p[13], B, Lcap // 16, ps, pages, hs, hn, d,
                                         dv, eps, P(ws), need if ws_bytes is None else ws_bytes, None)


@pytest.mark.parametrize("call", [decode, paged])
def test_decode_refuses(lib, call):
    for i in range(14):
        assert call(lib, p=ptrs(14, **{f"p{i}": None})) == INVALID
        assert call(lib, p=ptrs(14, **{f"p{i}": A + 2})) == MISALIGNED
    for bad in (dict(B=0), dict(Lcap=0), dict(hs=6, hn=4), dict(eps=-1.0), dict(lam0=float("inf"))):
        assert call(lib, **bad) == INVALID
    for bad in (dict(d=96), dict(dv=96), dict(hs=128, hn=1), dict(B=65536)):
        assert call(lib, **bad) == UNSUPPORTED
    for bad in (dict(Lcap=0x7ffffff1), dict(Lcap=0x7fffffff), dict(Lcap=(1 << 30) + 16, B=32)):   # positions of 32 bits
        args = dict(bad, ps=bad["Lcap"], Lcap=16) if call is paged else bad                       # one page each
        assert call(lib, **args) == UNSUPPORTED
    assert call(lib, ws=None) == WORKSPACE and call(lib, ws=A + 8) == WORKSPACE
    need = lib.gda_attn_decode_fp4_workspace_size(4, 6, 2, 64, 128)
    assert need > 0 and call(lib, ws_bytes=need - 1) == WORKSPACE
    if not torch.cuda.is_available():
        assert call(lib) == CUDA


def test_paged_decode_refuses_tables(lib):
    assert paged(lib, table=None) == INVALID and paged(lib, table=A + 2) == MISALIGNED
    assert paged(lib, ps=0) == INVALID and paged(lib, pages=0) == INVALID and paged(lib, ps=1 << 30, Lcap=64) == INVALID


def test_ranges_of_the_longest_batch_fit_32_bits(lib):
    """The decode counts a range's positions in 32 bits: the fewest ranges of any supported shape against the most
    positions.  The workspace has (ranges + B) slots of h_s (2 dv + 4) floats, so its size gives the ranges."""
    fewest = 1 << 30
    for dv in (64, 128, 256):
        for hn in range(1, 65):
            for hs in range(hn, 129 - hn, hn):
                slots = lib.gda_attn_decode_fp4_workspace_size(1, hs, hn, 64, dv) / (4 * hs * (2 * dv + 4))
                fewest = min(fewest, int(slots) - 1)
    assert fewest >= 19 - 1 and (1 << 35) / 18 + 16 < 1 << 31


def test_sizes_past_32_bits_are_refused_by_the_binding(lib):
    import grouped_differential_attention_gb300 as gda
    for big in (1 << 31, (1 << 32) + 4, -(1 << 32) + 4):
        with pytest.raises(ValueError):
            gda.gda_attn_decode_fp4_workspace_size(big, 6, 2, 64, 128)
        with pytest.raises(ValueError):
            gda.gda_qk_norm_rope_bwd_workspace_size(big, 6, 2, 64)
    assert gda.gda_attn_decode_fp4_workspace_size(0, 6, 2, 64, 128) == 0


def test_binding_refuses_host_tensors():
    import grouped_differential_attention_gb300 as gda
    bf = torch.bfloat16
    x = torch.zeros(2, 2, 64, dtype=bf)
    w, pos, freq = torch.ones(4, 64), torch.zeros(2, dtype=torch.int32), torch.ones(32)
    u8 = lambda n: torch.zeros(1, 16, 2, n, dtype=torch.uint8)
    cache = (u8(32), u8(32), u8(64), u8(4), u8(4), u8(8), torch.ones(2), torch.ones(2), torch.ones(2))
    i = lambda *v: torch.tensor(v, dtype=torch.int32)
    calls = [lambda: gda.gda_qk_norm_rope(x, x, x, x, w, pos, freq),
             lambda: gda.gda_qk_norm_rope_bwd(x, x, x, x, w, pos, freq, *[x.float()] * 4),
             lambda: gda.gda_block_tables(i(1), i(1), i(0).view(1, 1), i(1), i(1), 16, 2, 4),
             lambda: gda.gda_cache_append_fp4(x, x, torch.zeros(2, 2, 128, dtype=bf), i(0, 1), *cache),
             lambda: gda.gda_cache_read_fp4(i(0, 1), *cache),
             lambda: gda.gda_attn_decode_fp4(x[:1], x[:1], *cache, i(3), torch.ones(2), 0.8),
             lambda: gda.gda_attn_decode_paged_fp4(x[:1], x[:1], *cache, i(0).view(1, 1), i(3), torch.ones(2), 0.8)]
    for call in calls:
        with pytest.raises((TypeError, ValueError)):
            call()
