"""Grouped differential attention on NVIDIA GB300 (sm_103a).

Python binding of ``libgda.so`` (C ABI in ``include/gda.h``).  The functions
below carry the C names and only marshal arguments: they check dtypes,
shapes, devices and contiguity on the PyTorch side, then pass raw device
pointers and the current CUDA stream to the library, whose kernels do every
step of the computation.  There is no CPU or PyTorch fallback: if the
library is missing, every call raises.

Operation (see ``include/gda.h``): for signal head h with noise head
g = h // (h_s // h_n),

    y_h = (1 - lambda_init) * RMSNorm( (softmax(Q1_h K1_h^T / sqrt d)
                                        - lambda_h softmax(Q2_g K2_g^T / sqrt d)) V_h )

Layouts: q_sig, k_sig [B, L, h_s, d]; q_noise, k_noise [B, L, h_n, d];
v and the output [B, L, h_s, dv]; lambda [h_s] float32.

Around the attention: ``gda_qk_norm_rope`` (per-head norm and rotation of the
four projections, with gradients), ``gda_block_tables`` (block table, slots and
positions of a serving step), and a 4-bit cache (``gda_cache_append_fp4``,
``gda_cache_read_fp4``, ``gda_attn_decode_fp4``, ``gda_attn_decode_paged_fp4``).
An 8-bit cache with a scale for each block of tokens and head
(``gda_cache_append_fp8_block``, ``gda_cache_read_fp8_block``), decodes over all
of it (``gda_attn_decode_fp8_block``, ``gda_attn_decode_paged_fp8_block``), and
over the blocks that an estimate of their logits keeps (``gda_block_select``,
``gda_attn_decode_sparse_fp8_block``).
"""
from __future__ import annotations

import ctypes
import functools
import operator
import os
import threading

import torch

__all__ = [
    "GDAError", "gda_attn_fwd", "gda_attn_fwd_f32", "gda_attn_decode",
    "gda_attn_decode_workspace_size", "gda_status_string", "gda_device_error",
    "library_path", "GDA_FLAG_NO_NORM", "GDA_FLAG_SINGLE_PASS",
    "gda_attn_decode_noalloc",
    "gda_attn_bwd", "gda_attn_bwd_workspace_size", "gda_attn_fwd_2pass",
    "gda_attn_fwd_2pass_workspace_size", "gda_attn_bwd_bf16", "gda_attn_bwd_bf16_workspace_size",
    "gda_attn_decode_paged_fp8", "gda_attn_fwd_chunk", "gda_attn_fwd_chunk_2pass",
    "gda_qk_norm_rope", "gda_qk_norm_rope_bwd", "gda_qk_norm_rope_bwd_workspace_size", "gda_block_tables",
    "gda_cache_append_fp4", "gda_cache_read_fp4", "gda_attn_decode_fp4", "gda_attn_decode_paged_fp4",
    "gda_attn_decode_fp4_workspace_size", "GDA_FLAG_ROPE_INTERLEAVED",
    "gda_cache_append_fp8_block", "gda_cache_append_fp8_block_workspace_size", "gda_cache_read_fp8_block",
    "gda_block_select", "gda_block_select_workspace_size", "gda_attn_decode_fp8_block",
    "gda_attn_decode_paged_fp8_block", "gda_attn_decode_sparse_fp8_block", "gda_attn_decode_fp8_block_workspace_size",
]

GDA_OK = 0
GDA_ERR_INVALID_ARG = -1
GDA_ERR_UNSUPPORTED = -2
GDA_ERR_MISALIGNED = -3
GDA_ERR_WORKSPACE = -4
GDA_ERR_CUDA = -5
GDA_ERR_DEVICE_TIMEOUT = -6
GDA_FLAG_NO_NORM = 0x1
GDA_FLAG_SINGLE_PASS = 0x2
GDA_FLAG_ROPE_INTERLEAVED = 0x4
GDA_DEVERR_PREFILL_TIMEOUT = 0x1
GDA_DEVERR_BAD_LENGTH = 0x2
GDA_DEVERR_DECODE_TIMEOUT = 0x4
GDA_DEVERR_BAD_PAGE = 0x8
GDA_DEVERR_NO_PAGES = 0x10

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "_build", "libgda.so")
_lock = threading.Lock()
_lib = None


class GDAError(RuntimeError):
    def __init__(self, status: int, what: str):
        extra = ""
        if status == GDA_ERR_CUDA:
            extra = f", cudaError {_load().gda_last_cuda_error()}"
        super().__init__(f"{what}: {gda_status_string(status)} (status {status}{extra})")
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def _load():
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise RuntimeError(
                    f"{_LIB_PATH} is missing: build it with "
                    "`python -m grouped_differential_attention_gb300.build`")
            lib = ctypes.CDLL(_LIB_PATH)
            P, I, F, U, Z = (ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_uint,
                             ctypes.c_size_t)
            fwd = [P, P, P, P, P, P, F, P, I, I, I, I, I, I, I, F]
            lib.gda_attn_fwd.argtypes = fwd + [P]
            lib.gda_attn_fwd_ex.argtypes = fwd + [U, P]
            lib.gda_attn_fwd_f32.argtypes = fwd + [P]
            lib.gda_attn_fwd_f32_ex.argtypes = fwd + [U, P]
            lib.gda_attn_decode_workspace_size.argtypes = [I, I, I, I, I]
            lib.gda_attn_decode_workspace_size.restype = Z
            lib.gda_attn_decode.argtypes = [P, P, P, P, P, P, P, F, P, I, I, I, I, I, I, F, P, Z, P]
            lib.gda_status_string.argtypes = [I]
            lib.gda_status_string.restype = ctypes.c_char_p
            lib.gda_attn_decode_noalloc.argtypes = [P, P, P, P, P, P, P, F, P, I, I, I, I, I, I, F, P]
            lib.gda_attn_decode_noalloc.restype = I
            lib.gda_attn_decode_fp8.argtypes = [P, P, P, P, P, P, P, P, P, P, F, P, I, I, I, I, I, I, F,
                                                P, Z, P]
            lib.gda_attn_decode_fp8.restype = I
            lib.gda_attn_decode_paged.argtypes = [P, P, P, P, P, P, P, P, F, P, I, I, I, I, I, I, I, I, F,
                                                  P, Z, P]
            lib.gda_attn_decode_paged.restype = I
            lib.gda_attn_fwd_chunk.argtypes = [P, P, P, P, P, P, F, P, I, I, I, I, I, I, I, I, F, U, P]
            lib.gda_attn_fwd_chunk.restype = I
            lib.gda_attn_fwd_chunk_2pass.argtypes = [P, P, P, P, P, P, F, P, I, I, I, I, I, I, I, I, F, U,
                                                     P, Z, P]
            lib.gda_attn_fwd_chunk_2pass.restype = I
            lib.gda_lambda_reparam.argtypes = [P, P, P, P, F, P, I, I, P]
            lib.gda_lambda_reparam.restype = I
            lib.gda_attn_decode_paged_fp8.argtypes = [P, P, P, P, P, P, P, P, P, P, P, F, P, I, I, I, I, I, I,
                                                      I, I, F, P, Z, P]
            lib.gda_attn_decode_paged_fp8.restype = I
            lib.gda_attn_fwd_2pass.argtypes = [P, P, P, P, P, P, F, P, I, I, I, I, I, I, I, F, U, P, Z, P]
            lib.gda_attn_fwd_2pass.restype = I
            lib.gda_attn_fwd_2pass_workspace_size.argtypes = [I, I, I, I]
            lib.gda_attn_fwd_2pass_workspace_size.restype = Z
            lib.gda_attn_bwd_bf16.argtypes = [P, P, P, P, P, P, F, P, P, P, P, P, P, P, I, I, I, I, I, I, I,
                                              F, U, P, Z, P]
            lib.gda_attn_bwd_bf16.restype = I
            lib.gda_attn_bwd_bf16_workspace_size.argtypes = [I, I, I, I, I]
            lib.gda_attn_bwd_bf16_workspace_size.restype = Z
            lib.gda_attn_bwd.argtypes = [P, P, P, P, P, P, F, P, P, P, P, P, P, P, I, I, I, I, I, I, I, F,
                                         U, P, Z, P]
            lib.gda_attn_bwd.restype = I
            lib.gda_attn_bwd_workspace_size.argtypes = [I, I, I, I, I]
            lib.gda_attn_bwd_workspace_size.restype = Z
            X = ctypes.c_longlong
            for name in ("gda_qk_norm_rope", "gda_qk_norm_rope_f32"):
                getattr(lib, name).argtypes = [P] * 11 + [I] * 5 + [X] * 4 + [F, U, P]
                getattr(lib, name).restype = I
            for name in ("gda_qk_norm_rope_bwd", "gda_qk_norm_rope_bwd_f32"):
                getattr(lib, name).argtypes = [P] * 16 + [I] * 5 + [P, F, U, P, Z, P]
                getattr(lib, name).restype = I
            lib.gda_qk_norm_rope_bwd_workspace_size.argtypes = [I] * 4
            lib.gda_qk_norm_rope_bwd_workspace_size.restype = Z
            lib.gda_block_tables.argtypes = [P] * 10 + [I] * 6 + [P]
            lib.gda_block_tables.restype = I
            lib.gda_cache_append_fp4.argtypes = [P] * 13 + [I] * 7 + [X] * 3 + [P]
            lib.gda_cache_append_fp4.restype = I
            lib.gda_cache_read_fp4.argtypes = [P] * 13 + [I] * 7 + [P]
            lib.gda_cache_read_fp4.restype = I
            lib.gda_attn_decode_fp4.argtypes = [P] * 13 + [F, P] + [I] * 6 + [F, P, Z, P]
            lib.gda_attn_decode_fp4.restype = I
            lib.gda_attn_decode_paged_fp4.argtypes = [P] * 14 + [F, P] + [I] * 8 + [F, P, Z, P]
            lib.gda_attn_decode_paged_fp4.restype = I
            lib.gda_attn_decode_fp4_workspace_size.argtypes = [I] * 5
            lib.gda_attn_decode_fp4_workspace_size.restype = Z
            lib.gda_cache_append_fp8_block.argtypes = [P] * 12 + [I] * 8 + [X] * 3 + [P, Z, P]
            lib.gda_cache_append_fp8_block.restype = I
            lib.gda_cache_append_fp8_block_workspace_size.argtypes = [I] * 3
            lib.gda_cache_append_fp8_block_workspace_size.restype = Z
            lib.gda_cache_read_fp8_block.argtypes = [P] * 10 + [I] * 8 + [P]
            lib.gda_cache_read_fp8_block.restype = I
            lib.gda_block_select.argtypes = [P] * 10 + [I] * 11 + [P, Z, P]
            lib.gda_block_select.restype = I
            lib.gda_block_select_workspace_size.argtypes = [I] * 4
            lib.gda_block_select_workspace_size.restype = Z
            lib.gda_attn_decode_fp8_block.argtypes = [P] * 10 + [F, P] + [I] * 7 + [F, P, Z, P]
            lib.gda_attn_decode_fp8_block.restype = I
            lib.gda_attn_decode_paged_fp8_block.argtypes = [P] * 11 + [F, P] + [I] * 9 + [F, P, Z, P]
            lib.gda_attn_decode_paged_fp8_block.restype = I
            lib.gda_attn_decode_sparse_fp8_block.argtypes = [P] * 13 + [F, P] + [I] * 10 + [F, P, Z, P]
            lib.gda_attn_decode_sparse_fp8_block.restype = I
            lib.gda_attn_decode_fp8_block_workspace_size.argtypes = [I] * 5
            lib.gda_attn_decode_fp8_block_workspace_size.restype = Z
            lib.gda_device_error.argtypes = [I]
            lib.gda_last_cuda_error.argtypes = []
            lib.gda_last_cuda_error.restype = I
            for name in ("gda_attn_fwd", "gda_attn_fwd_ex", "gda_attn_fwd_f32",
                         "gda_attn_fwd_f32_ex", "gda_attn_decode", "gda_device_error"):
                getattr(lib, name).restype = I
            _lib = lib
    return _lib


def gda_status_string(status: int) -> str:
    return _load().gda_status_string(int(status)).decode()


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check(rc: int, what: str):
    if rc != GDA_OK:
        raise GDAError(rc, what)


def _expect(t, name, dtype, shape, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _prefill(entry, dtype, q_sig, k_sig, q_noise, k_noise, v, lam, lambda_init, causal, eps,
             out, flags):
    dev = q_sig.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    if q_sig.dim() != 4 or q_noise.dim() != 4 or v.dim() != 4:
        raise ValueError("q_sig, q_noise and v must be 4-D [B, L, heads, dim]")
    B, L, hs, d = q_sig.shape
    hn = q_noise.shape[2]
    dv = v.shape[3]
    _expect(q_sig, "q_sig", dtype, (B, L, hs, d), dev)
    _expect(k_sig, "k_sig", dtype, (B, L, hs, d), dev)
    _expect(q_noise, "q_noise", dtype, (B, L, hn, d), dev)
    _expect(k_noise, "k_noise", dtype, (B, L, hn, d), dev)
    _expect(v, "v", dtype, (B, L, hs, dv), dev)
    _expect(lam, "lam", torch.float32, (hs,), dev)
    if out is None:
        out = torch.empty((B, L, hs, dv), dtype=dtype, device=dev)
    _expect(out, "out", dtype, (B, L, hs, dv), dev)
    with torch.cuda.device(dev):
        rc = entry(_ptr(q_sig), _ptr(k_sig), _ptr(q_noise), _ptr(k_noise), _ptr(v), _ptr(lam),
                   float(lambda_init), _ptr(out), B, L, hs, hn, d, dv, int(bool(causal)),
                   float(eps), int(flags), _stream(dev))
    _check(rc, "gda prefill")
    return out


def gda_attn_fwd(q_sig, k_sig, q_noise, k_noise, v, lam, lambda_init: float, *,
                 causal: bool = True, eps: float = 1e-5, out=None, flags: int = 0):
    """bf16 prefill on the tensor cores (tcgen05/TMEM, TMA); returns ``out``."""
    return _prefill(_load().gda_attn_fwd_ex, torch.bfloat16, q_sig, k_sig, q_noise, k_noise, v,
                    lam, lambda_init, causal, eps, out, flags)


def gda_attn_fwd_chunk(q_sig, k_sig, q_noise, k_noise, v, lam, lambda_init: float, *,
                       causal: bool = True, eps: float = 1e-5, out=None, flags: int = 0, workspace=None,
                       two_pass: bool = False):
    """Chunked bf16 prefill: L query rows at key positions Lk - L .. Lk - 1.

    q_sig [B, L, h_s, d], q_noise [B, L, h_n, d]; k_sig [B, Lk, h_s, d],
    k_noise [B, Lk, h_n, d], v [B, Lk, h_s, dv]; returns out [B, L, h_s, dv].
    ``two_pass`` calls gda_attn_fwd_chunk_2pass, whose statistics workspace
    (uint8 CUDA tensor of gda_attn_fwd_2pass_workspace_size(B, L, h_s, h_n)
    bytes) is ``workspace`` or allocated here.
    """
    dev = q_sig.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    B, L, hs, d = q_sig.shape
    hn = q_noise.shape[2]
    Lk = k_sig.shape[1]
    dv = v.shape[3]
    bf = torch.bfloat16
    _expect(q_sig, "q_sig", bf, (B, L, hs, d), dev)
    _expect(k_sig, "k_sig", bf, (B, Lk, hs, d), dev)
    _expect(q_noise, "q_noise", bf, (B, L, hn, d), dev)
    _expect(k_noise, "k_noise", bf, (B, Lk, hn, d), dev)
    _expect(v, "v", bf, (B, Lk, hs, dv), dev)
    _expect(lam, "lam", torch.float32, (hs,), dev)
    if out is None:
        out = torch.empty((B, L, hs, dv), dtype=bf, device=dev)
    _expect(out, "out", bf, (B, L, hs, dv), dev)
    args = (_ptr(q_sig), _ptr(k_sig), _ptr(q_noise), _ptr(k_noise), _ptr(v), _ptr(lam), float(lambda_init),
            _ptr(out), B, L, Lk, hs, hn, d, dv, int(bool(causal)), float(eps), int(flags))
    with torch.cuda.device(dev):
        if two_pass:
            need = gda_attn_fwd_2pass_workspace_size(B, L, hs, hn)
            if workspace is None:
                workspace = torch.empty((max(need, 16),), dtype=torch.uint8, device=dev)
            _expect(workspace, "workspace", torch.uint8, (workspace.numel(),), dev)
            rc = _load().gda_attn_fwd_chunk_2pass(*args, _ptr(workspace), workspace.numel(), _stream(dev))
        else:
            rc = _load().gda_attn_fwd_chunk(*args, _stream(dev))
    _check(rc, "gda chunked prefill")
    return out


def gda_attn_fwd_f32(q_sig, k_sig, q_noise, k_noise, v, lam, lambda_init: float, *,
                     causal: bool = True, eps: float = 1e-5, out=None, flags: int = 0):
    """float32 prefill on the CUDA cores; returns ``out``."""
    return _prefill(_load().gda_attn_fwd_f32_ex, torch.float32, q_sig, k_sig, q_noise, k_noise,
                    v, lam, lambda_init, causal, eps, out, flags)


def gda_attn_decode_fp8(q_sig, q_noise, k_sig_cache, k_noise_cache, v_cache, k_sig_scale,
                        k_noise_scale, v_scale, cache_lens, lam, lambda_init: float, *,
                        eps: float = 1e-5, out=None, workspace=None):
    """bf16 decode over fp8 (e4m3) caches: cached value = code * scale of its head.

    The caches are ``torch.float8_e4m3fn`` (or ``uint8`` holding the codes)
    CUDA tensors [B, Lcap, heads, dim]; scales are float32 [h_s], [h_n], [h_s].
    """
    dev = q_sig.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    B, hs, d = q_sig.shape
    hn = q_noise.shape[1]
    Lcap = k_sig_cache.shape[1]
    dv = v_cache.shape[3]
    bf = torch.bfloat16
    codes = []
    for t, name, shape in ((k_sig_cache, "k_sig_cache", (B, Lcap, hs, d)),
                           (k_noise_cache, "k_noise_cache", (B, Lcap, hn, d)),
                           (v_cache, "v_cache", (B, Lcap, hs, dv))):
        if t.dtype == torch.float8_e4m3fn:
            t = t.view(torch.uint8)
        _expect(t, name, torch.uint8, shape, dev)
        codes.append(t)
    _expect(q_sig, "q_sig", bf, (B, hs, d), dev)
    _expect(q_noise, "q_noise", bf, (B, hn, d), dev)
    _expect(k_sig_scale, "k_sig_scale", torch.float32, (hs,), dev)
    _expect(k_noise_scale, "k_noise_scale", torch.float32, (hn,), dev)
    _expect(v_scale, "v_scale", torch.float32, (hs,), dev)
    _expect(cache_lens, "cache_lens", torch.int32, (B,), dev)
    _expect(lam, "lam", torch.float32, (hs,), dev)
    if out is None:
        out = torch.empty((B, hs, dv), dtype=bf, device=dev)
    _expect(out, "out", bf, (B, hs, dv), dev)
    need = gda_attn_decode_workspace_size(B, Lcap, hs, hn, dv)
    if workspace is None:
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        rc = _load().gda_attn_decode_fp8(
            _ptr(q_sig), _ptr(q_noise), _ptr(codes[0]), _ptr(codes[1]), _ptr(codes[2]),
            _ptr(k_sig_scale), _ptr(k_noise_scale), _ptr(v_scale), _ptr(cache_lens), _ptr(lam),
            float(lambda_init), _ptr(out), B, Lcap, hs, hn, d, dv, float(eps), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(dev))
    _check(rc, "gda decode (fp8 cache)")
    return out


def gda_attn_decode_paged(q_sig, q_noise, k_sig_pool, k_noise_pool, v_pool, block_table, cache_lens,
                          lam, lambda_init: float, *, eps: float = 1e-5, out=None, workspace=None):
    """bf16 decode over paged caches.

    Pools [num_pages, page_size, heads, dim] (bf16); block_table [B,
    max_pages] int32: position j of sequence b is row j % page_size of page
    block_table[b, j // page_size].
    """
    dev = q_sig.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    B, hs, d = q_sig.shape
    hn = q_noise.shape[1]
    num_pages, page_size = k_sig_pool.shape[0], k_sig_pool.shape[1]
    dv = v_pool.shape[3]
    max_pages = block_table.shape[1]
    bf = torch.bfloat16
    _expect(q_sig, "q_sig", bf, (B, hs, d), dev)
    _expect(q_noise, "q_noise", bf, (B, hn, d), dev)
    _expect(k_sig_pool, "k_sig_pool", bf, (num_pages, page_size, hs, d), dev)
    _expect(k_noise_pool, "k_noise_pool", bf, (num_pages, page_size, hn, d), dev)
    _expect(v_pool, "v_pool", bf, (num_pages, page_size, hs, dv), dev)
    _expect(block_table, "block_table", torch.int32, (B, max_pages), dev)
    _expect(cache_lens, "cache_lens", torch.int32, (B,), dev)
    _expect(lam, "lam", torch.float32, (hs,), dev)
    if out is None:
        out = torch.empty((B, hs, dv), dtype=bf, device=dev)
    _expect(out, "out", bf, (B, hs, dv), dev)
    need = gda_attn_decode_workspace_size(B, max_pages * page_size, hs, hn, dv)
    if workspace is None:
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        rc = _load().gda_attn_decode_paged(
            _ptr(q_sig), _ptr(q_noise), _ptr(k_sig_pool), _ptr(k_noise_pool), _ptr(v_pool),
            _ptr(block_table), _ptr(cache_lens), _ptr(lam), float(lambda_init), _ptr(out), B,
            max_pages, page_size, num_pages, hs, hn, d, dv, float(eps), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(dev))
    _check(rc, "gda decode (paged caches)")
    return out


def gda_attn_decode_paged_fp8(q_sig, q_noise, k_sig_pool, k_noise_pool, v_pool, k_sig_scale, k_noise_scale,
                              v_scale, block_table, cache_lens, lam, lambda_init: float, *, eps: float = 1e-5,
                              out=None, workspace=None):
    """bf16 decode over paged fp8 (e4m3) caches: pools [num_pages, page_size,
    heads, dim] of float8_e4m3fn (or uint8 codes), per-head float32 scales,
    block_table [B, max_pages] int32."""
    dev = q_sig.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    B, hs, d = q_sig.shape
    hn = q_noise.shape[1]
    num_pages, page_size = k_sig_pool.shape[0], k_sig_pool.shape[1]
    dv = v_pool.shape[3]
    max_pages = block_table.shape[1]
    bf = torch.bfloat16
    pools = []
    for t, name, shape in ((k_sig_pool, "k_sig_pool", (num_pages, page_size, hs, d)),
                           (k_noise_pool, "k_noise_pool", (num_pages, page_size, hn, d)),
                           (v_pool, "v_pool", (num_pages, page_size, hs, dv))):
        if t.dtype == torch.float8_e4m3fn:
            t = t.view(torch.uint8)
        _expect(t, name, torch.uint8, shape, dev)
        pools.append(t)
    _expect(q_sig, "q_sig", bf, (B, hs, d), dev)
    _expect(q_noise, "q_noise", bf, (B, hn, d), dev)
    _expect(k_sig_scale, "k_sig_scale", torch.float32, (hs,), dev)
    _expect(k_noise_scale, "k_noise_scale", torch.float32, (hn,), dev)
    _expect(v_scale, "v_scale", torch.float32, (hs,), dev)
    _expect(block_table, "block_table", torch.int32, (B, max_pages), dev)
    _expect(cache_lens, "cache_lens", torch.int32, (B,), dev)
    _expect(lam, "lam", torch.float32, (hs,), dev)
    if out is None:
        out = torch.empty((B, hs, dv), dtype=bf, device=dev)
    _expect(out, "out", bf, (B, hs, dv), dev)
    need = gda_attn_decode_workspace_size(B, max_pages * page_size, hs, hn, dv)
    if workspace is None:
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        rc = _load().gda_attn_decode_paged_fp8(
            _ptr(q_sig), _ptr(q_noise), *[_ptr(t) for t in pools], _ptr(k_sig_scale), _ptr(k_noise_scale),
            _ptr(v_scale), _ptr(block_table), _ptr(cache_lens), _ptr(lam), float(lambda_init), _ptr(out), B,
            max_pages, page_size, num_pages, hs, hn, d, dv, float(eps), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(dev))
    _check(rc, "gda decode (paged fp8 caches)")
    return out


def gda_attn_fwd_2pass_workspace_size(B: int, L: int, h_s: int, h_n: int) -> int:
    return int(_load().gda_attn_fwd_2pass_workspace_size(B, L, h_s, h_n))


def gda_attn_fwd_2pass(q_sig, k_sig, q_noise, k_noise, v, lam, lambda_init: float, *,
                       causal: bool = True, eps: float = 1e-5, out=None, flags: int = 0, workspace=None):
    """Two-pass bf16 prefill (difference map before the value product); returns ``out``.

    ``workspace`` (uint8 CUDA tensor) receives the rows' base-2 log-sum-exp
    values as float32 [B, h_s + h_n, L].
    """
    B, L, hs, _ = q_sig.shape
    hn = q_noise.shape[2]
    need = gda_attn_fwd_2pass_workspace_size(B, L, hs, hn)
    if workspace is None:
        workspace = torch.empty((max(need, 16),), dtype=torch.uint8, device=q_sig.device)
    _expect(workspace, "workspace", torch.uint8, (workspace.numel(),), q_sig.device)
    ws = workspace

    def entry(*args):
        *head, fl, stream = args
        return _load().gda_attn_fwd_2pass(*head, fl, _ptr(ws), ws.numel(), stream)
    return _prefill(entry, torch.bfloat16, q_sig, k_sig, q_noise, k_noise, v, lam, lambda_init, causal,
                    eps, out, flags)


def _given(tensors, count, what):
    """The caller's output tensors as a tuple of exactly `count`: the C entries take a pointer for each."""
    tensors = tuple(tensors)
    if len(tensors) != count:
        raise ValueError(f"{what} holds {len(tensors)} tensors, expected {count}")
    return tensors


def gda_attn_bwd_workspace_size(B: int, L: int, h_s: int, d: int, dv: int) -> int:
    return int(_load().gda_attn_bwd_workspace_size(B, L, h_s, d, dv))


def gda_attn_bwd(q_sig, k_sig, q_noise, k_noise, v, lam, lambda_init: float, dy, *,
                 causal: bool = True, eps: float = 1e-5, flags: int = 0, workspace=None, grads=None):
    """float32 gradients of the operation; returns (dq_sig, dk_sig, dq_noise, dk_noise, dv, dlambda).

    Inputs as for ``gda_attn_fwd_f32`` plus ``dy`` [B, L, h_s, dv] (the
    gradient of the loss with respect to the output).  ``grads`` may hold the
    six output tensors to overwrite.
    """
    dev = q_sig.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    if q_sig.dim() != 4 or q_noise.dim() != 4 or v.dim() != 4:
        raise ValueError("q_sig, q_noise and v must be 4-D [B, L, heads, dim]")
    f32 = torch.float32
    B, L, hs, d = q_sig.shape
    hn = q_noise.shape[2]
    dv = v.shape[3]
    shapes = ((B, L, hs, d), (B, L, hs, d), (B, L, hn, d), (B, L, hn, d), (B, L, hs, dv), (hs,))
    for t, name, shape in zip((q_sig, k_sig, q_noise, k_noise, v, lam), ("q_sig", "k_sig", "q_noise",
                              "k_noise", "v", "lam"), shapes):
        _expect(t, name, f32, shape, dev)
    _expect(dy, "dy", f32, (B, L, hs, dv), dev)
    if grads is None:
        grads = tuple(torch.empty(s, dtype=f32, device=dev) for s in shapes)
    grads = _given(grads, 6, "grads")
    for t, name, shape in zip(grads, ("dq_sig", "dk_sig", "dq_noise", "dk_noise", "dv", "dlambda"), shapes):
        _expect(t, name, f32, shape, dev)
    need = gda_attn_bwd_workspace_size(B, L, hs, d, dv)
    if workspace is None:
        workspace = torch.empty((max(need, 16),), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        rc = _load().gda_attn_bwd(
            _ptr(q_sig), _ptr(k_sig), _ptr(q_noise), _ptr(k_noise), _ptr(v), _ptr(lam),
            float(lambda_init), _ptr(dy), *[_ptr(t) for t in grads], B, L, hs, hn, d, dv,
            int(bool(causal)), float(eps), int(flags), _ptr(workspace), workspace.numel(), _stream(dev))
    _check(rc, "gda backward")
    return tuple(grads)


def gda_attn_bwd_bf16_workspace_size(B: int, L: int, h_s: int, h_n: int, dv: int) -> int:
    return int(_load().gda_attn_bwd_bf16_workspace_size(B, L, h_s, h_n, dv))


def gda_attn_bwd_bf16(q_sig, k_sig, q_noise, k_noise, v, lam, lambda_init: float, dy, *,
                      causal: bool = True, eps: float = 1e-5, flags: int = 0, workspace=None, grads=None):
    """Tensor-core gradients from bf16 inputs; returns float32
    (dq_sig, dk_sig, dq_noise, dk_noise, dv, dlambda)."""
    dev = q_sig.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    if q_sig.dim() != 4 or q_noise.dim() != 4 or v.dim() != 4:
        raise ValueError("q_sig, q_noise and v must be 4-D [B, L, heads, dim]")
    bf, f32 = torch.bfloat16, torch.float32
    B, L, hs, d = q_sig.shape
    hn = q_noise.shape[2]
    dv = v.shape[3]
    shapes = ((B, L, hs, d), (B, L, hs, d), (B, L, hn, d), (B, L, hn, d), (B, L, hs, dv), (hs,))
    for t, name, shape in zip((q_sig, k_sig, q_noise, k_noise, v), ("q_sig", "k_sig", "q_noise", "k_noise", "v"),
                              shapes):
        _expect(t, name, bf, shape, dev)
    _expect(lam, "lam", f32, (hs,), dev)
    _expect(dy, "dy", bf, (B, L, hs, dv), dev)
    if grads is None:
        grads = tuple(torch.empty(s, dtype=f32, device=dev) for s in shapes)
    grads = _given(grads, 6, "grads")
    for t, name, shape in zip(grads, ("dq_sig", "dk_sig", "dq_noise", "dk_noise", "dv", "dlambda"), shapes):
        _expect(t, name, f32, shape, dev)
    need = gda_attn_bwd_bf16_workspace_size(B, L, hs, hn, dv)
    if workspace is None:
        workspace = torch.empty((max(need, 16),), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        rc = _load().gda_attn_bwd_bf16(
            _ptr(q_sig), _ptr(k_sig), _ptr(q_noise), _ptr(k_noise), _ptr(v), _ptr(lam),
            float(lambda_init), _ptr(dy), *[_ptr(t) for t in grads], B, L, hs, hn, d, dv,
            int(bool(causal)), float(eps), int(flags), _ptr(workspace), workspace.numel(), _stream(dev))
    _check(rc, "gda backward (bf16)")
    return tuple(grads)


def gda_lambda_reparam(lambda_q1, lambda_k1, lambda_q2, lambda_k2, lambda_init: float, *, out=None):
    """lambda[h] = exp(lq1[h].lk1[h]) - exp(lq2[h].lk2[h]) + lambda_init on the device.

    The four vectors are float32 CUDA tensors [h_s, d]; returns ``out``
    (float32 [h_s]), ready to pass as ``lam`` to the attention calls.
    """
    dev = lambda_q1.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    if lambda_q1.dim() != 2:
        raise ValueError("lambda vectors must be 2-D [h_s, d]")
    hs, d = lambda_q1.shape
    for t, name in ((lambda_q1, "lambda_q1"), (lambda_k1, "lambda_k1"), (lambda_q2, "lambda_q2"),
                    (lambda_k2, "lambda_k2")):
        _expect(t, name, torch.float32, (hs, d), dev)
    if out is None:
        out = torch.empty((hs,), dtype=torch.float32, device=dev)
    _expect(out, "out", torch.float32, (hs,), dev)
    with torch.cuda.device(dev):
        rc = _load().gda_lambda_reparam(_ptr(lambda_q1), _ptr(lambda_k1), _ptr(lambda_q2),
                                        _ptr(lambda_k2), float(lambda_init), _ptr(out), hs, d,
                                        _stream(dev))
    _check(rc, "gda lambda re-parameterisation")
    return out


def gda_attn_decode_workspace_size(B: int, Lcap: int, h_s: int, h_n: int, dv: int) -> int:
    return int(_load().gda_attn_decode_workspace_size(B, Lcap, h_s, h_n, dv))


def gda_attn_decode(q_sig, q_noise, k_sig_cache, k_noise_cache, v_cache, cache_lens, lam,
                    lambda_init: float, *, eps: float = 1e-5, out=None, workspace=None):
    """bf16 decode of one query token per sequence over its KV cache; returns ``out``.

    ``workspace`` (a CUDA uint8 tensor of at least
    ``gda_attn_decode_workspace_size(...)`` bytes) is allocated here when not
    given.
    """
    dev = q_sig.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    if q_sig.dim() != 3 or k_sig_cache.dim() != 4 or v_cache.dim() != 4:
        raise ValueError("bad ranks: q [B, heads, d], caches [B, Lcap, heads, dim]")
    B, hs, d = q_sig.shape
    hn = q_noise.shape[1]
    Lcap = k_sig_cache.shape[1]
    dv = v_cache.shape[3]
    bf = torch.bfloat16
    _expect(q_sig, "q_sig", bf, (B, hs, d), dev)
    _expect(q_noise, "q_noise", bf, (B, hn, d), dev)
    _expect(k_sig_cache, "k_sig_cache", bf, (B, Lcap, hs, d), dev)
    _expect(k_noise_cache, "k_noise_cache", bf, (B, Lcap, hn, d), dev)
    _expect(v_cache, "v_cache", bf, (B, Lcap, hs, dv), dev)
    _expect(cache_lens, "cache_lens", torch.int32, (B,), dev)
    _expect(lam, "lam", torch.float32, (hs,), dev)
    if out is None:
        out = torch.empty((B, hs, dv), dtype=bf, device=dev)
    _expect(out, "out", bf, (B, hs, dv), dev)
    need = gda_attn_decode_workspace_size(B, Lcap, hs, hn, dv)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    ws_bytes = workspace.numel() * workspace.element_size()
    with torch.cuda.device(dev):
        rc = _load().gda_attn_decode(
            _ptr(q_sig), _ptr(q_noise), _ptr(k_sig_cache), _ptr(k_noise_cache), _ptr(v_cache),
            _ptr(cache_lens), _ptr(lam), float(lambda_init), _ptr(out), B, Lcap, hs, hn, d, dv,
            float(eps), _ptr(workspace), ws_bytes, _stream(dev))
    _check(rc, "gda decode")
    return out


def gda_attn_decode_noalloc(q_sig, q_noise, k_sig_cache, k_noise_cache, v_cache, cache_lens,
                            lam, lambda_init: float, *, eps: float = 1e-5, out=None):
    """Decode without a workspace: the library's fixed scratch array holds the split partials.

    For callers that cannot allocate device memory.  Calls that overlap on
    the GPU race on the shared scratch array; see include/gda.h.
    """
    dev = q_sig.device
    B, hs, d = q_sig.shape
    hn = q_noise.shape[1]
    Lcap = k_sig_cache.shape[1]
    dv = v_cache.shape[3]
    bf = torch.bfloat16
    _expect(q_sig, "q_sig", bf, (B, hs, d), dev)
    _expect(q_noise, "q_noise", bf, (B, hn, d), dev)
    _expect(k_sig_cache, "k_sig_cache", bf, (B, Lcap, hs, d), dev)
    _expect(k_noise_cache, "k_noise_cache", bf, (B, Lcap, hn, d), dev)
    _expect(v_cache, "v_cache", bf, (B, Lcap, hs, dv), dev)
    _expect(cache_lens, "cache_lens", torch.int32, (B,), dev)
    _expect(lam, "lam", torch.float32, (hs,), dev)
    if out is None:
        out = torch.empty((B, hs, dv), dtype=bf, device=dev)
    _expect(out, "out", bf, (B, hs, dv), dev)
    with torch.cuda.device(dev):
        rc = _load().gda_attn_decode_noalloc(
            _ptr(q_sig), _ptr(q_noise), _ptr(k_sig_cache), _ptr(k_noise_cache), _ptr(v_cache),
            _ptr(cache_lens), _ptr(lam), float(lambda_init), _ptr(out), B, Lcap, hs, hn, d, dv,
            float(eps), _stream(dev))
    _check(rc, "gda decode (no allocation)")
    return out


# The raw handle of a device's current stream, without a Stream object around it (2 us of a call's 10).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _enqueue(entry, what, device, *args):
    """Calls entry(*args, stream) with `device` current, on its current stream."""
    index = device.index
    if torch.cuda.current_device() == index:
        rc = entry(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            rc = entry(*args, _raw_stream(index))
    if rc != GDA_OK:
        raise GDAError(rc, what)


def _int32(*sizes):
    """Refuses sizes that a C int does not hold (ctypes would pass their low 32 bits)."""
    if min(sizes) < -0x80000000 or max(sizes) > 0x7fffffff:
        raise ValueError(f"sizes {sizes} do not all fit 32 bits")


def _workspace(workspace, need, device):
    if workspace is None:
        return torch.empty((max(need, 16),), dtype=torch.uint8, device=device)
    _expect(workspace, "workspace", torch.uint8, (workspace.numel(),), device)
    return workspace


def _expect_all(device, *wanted):
    """_expect for several (tensor, name, dtype, shape) at once: the checks without a call for each."""
    index = device.index
    for t, name, dtype, shape in wanted:
        if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == index
                and t.is_contiguous()):
            _expect(t, name, dtype, shape, device)


def _token_stride(t, name, dtype, shape, device):
    """Checks t [*tokens, heads, dim] and returns the elements between its tokens.

    A token's heads are dense; the tokens are a constant number of elements
    apart (a slice of a fused projection, or a dense tensor).
    """
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != device.index:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    heads, dim = shape[-2], shape[-1]
    strides = t.stride()
    if strides[-1] != 1 or (strides[-2] != dim and heads > 1):
        raise ValueError(f"{name}: the heads of a token must be dense")
    if len(strides) == 3:
        return strides[0] if shape[0] > 1 else heads * dim
    step, expect = heads * dim, None
    for i in range(len(strides) - 3, -1, -1):
        size, stride = shape[i], strides[i]
        if size == 1:
            continue
        if expect is None:
            step = stride
        elif stride != expect:
            raise ValueError(f"{name}: its tokens must be a constant number of elements apart")
        expect = stride * size
    return step


def _norm_rope_sizes(q_sig, q_noise, weight, positions, inv_freq):
    dev = q_sig.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    if q_sig.dim() < 3 or q_noise.dim() != q_sig.dim():
        raise ValueError("projections must be [*tokens, heads, d]")
    if q_sig.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"q_sig has dtype {q_sig.dtype}, expected bfloat16 or float32")
    *lead, hs, d = q_sig.shape
    lead = tuple(lead)
    hn = q_noise.shape[-2]
    half = inv_freq.numel()
    _expect_all(dev, (weight, "weight", torch.float32, (4, d)), (positions, "positions", torch.int32, lead),
                (inv_freq, "inv_freq", torch.float32, (half,)))
    sig, noise = lead + (hs, d), lead + (hn, d)
    shapes = (sig, sig, noise, noise)
    return dev, q_sig.dtype, positions.numel(), hs, hn, d, 2 * half, shapes


_PROJECTIONS = ("q_sig", "k_sig", "q_noise", "k_noise")


def gda_qk_norm_rope(q_sig, k_sig, q_noise, k_noise, weight, positions, inv_freq, *, eps: float = 1e-5,
                     interleaved: bool = False, out=None):
    """Per-head RMSNorm and rotation by position of the four projections, in one pass.

    q_sig, k_sig [*tokens, h_s, d] and q_noise, k_noise [*tokens, h_n, d]
    (bf16 or float32; one or two token dims, dense or slices of a fused
    projection), weight [4, d] float32 (the rows of the four), positions
    [*tokens] int32, inv_freq [rot / 2] float32: the first rot dims of a head
    rotate, in pairs (i, i + rot / 2), or (2i, 2i + 1) with ``interleaved``.
    Returns the four dense outputs (``out`` may hold them; a dense input may
    be its own output).
    """
    dev, dt, T, hs, hn, d, rot, shapes = _norm_rope_sizes(q_sig, q_noise, weight, positions, inv_freq)
    x = (q_sig, k_sig, q_noise, k_noise)
    strides = [_token_stride(t, n, dt, s, dev) for t, n, s in zip(x, _PROJECTIONS, shapes)]
    if out is None:
        out = tuple([torch.empty(s, dtype=dt, device=dev) for s in shapes])
    else:
        out = _given(out, 4, "out")
        for t, n, s in zip(out, _PROJECTIONS, shapes):
            _expect(t, "out " + n, dt, s, dev)
    lib = _load()
    _enqueue(lib.gda_qk_norm_rope if dt is torch.bfloat16 else lib.gda_qk_norm_rope_f32, "gda norm and rotation", dev,
             *[t.data_ptr() for t in (*x, weight, positions, inv_freq, *out)], T, hs, hn, d, rot, *strides, float(eps),
             GDA_FLAG_ROPE_INTERLEAVED if interleaved else 0)
    return tuple(out)


def gda_qk_norm_rope_bwd_workspace_size(T: int, h_s: int, h_n: int, d: int) -> int:
    _int32(T, h_s, h_n, d)
    return int(_load().gda_qk_norm_rope_bwd_workspace_size(T, h_s, h_n, d))


def gda_qk_norm_rope_bwd(q_sig, k_sig, q_noise, k_noise, weight, positions, inv_freq, dq_sig, dk_sig, dq_noise,
                         dk_noise, *, eps: float = 1e-5, interleaved: bool = False, grads=None, workspace=None):
    """Gradients of ``gda_qk_norm_rope``: (dq_sig, dk_sig, dq_noise, dk_noise, dweight).

    Inputs as for the forward call plus the float32 gradients of its outputs
    (dense, as ``gda_attn_bwd`` and ``gda_attn_bwd_bf16`` return them).  The
    input gradients have the inputs' type, dweight [4, d] is float32.
    ``grads`` may hold the five to overwrite (the first four may be slices of
    one fused gradient).
    """
    dev, dt, T, hs, hn, d, rot, shapes = _norm_rope_sizes(q_sig, q_noise, weight, positions, inv_freq)
    x, dy = (q_sig, k_sig, q_noise, k_noise), (dq_sig, dk_sig, dq_noise, dk_noise)
    strides = [_token_stride(t, n, dt, s, dev) for t, n, s in zip(x, _PROJECTIONS, shapes)]
    if grads is None:
        grads = (*[torch.empty(s, dtype=dt, device=dev) for s in shapes],
                 torch.empty((4, d), dtype=torch.float32, device=dev))
        strides += [hs * d, hs * d, hn * d, hn * d]
    else:
        grads = _given(grads, 5, "grads")
        strides += [_token_stride(t, "grads " + n, dt, s, dev) for t, n, s in zip(grads, _PROJECTIONS, shapes)]
        _expect(grads[4], "dweight", torch.float32, (4, d), dev)
    f32 = torch.float32
    _expect_all(dev, (dq_sig, "dq_sig", f32, shapes[0]), (dk_sig, "dk_sig", f32, shapes[1]),
                (dq_noise, "dq_noise", f32, shapes[2]), (dk_noise, "dk_noise", f32, shapes[3]))
    lib = _load()
    workspace = _workspace(workspace, lib.gda_qk_norm_rope_bwd_workspace_size(T, hs, hn, d), dev)
    _enqueue(lib.gda_qk_norm_rope_bwd if dt is torch.bfloat16 else lib.gda_qk_norm_rope_bwd_f32,
             "gda norm and rotation backward", dev,
             *[t.data_ptr() for t in (*x, weight, positions, inv_freq, *dy, *grads)], T, hs, hn, d, rot,
             (ctypes.c_longlong * 8)(*strides), float(eps), GDA_FLAG_ROPE_INTERLEAVED if interleaved else 0,
             workspace.data_ptr(), workspace.numel())
    return tuple(grads)


def gda_block_tables(cache_lens, new_lens, block_table, free_pages, free_count, page_size: int, num_pages: int,
                     max_rows: int, *, out=None):
    """Block table, slots and positions of a step's new tokens, from the sequences' lengths.

    int32 CUDA tensors: cache_lens [B] (positions held), new_lens [B] (tokens
    to add, 0 for none), block_table [B, max_pages] (updated in place),
    free_pages [F] and free_count [1] (a stack, its top at free_count - 1).
    Returns (slot_map [max_rows], positions [max_rows], row_starts [B + 1],
    lens [B], free_left [1]): the new tokens' rows follow sequence after
    sequence, rows past the last one and rows of a refused sequence have slot
    -1.  ``out`` may hold the five; its lens may be cache_lens and its
    free_left free_count.  See include/gda.h for refusals.
    """
    dev = cache_lens.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    if block_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("block_table must be [B, max_pages] and free_pages 1-D")
    i32 = torch.int32
    B, max_pages = block_table.shape
    free = free_pages.numel()
    _int32(page_size, num_pages, max_rows, free, max_pages)
    _expect_all(dev, (cache_lens, "cache_lens", i32, (B,)), (new_lens, "new_lens", i32, (B,)),
                (block_table, "block_table", i32, (B, max_pages)), (free_pages, "free_pages", i32, (free,)),
                (free_count, "free_count", i32, (1,)))
    shapes = ((max_rows,), (max_rows,), (B + 1,), (B,), (1,))
    if out is None:
        out = tuple([torch.empty(s, dtype=i32, device=dev) for s in shapes])
    else:
        out = _given(out, 5, "out")
        for t, n, s in zip(out, ("slot_map", "positions", "row_starts", "lens", "free_left"), shapes):
            _expect(t, n, i32, s, dev)
    _enqueue(_load().gda_block_tables, "gda block tables", dev,
             *[t.data_ptr() for t in (cache_lens, new_lens, block_table, free_pages, free_count, *out)], B, max_pages,
             page_size, num_pages, free, max_rows)
    return tuple(out)


_FP4 = getattr(torch, "float4_e2m1fn_x2", torch.uint8)
_FP8 = torch.float8_e4m3fn


def _fp4_cache(pools, blocks, scales, rows, hs, hn, d, dv, dev):
    """Checks the nine tensors of a 4-bit cache; returns their addresses in the order of the C entries."""
    f32, sig, noise = torch.float32, rows + (hs, d // 2), rows + (hn, d // 2)
    # one-byte tensors: uint8, or all of a kind in their own type
    code = _FP4 if getattr(pools[0], "dtype", None) is _FP4 else torch.uint8
    block = _FP8 if getattr(blocks[0], "dtype", None) is _FP8 else torch.uint8
    _expect_all(dev, (pools[0], "k_sig codes", code, sig), (pools[1], "k_noise codes", code, noise),
                (pools[2], "v codes", code, rows + (hs, dv // 2)),
                (blocks[0], "k_sig_block_scale", block, rows + (hs, d // 16)),
                (blocks[1], "k_noise_block_scale", block, rows + (hn, d // 16)),
                (blocks[2], "v_block_scale", block, rows + (hs, dv // 16)), (scales[0], "k_sig_scale", f32, (hs,)),
                (scales[1], "k_noise_scale", f32, (hn,)), (scales[2], "v_scale", f32, (hs,)))
    return [t.data_ptr() for t in (*pools, *blocks, *scales)]


def gda_cache_append_fp4(k_sig, k_noise, v, slot_map, k_sig_pool, k_noise_pool, v_pool, k_sig_block_scale,
                         k_noise_block_scale, v_block_scale, k_sig_scale, k_noise_scale, v_scale):
    """Writes tokens' K and V rows (bf16 [T, heads, dim]) into a 4-bit cache, in place.

    slot_map [T] int32: the slot of each token (page * page_size + offset, as
    ``gda_block_tables`` gives them), negative to leave it out; the slots of a
    call differ.  Pools [num_pages, page_size, heads, dim / 2] uint8 (e2m1, two
    to a byte; a contiguous cache [B, Lcap, ...] is B pages of Lcap), block
    scales [num_pages, page_size, heads, dim / 16] float8_e4m3fn (or uint8),
    head scales [heads] float32.  The rows may be slices of a fused projection.
    """
    dev = k_sig.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    if k_sig.dim() != 3 or k_noise.dim() != 3 or v.dim() != 3 or k_sig_pool.dim() != 4:
        raise ValueError("rows must be [T, heads, dim] and pools [num_pages, page_size, heads, dim / 2]")
    T, hs, d = k_sig.shape
    hn, dv = k_noise.shape[1], v.shape[2]
    rows = tuple(k_sig_pool.shape[:2])
    bf = torch.bfloat16
    strides = [_token_stride(t, n, bf, (T, h, dim), dev)
               for t, n, h, dim in ((k_sig, "k_sig", hs, d), (k_noise, "k_noise", hn, d), (v, "v", hs, dv))]
    _expect(slot_map, "slot_map", torch.int32, (T,), dev)
    cache = _fp4_cache((k_sig_pool, k_noise_pool, v_pool), (k_sig_block_scale, k_noise_block_scale, v_block_scale),
                       (k_sig_scale, k_noise_scale, v_scale), rows, hs, hn, d, dv, dev)
    _enqueue(_load().gda_cache_append_fp4, "gda 4-bit cache append", dev, k_sig.data_ptr(), k_noise.data_ptr(),
             v.data_ptr(), slot_map.data_ptr(), *cache, T, *rows, hs, hn, d, dv, *strides)


def gda_cache_read_fp4(slot_map, k_sig_pool, k_noise_pool, v_pool, k_sig_block_scale, k_noise_block_scale,
                       v_block_scale, k_sig_scale, k_noise_scale, v_scale, *, out=None):
    """The rows of a 4-bit cache at slot_map [T] as bf16: (k_sig, k_noise, v), each [T, heads, dim].

    Zero rows for negative slots.  ``out`` may hold the three tensors.  The
    cache is as in ``gda_cache_append_fp4``; the rows of a sequence's slots, in
    order, are the keys and values of a prefix for ``gda_attn_fwd_chunk``.
    """
    dev = slot_map.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    if slot_map.dim() != 1 or k_sig_pool.dim() != 4 or k_noise_pool.dim() != 4 or v_pool.dim() != 4:
        raise ValueError("slot_map must be 1-D and pools [num_pages, page_size, heads, dim / 2]")
    T = slot_map.numel()
    rows = tuple(k_sig_pool.shape[:2])
    hs, d = k_sig_pool.shape[2], 2 * k_sig_pool.shape[3]
    hn, dv = k_noise_pool.shape[2], 2 * v_pool.shape[3]
    _expect(slot_map, "slot_map", torch.int32, (T,), dev)
    cache = _fp4_cache((k_sig_pool, k_noise_pool, v_pool), (k_sig_block_scale, k_noise_block_scale, v_block_scale),
                       (k_sig_scale, k_noise_scale, v_scale), rows, hs, hn, d, dv, dev)
    shapes = ((T, hs, d), (T, hn, d), (T, hs, dv))
    if out is None:
        out = tuple([torch.empty(s, dtype=torch.bfloat16, device=dev) for s in shapes])
    else:
        out = _given(out, 3, "out")
        for t, n, s in zip(out, ("k_sig", "k_noise", "v"), shapes):
            _expect(t, n, torch.bfloat16, s, dev)
    _enqueue(_load().gda_cache_read_fp4, "gda 4-bit cache read", dev, slot_map.data_ptr(), *cache,
             *[t.data_ptr() for t in out], T, *rows, hs, hn, d, dv)
    return tuple(out)


def gda_attn_decode_fp4_workspace_size(B: int, h_s: int, h_n: int, d: int, dv: int) -> int:
    _int32(B, h_s, h_n, d, dv)
    return int(_load().gda_attn_decode_fp4_workspace_size(B, h_s, h_n, d, dv))


def _decode_fp4(q_sig, q_noise, pools, blocks, scales, block_table, cache_lens, lam, lambda_init, eps, out, workspace):
    dev = q_sig.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    if q_sig.dim() != 3 or q_noise.dim() != 3 or pools[0].dim() != 4 or pools[2].dim() != 4:
        raise ValueError("bad ranks: q [B, heads, d], caches [.., .., heads, dim / 2]")
    B, hs, d = q_sig.shape
    hn, dv = q_noise.shape[1], 2 * pools[2].shape[3]
    rows = tuple(pools[0].shape[:2])
    bf = torch.bfloat16
    _expect_all(dev, (q_sig, "q_sig", bf, (B, hs, d)), (q_noise, "q_noise", bf, (B, hn, d)),
                (cache_lens, "cache_lens", torch.int32, (B,)), (lam, "lam", torch.float32, (hs,)))
    cache = _fp4_cache(pools, blocks, scales, rows, hs, hn, d, dv, dev)
    if out is None:
        out = torch.empty((B, hs, dv), dtype=bf, device=dev)
    else:
        _expect(out, "out", bf, (B, hs, dv), dev)
    workspace = _workspace(workspace, _load().gda_attn_decode_fp4_workspace_size(B, hs, hn, d, dv), dev)
    head = (q_sig.data_ptr(), q_noise.data_ptr(), *cache)
    tail = (hs, hn, d, dv, float(eps), workspace.data_ptr(), workspace.numel())
    if block_table is None:
        if rows[0] != B:
            raise ValueError(f"caches hold {rows[0]} sequences, expected {B}")
        _enqueue(_load().gda_attn_decode_fp4, "gda decode (4-bit cache)", dev, *head, cache_lens.data_ptr(),
                 lam.data_ptr(), float(lambda_init), out.data_ptr(), B, rows[1], *tail)
    else:
        if block_table.dim() != 2:
            raise ValueError("block_table must be [B, max_pages]")
        max_pages = block_table.shape[1]
        _expect(block_table, "block_table", torch.int32, (B, max_pages), dev)
        _enqueue(_load().gda_attn_decode_paged_fp4, "gda decode (4-bit cache)", dev, *head, block_table.data_ptr(),
                 cache_lens.data_ptr(), lam.data_ptr(), float(lambda_init), out.data_ptr(), B, max_pages, rows[1],
                 rows[0], *tail)
    return out


def gda_attn_decode_fp4(q_sig, q_noise, k_sig_cache, k_noise_cache, v_cache, k_sig_block_scale, k_noise_block_scale,
                        v_block_scale, k_sig_scale, k_noise_scale, v_scale, cache_lens, lam, lambda_init: float, *,
                        eps: float = 1e-5, out=None, workspace=None):
    """bf16 decode over 4-bit caches: cached value = e2m1 code * block scale * head scale.

    Caches [B, Lcap, heads, dim / 2] uint8, block scales [B, Lcap, heads,
    dim / 16] float8_e4m3fn (or uint8), head scales [heads] float32, as
    ``gda_cache_append_fp4`` writes them.  A cache length of 0 gives a zero row.
    """
    return _decode_fp4(q_sig, q_noise, (k_sig_cache, k_noise_cache, v_cache),
                       (k_sig_block_scale, k_noise_block_scale, v_block_scale), (k_sig_scale, k_noise_scale, v_scale),
                       None, cache_lens, lam, lambda_init, eps, out, workspace)


def gda_attn_decode_paged_fp4(q_sig, q_noise, k_sig_pool, k_noise_pool, v_pool, k_sig_block_scale,
                              k_noise_block_scale, v_block_scale, k_sig_scale, k_noise_scale, v_scale, block_table,
                              cache_lens, lam, lambda_init: float, *, eps: float = 1e-5, out=None, workspace=None):
    """``gda_attn_decode_fp4`` over page pools [num_pages, page_size, heads, ..] and a block table
    [B, max_pages] int32 (position j of sequence b is row j % page_size of page block_table[b, j // page_size])."""
    if not isinstance(block_table, torch.Tensor):
        raise TypeError("block_table must be a torch.Tensor")
    return _decode_fp4(q_sig, q_noise, (k_sig_pool, k_noise_pool, v_pool),
                       (k_sig_block_scale, k_noise_block_scale, v_block_scale), (k_sig_scale, k_noise_scale, v_scale),
                       block_table, cache_lens, lam, lambda_init, eps, out, workspace)


_shape_of, _dtype_of = operator.attrgetter("shape"), operator.attrgetter("dtype")
_device_of, _is_dense, _address_of = torch.Tensor.get_device, torch.Tensor.is_contiguous, torch.Tensor.data_ptr


def _alike(index, wanted, tensors):
    """Whether the tensors have the dtypes and shapes of wanted = (names, dtypes, shapes) and are on device ``index``.

    Whole columns at once: the checks of a small call take as long as its kernels."""
    try:
        return (tuple(map(_dtype_of, tensors)) == wanted[1] and tuple(map(_shape_of, tensors)) == wanted[2]
                and set(map(_device_of, tensors)) == {index})
    except (AttributeError, TypeError):
        return False                      # not a tensor: the caller's check names it


def _addresses(index, device, wanted, tensors):
    """Checks tensors against wanted = (names, dtypes, shapes) as ``_expect`` does, and returns their addresses."""
    if not _alike(index, wanted, tensors) or not all(map(_is_dense, tensors)):
        for t, name, dtype, shape in zip(tensors, *wanted):
            _expect(t, name, dtype, shape, device)
    return list(map(_address_of, tensors))


def _token_strides(index, device, wanted, rows):
    """``_token_stride`` of rows [T, heads, dim]."""
    if _alike(index, wanted, rows):
        strides = [t.stride() for t in rows]
        if all(s[2] == 1 and (s[1] == n or h == 1) for s, (_, h, n) in zip(strides, wanted[2])):
            return [s[0] if T > 1 else h * n for s, (T, h, n) in zip(strides, wanted[2])]
    return [_token_stride(t, name, dtype, shape, device) for t, name, dtype, shape in zip(rows, *wanted)]


def _cuda_index(t):
    """The device index of the tensor that the others are to share their device with."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("inputs must be torch.Tensors")
    index = t.get_device()
    if index < 0:
        raise ValueError("inputs must be CUDA tensors")
    return index


def _bytes_of(name, *sizes):
    """A workspace size of the library."""
    _int32(*sizes)
    return int(getattr(_load(), name)(*sizes))


# What the calls over the 8-bit cache check of their tensors follows from sizes alone: worked out once for each set of
# them, as (names, dtypes, shapes) with what else the call needs.
_plan = functools.lru_cache(maxsize=256)


def _blocks_of_a_page(scale):
    shape = getattr(scale, "shape", ())
    if len(shape) != 3:
        raise ValueError("scales must be [num_pages, page_size / block, heads]")
    return shape[1]


def _fp8_block_cache(pages, size, per, hs, hn, d, dv, code):
    """(name, dtype, shape) of the six tensors of an 8-bit cache with block scales, and the tokens of a block."""
    if per < 1 or size % per != 0:
        raise ValueError(f"pages of {size} rows do not hold {per} blocks of equal size")
    _int32(pages, size, hs, hn, d, dv)
    f32, sig, noise = torch.float32, (pages, per, hs), (pages, per, hn)
    return (("k_sig codes", code, (pages, size, hs, d)), ("k_noise codes", code, (pages, size, hn, d)),
            ("v codes", code, (pages, size, hs, dv)), ("k_sig_scale", f32, sig), ("k_noise_scale", f32, noise),
            ("v_scale", f32, sig)), size // per


def _code_of(pool):
    return _FP8 if pool.dtype is _FP8 else torch.uint8


@_plan
def _append_fp8_block_plan(T, hs, hn, d, dv, pages, size, per, code, bounds):
    cache, block = _fp8_block_cache(pages, size, per, hs, hn, d, dv, code)
    bf, i8 = torch.bfloat16, torch.int8
    rows = (("k_sig", bf, (T, hs, d)), ("k_noise", bf, (T, hn, d)), ("v", bf, (T, hs, dv)))
    rest = (("slot_map", torch.int32, (T,)), *cache)
    if bounds:
        rest += (("k_sig_bounds", i8, (pages, per, hs, 2, d)), ("k_noise_bounds", i8, (pages, per, hn, 2, d)))
    return tuple(zip(*rows)), tuple(zip(*rest)), block, _bytes_of("gda_cache_append_fp8_block_workspace_size", T, pages, size)


@_plan
def _read_fp8_block_plan(T, hs, hn, d, dv, pages, size, per, code):
    cache, block = _fp8_block_cache(pages, size, per, hs, hn, d, dv, code)
    _int32(T)
    bf = torch.bfloat16
    out = (("out k_sig", bf, (T, hs, d)), ("out k_noise", bf, (T, hn, d)), ("out v", bf, (T, hs, dv)))
    return tuple(zip(("slot_map", torch.int32, (T,)), *cache, *out)), block


def _pages_of_sequences(block_table):
    """The pages of a sequence, or None: contiguous caches are a page for each."""
    if block_table is None:
        return None
    shape = getattr(block_table, "shape", None)
    if shape is None:
        raise TypeError("block_table must be a torch.Tensor")
    if len(shape) != 2:
        raise ValueError("block_table must be [B, max_pages]")
    return shape[1]


def _block_table(B, pages, max_pages):
    """(name, dtype, shape) of a block table, or of none."""
    if max_pages is not None:
        _int32(max_pages)
        return (("block_table", torch.int32, (B, max_pages)),)
    if pages != B:
        raise ValueError(f"caches hold {pages} sequences, expected {B}")
    return ()


@_plan
def _block_select_plan(B, hs, hn, d, pages, per, max_pages, block, keep, first, last):
    bf, i8, i32, f32 = torch.bfloat16, torch.int8, torch.int32, torch.float32
    table = _block_table(B, pages, max_pages)
    most = per * (max_pages if table else 1)
    _int32(pages, per * block, keep, first, last, most, d)
    wanted = (("q_sig", bf, (B, hs, d)), ("q_noise", bf, (B, hn, d)), ("k_sig_bounds", i8, (pages, per, hs, 2, d)),
              ("k_noise_bounds", i8, (pages, per, hn, 2, d)), ("k_sig_scale", f32, (pages, per, hs)),
              ("k_noise_scale", f32, (pages, per, hn)), *table, ("cache_lens", i32, (B,)),
              ("block_list", i32, (B, hn, keep)), ("block_count", i32, (B,)))
    return tuple(zip(*wanted)), _bytes_of("gda_block_select_workspace_size", B, most, hs, hn)


@_plan
def _decode_fp8_block_plan(B, hs, hn, d, dv, pages, size, per, code, max_pages, keep):
    cache, block = _fp8_block_cache(pages, size, per, hs, hn, d, dv, code)
    bf, i32 = torch.bfloat16, torch.int32
    lists = ()
    if keep is not None:
        _int32(keep)
        lists = (("block_list", i32, (B, hn, keep)), ("block_count", i32, (B,)))
    wanted = (("q_sig", bf, (B, hs, d)), ("q_noise", bf, (B, hn, d)), *cache, *_block_table(B, pages, max_pages), *lists,
              ("cache_lens", i32, (B,)), ("lam", torch.float32, (hs,)), ("out", bf, (B, hs, dv)))
    return tuple(zip(*wanted)), block, _bytes_of("gda_attn_decode_fp8_block_workspace_size", B, hs, hn, d, dv)


def gda_cache_append_fp8_block_workspace_size(T: int, num_pages: int, page_size: int) -> int:
    return _bytes_of("gda_cache_append_fp8_block_workspace_size", T, num_pages, page_size)


def gda_cache_append_fp8_block(k_sig, k_noise, v, slot_map, k_sig_pool, k_noise_pool, v_pool, k_sig_scale,
                               k_noise_scale, v_scale, *, k_sig_bounds=None, k_noise_bounds=None, workspace=None):
    """Writes tokens' K and V rows (bf16 [T, heads, dim]) into an 8-bit cache with block scales, in place.

    slot_map [T] int32 as for ``gda_cache_append_fp4``.  Pools [num_pages,
    page_size, heads, dim] float8_e4m3fn (or uint8); scales [num_pages,
    page_size / block, heads] float32, one for ``block`` (16, 32, 64 or 128)
    consecutive rows of a page: a contiguous cache [B, Lcap, ...] is B pages of
    Lcap.  A call that writes the first row of a block starts it anew, others
    may raise its scale, and then the codes that are there follow.
    k_sig_bounds, k_noise_bounds [num_pages, page_size / block, heads, 2, d]
    int8 (both or neither) are kept for ``gda_block_select``.  The rows may be
    slices of a fused projection.  See include/gda.h.
    """
    index = _cuda_index(k_sig)
    dev = k_sig.device
    if k_sig.dim() != 3 or k_noise.dim() != 3 or v.dim() != 3 or k_sig_pool.dim() != 4:
        raise ValueError("rows must be [T, heads, dim] and pools [num_pages, page_size, heads, dim]")
    if (k_sig_bounds is None) != (k_noise_bounds is None):
        raise ValueError("k_sig_bounds and k_noise_bounds are given both or not at all")
    T, hs, d = k_sig.shape
    hn, dv = k_noise.shape[1], v.shape[2]
    pages, size, _, _ = k_sig_pool.shape
    bounds = () if k_sig_bounds is None else (k_sig_bounds, k_noise_bounds)
    rows, rest, block, need = _append_fp8_block_plan(T, hs, hn, d, dv, pages, size, _blocks_of_a_page(k_sig_scale),
                                                     _code_of(k_sig_pool), len(bounds))
    strides = _token_strides(index, dev, rows, (k_sig, k_noise, v))
    at = _addresses(index, dev, rest, (slot_map, k_sig_pool, k_noise_pool, v_pool, k_sig_scale, k_noise_scale, v_scale,
                                       *bounds))
    if not bounds:
        at += (None, None)
    if workspace is not None or need:
        workspace = _workspace(workspace, need, dev)
        space = (workspace.data_ptr(), workspace.numel())
    else:
        space = (None, 0)
    _enqueue(_load().gda_cache_append_fp8_block, "gda 8-bit block cache append", dev, k_sig.data_ptr(), k_noise.data_ptr(),
             v.data_ptr(), *at, T, pages, size, block, hs, hn, d, dv, *strides, *space)


def gda_cache_read_fp8_block(slot_map, k_sig_pool, k_noise_pool, v_pool, k_sig_scale, k_noise_scale, v_scale, *,
                             out=None):
    """The rows of an 8-bit cache with block scales at slot_map [T] as bf16: (k_sig, k_noise, v), each [T, heads, dim].

    Zero rows for negative slots.  ``out`` may hold the three tensors.  The
    cache is as in ``gda_cache_append_fp8_block``; the rows of a sequence's
    slots, in order, are the keys and values of a prefix for
    ``gda_attn_fwd_chunk``.
    """
    index = _cuda_index(slot_map)
    dev = slot_map.device
    if slot_map.dim() != 1 or k_sig_pool.dim() != 4 or k_noise_pool.dim() != 4 or v_pool.dim() != 4:
        raise ValueError("slot_map must be 1-D and pools [num_pages, page_size, heads, dim]")
    T = slot_map.numel()
    pages, size, hs, d = k_sig_pool.shape
    hn, dv = k_noise_pool.shape[2], v_pool.shape[3]
    wanted, block = _read_fp8_block_plan(T, hs, hn, d, dv, pages, size, _blocks_of_a_page(k_sig_scale),
                                         _code_of(k_sig_pool))
    if out is None:
        bf = torch.bfloat16
        out = (torch.empty((T, hs, d), dtype=bf, device=dev), torch.empty((T, hn, d), dtype=bf, device=dev),
               torch.empty((T, hs, dv), dtype=bf, device=dev))
    else:
        out = _given(out, 3, "out")
    at = _addresses(index, dev, wanted, (slot_map, k_sig_pool, k_noise_pool, v_pool, k_sig_scale, k_noise_scale, v_scale,
                                         *out))
    _enqueue(_load().gda_cache_read_fp8_block, "gda 8-bit block cache read", dev, *at, T, pages, size, block, hs, hn, d, dv)
    return tuple(out)


def gda_block_select_workspace_size(B: int, max_blocks: int, h_s: int, h_n: int) -> int:
    return _bytes_of("gda_block_select_workspace_size", B, max_blocks, h_s, h_n)


def gda_block_select(q_sig, q_noise, k_sig_bounds, k_noise_bounds, k_sig_scale, k_noise_scale, cache_lens, block: int,
                     keep: int, *, block_table=None, first: int = 1, last: int = 1, out=None, workspace=None):
    """The ``keep`` blocks of each sequence that its queries are to attend, by an estimate of their largest logits.

    q_sig [B, h_s, d], q_noise [B, h_n, d] bf16 (as the decode takes them);
    bounds and key scales as ``gda_cache_append_fp8_block`` keeps them for
    blocks of ``block`` tokens; cache_lens [B] int32; block_table [B, max_pages]
    int32, or None for contiguous caches.  Returns (block_list [B, h_n, keep]
    int32, ascending and then -1, block_count [B] int32) for
    ``gda_attn_decode_sparse_fp8_block``: all blocks of a sequence that has no
    more, else its first ``first`` and last ``last`` ones and those of the
    highest score (include/gda.h).  ``out`` may hold the two.
    """
    index = _cuda_index(q_sig)
    dev = q_sig.device
    if q_sig.dim() != 3 or q_noise.dim() != 3:
        raise ValueError("queries must be [B, heads, d]")
    if k_sig_bounds.dim() != 5:
        raise ValueError("bounds must be [num_pages, page_size / block, heads, 2, d]")
    B, hs, d = q_sig.shape
    hn = q_noise.shape[1]
    pages, per, _, _, _ = k_sig_bounds.shape
    max_pages = _pages_of_sequences(block_table)
    wanted, need = _block_select_plan(B, hs, hn, d, pages, per, max_pages, block, keep, first, last)
    if out is None:
        i32 = torch.int32
        out = (torch.empty((B, hn, keep), dtype=i32, device=dev), torch.empty((B,), dtype=i32, device=dev))
    else:
        out = _given(out, 2, "out")
    table = () if block_table is None else (block_table,)
    at = _addresses(index, dev, wanted, (q_sig, q_noise, k_sig_bounds, k_noise_bounds, k_sig_scale, k_noise_scale, *table,
                                         cache_lens, *out))
    if not table:
        at.insert(6, None)
    if workspace is not None or need:
        workspace = _workspace(workspace, need, dev)
        space = (workspace.data_ptr(), workspace.numel())
    else:
        space = (None, 0)
    _enqueue(_load().gda_block_select, "gda block selection", dev, *at, B, max_pages if table else 1, per * block, pages, block, keep,
             first, last, hs, hn, d, *space)
    return tuple(out)


def gda_attn_decode_fp8_block_workspace_size(B: int, h_s: int, h_n: int, d: int, dv: int) -> int:
    return _bytes_of("gda_attn_decode_fp8_block_workspace_size", B, h_s, h_n, d, dv)


def _decode_fp8_block(q_sig, q_noise, pools, scales, block_table, lists, cache_lens, lam, lambda_init, eps, out,
                      workspace):
    index = _cuda_index(q_sig)
    dev = q_sig.device
    if q_sig.dim() != 3 or q_noise.dim() != 3 or pools[0].dim() != 4 or pools[2].dim() != 4:
        raise ValueError("bad ranks: q [B, heads, d], caches [.., .., heads, dim]")
    B, hs, d = q_sig.shape
    hn, dv = q_noise.shape[1], pools[2].shape[3]
    pages, size, _, _ = pools[0].shape
    max_pages = _pages_of_sequences(block_table)
    keep = None
    if lists is not None:
        shape = getattr(lists[0], "shape", ())
        if len(shape) != 3:
            raise ValueError("block_list must be [B, h_n, keep]")
        keep = shape[2]
    wanted, block, need = _decode_fp8_block_plan(B, hs, hn, d, dv, pages, size, _blocks_of_a_page(scales[0]),
                                                 _code_of(pools[0]), max_pages, keep)
    if out is None:
        out = torch.empty((B, hs, dv), dtype=torch.bfloat16, device=dev)
    table = () if block_table is None else (block_table,)
    at = _addresses(index, dev, wanted, (q_sig, q_noise, *pools, *scales, *table, *(lists or ()), cache_lens, lam, out))
    workspace = _workspace(workspace, need, dev)
    at.insert(-1, float(lambda_init))
    tail = (hs, hn, d, dv, float(eps), workspace.data_ptr(), workspace.numel())
    what = "gda decode (8-bit block cache)"
    lib = _load()
    if lists is not None:
        if not table:
            at.insert(8, None)
        _enqueue(lib.gda_attn_decode_sparse_fp8_block, what, dev, *at, B, max_pages if table else 1, size, pages,
                 block, keep, *tail)
    elif not table:
        _enqueue(lib.gda_attn_decode_fp8_block, what, dev, *at, B, size, block, *tail)
    else:
        _enqueue(lib.gda_attn_decode_paged_fp8_block, what, dev, *at, B, max_pages, size, pages, block, *tail)
    return out


def gda_attn_decode_fp8_block(q_sig, q_noise, k_sig_cache, k_noise_cache, v_cache, k_sig_scale, k_noise_scale, v_scale,
                              cache_lens, lam, lambda_init: float, *, eps: float = 1e-5, out=None, workspace=None):
    """bf16 decode over 8-bit caches with a scale for each block of tokens and head: cached value = code * scale.

    Caches [B, Lcap, heads, dim] float8_e4m3fn (or uint8), scales [B, Lcap /
    block, heads] float32, as ``gda_cache_append_fp8_block`` writes them.  A
    cache length of 0 gives a zero row.
    """
    return _decode_fp8_block(q_sig, q_noise, (k_sig_cache, k_noise_cache, v_cache), (k_sig_scale, k_noise_scale, v_scale),
                             None, None, cache_lens, lam, lambda_init, eps, out, workspace)


def gda_attn_decode_paged_fp8_block(q_sig, q_noise, k_sig_pool, k_noise_pool, v_pool, k_sig_scale, k_noise_scale,
                                    v_scale, block_table, cache_lens, lam, lambda_init: float, *, eps: float = 1e-5,
                                    out=None, workspace=None):
    """``gda_attn_decode_fp8_block`` over page pools [num_pages, page_size, heads, dim], scales [num_pages, page_size /
    block, heads] and a block table [B, max_pages] int32 (position j of sequence b is row j % page_size of page
    block_table[b, j // page_size])."""
    if not isinstance(block_table, torch.Tensor):
        raise TypeError("block_table must be a torch.Tensor")
    return _decode_fp8_block(q_sig, q_noise, (k_sig_pool, k_noise_pool, v_pool), (k_sig_scale, k_noise_scale, v_scale),
                             block_table, None, cache_lens, lam, lambda_init, eps, out, workspace)


def gda_attn_decode_sparse_fp8_block(q_sig, q_noise, k_sig_pool, k_noise_pool, v_pool, k_sig_scale, k_noise_scale,
                                     v_scale, block_list, block_count, cache_lens, lam, lambda_init: float, *,
                                     block_table=None, eps: float = 1e-5, out=None, workspace=None):
    """The decode over listed blocks only: block_list [B, h_n, keep] and block_count [B] int32 as ``gda_block_select``
    gives them (a block counts as often as it is listed, negative entries are passed over).

    Page pools and ``block_table`` as in ``gda_attn_decode_paged_fp8_block``, or contiguous caches without one.  Both
    softmax maps are normalised over the listed positions; a row without any is zero.
    """
    return _decode_fp8_block(q_sig, q_noise, (k_sig_pool, k_noise_pool, v_pool), (k_sig_scale, k_noise_scale, v_scale),
                             block_table, (block_list, block_count), cache_lens, lam, lambda_init, eps, out, workspace)


def gda_device_error(clear: bool = True) -> int:
    """Device error word of the current device (synchronises it); see include/gda.h."""
    rc = _load().gda_device_error(int(bool(clear)))
    if rc < 0:
        raise GDAError(rc, "gda_device_error")
    return rc

