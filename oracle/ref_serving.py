"""Plain 64-bit references of the operators around the attention (test infrastructure only).

* ``norm_rope`` / ``norm_rope_grads``: RMSNorm of every head row and its
  rotation by position, and float64 autograd gradients of it.
* ``block_tables``: block table, slots and positions of a serving step, one
  sequence after the other in plain Python.
* ``quantise_fp4`` / ``dequantise_fp4``: the 4-bit cache format, one element
  at a time in meaning: nearest of the eight e2m1 magnitudes, ties to even.
"""
from __future__ import annotations

import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = 16


def _pair_index(rot: int, interleaved: bool):
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def norm_rope(x, w, positions, inv_freq, eps=1e-5, interleaved=False):
    """One projection x [*tokens, heads, d] with weight row w [d]; float64 torch."""
    x, w = x.double(), w.double()
    ia, ib = _pair_index(2 * inv_freq.numel(), interleaved)
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    t = positions.double()[..., None, None] * inv_freq.double()
    y = n.clone()
    y[..., ia] = n[..., ia] * t.cos() - n[..., ib] * t.sin()
    y[..., ib] = n[..., ib] * t.cos() + n[..., ia] * t.sin()
    return y


def norm_rope_size(x, w, inv_freq, eps=1e-5, interleaved=False):
    """|n_a| + |n_b| of each output's pair (|n| beyond the rotated dims): what its rounding errors scale with."""
    x, w = x.double(), w.double()
    ia, ib = _pair_index(2 * inv_freq.numel(), interleaved)
    n = (x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w).abs()
    size = n.clone()
    size[..., ia] = size[..., ib] = n[..., ia] + n[..., ib]
    return size


def norm_rope_grads(x, w, positions, inv_freq, dy, eps=1e-5, interleaved=False):
    """(dx, dw) by float64 autograd."""
    x = x.double().detach().requires_grad_(True)
    w = w.double().detach().requires_grad_(True)
    y = norm_rope(x, w, positions, inv_freq, eps, interleaved)
    return torch.autograd.grad(y, (x, w), dy.double())


def norm_rope_grad_size(x, w, inv_freq, dy, eps=1e-5, interleaved=False):
    """Sums of the absolute terms of dx (per element) and dw (per dim)."""
    x, w, dy = x.double(), w.double(), dy.double()
    ia, ib = _pair_index(2 * inv_freq.numel(), interleaved)
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    g = dy.abs().clone()
    g[..., ia] = g[..., ib] = dy[..., ia].abs() + dy[..., ib].abs()
    t = g * w.abs()
    dx = r * (t + x.abs() * r * r * (t * x.abs()).mean(-1, keepdim=True))
    return dx, (g * x.abs() * r).flatten(0, -2).sum(0)


def block_tables(lens, new, table, free, count, page_size, num_pages, max_rows):
    """(slot_map, positions, row_starts, lens_out, free_left, table) as Python lists / arrays."""
    table = np.array(table).copy()
    B, max_pages = table.shape
    slots, positions = [-1] * max_rows, [0] * max_rows
    starts, lens_out = [0], []
    short = False                       # the stack has failed a sequence: nobody gets a page any more
    for b in range(B):
        have, add = int(lens[b]), int(new[b])
        n, r0 = max(add, 0), starts[-1]
        starts.append(r0 + n)
        ok = have >= 0 and add >= 0 and have + n <= max_pages * page_size and r0 + n <= max_rows
        if ok:
            held, top = -(-have // page_size), -(-(have + n) // page_size)
            if top > held and (short or top - held > count):
                short, ok = True, False
        if ok:
            for j in range(held, top):
                count -= 1
                table[b, j] = free[count]
            for i in range(n):
                pos = have + i
                page = int(table[b, pos // page_size])
                if 0 <= page < num_pages:
                    slots[r0 + i], positions[r0 + i] = page * page_size + pos % page_size, pos
        lens_out.append(have + n if ok else have)
    return slots, positions, starts, lens_out, count, table


def e4m3_value(byte):
    return torch.as_tensor(byte, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()


def quantise_fp4(x, scale):
    """(codes, blocks) of x [rows, heads, n] (bf16 torch): unpacked codes uint8 [rows, heads, n], bytes [.., n/16]."""
    x = x.float().numpy()
    rows, heads, n = x.shape
    g = np.asarray(scale, dtype=np.float32)[None, :, None]
    xb = x.reshape(rows, heads, n // BLOCK, BLOCK)
    with np.errstate(all="ignore"):
        amax = np.abs(xb).max(-1)
        t = (amax / (np.float32(6) * g)).astype(np.float32)
        s8 = torch.from_numpy(np.minimum(t, np.float32(448))).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        s8 = np.where(np.isnan(t), np.uint8(0x7F), s8)
        s = e4m3_value(s8).astype(np.float32)
        r = np.where(s > 0, np.float32(1) / (s * g).astype(np.float32), np.float32(0)).astype(np.float32)
        y = (xb * r[..., None]).astype(np.float32).astype(np.float64)
        y = np.where((r > 0)[..., None], y, 0.0)
        off = np.abs(np.minimum(np.abs(y), 6.0)[..., None] - E2M1)
        near = off == off.min(-1, keepdims=True)
        # of two as near, the even code
        code = np.where(near, np.where(np.arange(8) % 2 == 0, np.arange(8), np.arange(8) + 100), 1000).argmin(-1)
        code = code + 8 * (np.signbit(y) & (r > 0)[..., None])
    return code.reshape(rows, heads, n).astype(np.uint8), s8


def dequantise_fp4(codes, blocks, scale):
    """float64 values of unpacked codes [..., heads, n] and block bytes [..., heads, n / 16]."""
    codes = np.asarray(codes)
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.repeat(e4m3_value(np.asarray(blocks)), BLOCK, axis=-1)
    return v * s * np.asarray(scale, dtype=np.float64)[:, None]


def pack(codes):
    codes = np.asarray(codes)
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    packed = np.asarray(packed)
    out = np.empty(packed.shape[:-1] + (2 * packed.shape[-1],), dtype=np.uint8)
    out[..., 0::2], out[..., 1::2] = packed & 15, packed >> 4
    return out
