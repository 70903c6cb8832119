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


# ---- 8-bit cache with a scale for each block of tokens and head ----

def round_e4m3(x):
    """float64 x to the nearest e4m3 value, ties to even, at most 448 in magnitude; NaN stays."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(all="ignore"):
        step = np.exp2(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 3)
        y = np.round(x / step) * step                       # np.round: ties to even
    return np.clip(y, -448.0, 448.0)


def e4m3_byte(values):
    """Bytes of float64 e4m3 values (exact)."""
    return torch.from_numpy(np.asarray(values, dtype=np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def append_fp8_block(x, slots, codes, scale, bounds=None):
    """Rows x [T, heads, n] (bf16 torch) into codes [slots, heads, n] uint8, scale [slots / block, heads] float32 and
    bounds [slots / block, heads, 2, n] int8 (numpy, in place), one block of tokens after the other."""
    x = x.double().numpy()
    slots = np.asarray(slots)
    block = codes.shape[0] // scale.shape[0]
    f32 = np.float32
    rows_of = {}
    for t, s in enumerate(slots):
        if 0 <= s < codes.shape[0]:
            rows_of.setdefault(s // block, []).append(t)
    for blk, rows in rows_of.items():
        first = blk * block
        fresh = first in slots[rows]
        for h in range(x.shape[1]):
            v = x[rows, h]
            amax = float(np.abs(v[np.isfinite(v)]).max(initial=0.0))
            need = 2.0 ** -126
            while amax > 448 * need:
                need *= 2
            old = f32(0) if fresh else scale[blk, h]
            new = max(f32(need), old)
            scale[blk, h] = new
            with np.errstate(all="ignore"):
                shift = f32(1) if fresh else old / new
                if shift != 1:
                    was = e4m3_value(codes[first:first + block, h]).astype(f32)
                    codes[first:first + block, h] = e4m3_byte(round_e4m3((was * shift).astype(f32)))
                y = (v.astype(f32) * (f32(1) / new)).astype(f32)
                limit = min(f32(448), f32(1.875 * 2.0 ** 127) / new)     # the next code would stand for 2^128
                y = np.clip(y, -limit, limit)
            y = round_e4m3(np.where(np.isfinite(v), y, np.nan))
            codes[slots[rows], h] = e4m3_byte(y)
            if bounds is None:
                continue
            top, low = bounds[blk, h].astype(np.float64)
            if fresh:
                top, low = np.full_like(top, -128), np.full_like(low, 127)
            else:
                far = [round_e4m3((f32(4) * b.astype(f32) * shift).astype(f32)) / 4 for b in (top, low)]
                top, low = np.ceil(top * shift), np.floor(low * shift)
                if np.frexp(shift)[0] != 0.5:               # codes are rounded both ways: as far as 4 * bound goes
                    top, low = np.maximum(top, np.ceil(far[0])), np.minimum(low, np.floor(far[1]))
            known = np.isfinite(y)
            top = np.maximum(top, np.where(known, np.ceil(y / 4), -128).max(0))
            low = np.minimum(low, np.where(known, np.floor(y / 4), 127).min(0))
            bounds[blk, h] = np.stack((top, low)).astype(np.int8)


def block_select(q1, q2, bounds, scales, table, lens, block, keep, first, last):
    """(lists [B][hn], counts [B]) in whole numbers and float32, one sequence and noise head at a time.

    bounds, scales: numpy pairs [pages, blocks of a page, heads, ..]; table [B, max_pages] or None."""
    f32 = np.float32
    q = [t.float().numpy() for t in (q1, q2)]
    B, hs, hn = len(lens), q[0].shape[1], q[1].shape[1]
    per = bounds[0].shape[1]
    lists, counts = [], []
    for b in range(B):
        n = -(-int(lens[b]) // block)
        counts.append(min(n, keep))
        at = [(int(table[b, j // per]) if table is not None else b, j % per) for j in range(n)]
        lists.append([])
        for g in range(hn):
            if n <= keep:
                lists[-1].append(list(range(n)))
                continue
            score = np.zeros(n, dtype=f32)
            r = hs // hn
            for i, h in [(0, h) for h in range(g * r, g * r + r)] + [(1, g)]:
                x = q[i][b, h]
                amax = f32(np.abs(x).max())
                if not (np.isfinite(x).all() and amax >= 2.0 ** -100):
                    continue
                q8 = np.rint((x * f32(f32(127) * (f32(1) / amax))).astype(f32)).astype(np.int64)
                v = np.empty(n, dtype=f32)
                for j, place in enumerate(at):
                    hi, lo = bounds[i][place][h].astype(np.int64)
                    ub = int((np.maximum(q8, 0) * hi + np.minimum(q8, 0) * lo).sum())
                    with np.errstate(over="ignore"):
                        v[j] = f32(f32(ub) * scales[i][place][h]) * amax
                if np.isinf(v.max()):
                    continue
                unit = f32(4 / 127 / np.log(2) / np.sqrt(x.size))
                t = np.maximum(((v - v.max()).astype(f32) * unit).astype(f32), f32(-126))
                e = np.floor(t)
                line = 2.0 ** 23 + np.rint((t - e).astype(f32) * 2.0 ** 23).astype(np.float64)
                w = line * 2.0 ** (e.astype(np.float64) - 23)
                total = f32(sum(int(k) for k in np.floor(w * 2.0 ** 40))) * f32(2.0 ** -40)
                score = np.maximum(score, (w.astype(f32) * (f32(1) / total)).astype(f32))
            forced = [j for j in range(n) if j < first or j >= n - last]
            rest = sorted((j for j in range(n) if j not in forced), key=lambda j: (-score[j], j))
            lists[-1].append(sorted(forced + rest[:keep - len(forced)]))
    return lists, counts
