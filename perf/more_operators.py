"""Calls to measure: an 8-bit cache with a scale for each block of tokens, and the attention that reads it.

Five operators, as a serving loop runs them:

* ``cache``: rows of K and V quantised into the cache as they are written, with
  the bounds of the keys of every block, and rows read back as bf16
  (``gda_cache_append_fp8_block``, ``gda_cache_read_fp8_block``);
* ``decode``: one query token per sequence over all of that cache, contiguous or
  paged (``gda_attn_decode_fp8_block``, ``gda_attn_decode_paged_fp8_block``);
* ``select``: the blocks of each sequence and noise head that a score over the
  bounds keeps: the largest share that the block has, by the bound on its
  logits, in one of the group's heads (``gda_block_select``);
* ``sparse``: one query token per sequence over listed blocks only
  (``gda_attn_decode_sparse_fp8_block``).

The cache: e4m3 codes [pages, page, heads, dim], a float32 scale for each block
of tokens and head [pages, page / block, heads]; value = code * scale.  With
``own`` false, ``run`` computes the same from elementary torch operations.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
LAMBDA_INIT = 0.8
TOP = 448.0            # the largest e4m3 magnitude


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # a decode step: each of 64 sequences writes one row somewhere in a block that has rows already
        {"name": "cache_step_b64", "op": "cache", "B": 64, "n": 1, "held": 256, "hs": 12, "hn": 4, "d": 64, "dv": 128,
         "page": 64, "block": 64, "back": "new", "mixed": False},
        # a prompt chunk of 8192 rows, whole blocks
        {"name": "cache_chunk_t8192", "op": "cache", "B": 1, "n": 8192, "held": 0, "hs": 12, "hn": 4, "d": 64,
         "dv": 128, "page": 64, "block": 64, "back": "new", "mixed": False},
        # ragged pieces that continue blocks, wide heads, small blocks, all rows of the blocks read back
        {"name": "cache_ragged_d128_dv256", "op": "cache", "B": 9, "n": 227, "held": 61, "hs": 16, "hn": 4, "d": 128,
         "dv": 256, "page": 48, "block": 16, "back": "all", "mixed": False},
        # a few short conversations, small pages: latency
        {"name": "decode_b4_short", "op": "decode", "B": 4, "lo": 37, "hi": 600, "hs": 6, "hn": 2, "d": 64, "dv": 128,
         "page": 16, "block": 16},
        # the serving batch: 64 sequences of 4096 to 8192 positions, contiguous caches
        {"name": "decode_b64_len8192", "op": "decode", "B": 64, "lo": 4096, "hi": 8192, "hs": 12, "hn": 4, "d": 64,
         "dv": 128, "page": 0, "block": 64},
        # wide heads, 4:1 groups, pages, lengths from one token on
        {"name": "decode_b16_d128_dv256", "op": "decode", "B": 16, "lo": 1, "hi": 8191, "hs": 16, "hn": 4, "d": 128,
         "dv": 256, "page": 64, "block": 32},
        # one long document, 24 + 8 heads, large pages and blocks
        {"name": "decode_b1_len131072", "op": "decode", "B": 1, "lo": 131072, "hi": 131072, "hs": 24, "hn": 8, "d": 64,
         "dv": 128, "page": 128, "block": 128},
        # the serving batch's blocks: 16 of up to 128
        {"name": "select_b64_len8192", "op": "select", "B": 64, "lo": 4096, "hi": 8192, "hs": 12, "hn": 4, "d": 64,
         "page": 64, "block": 64, "keep": 16, "first": 1, "last": 1},
        # the long document's: 64 of 2048
        {"name": "select_b1_len131072", "op": "select", "B": 1, "lo": 131072, "hi": 131072, "hs": 24, "hn": 8, "d": 64,
         "page": 128, "block": 64, "keep": 64, "first": 1, "last": 2},
        # 1024 positions of each sequence of the serving batch
        {"name": "sparse_b64_keep16", "op": "sparse", "B": 64, "lo": 4096, "hi": 8192, "hs": 12, "hn": 4, "d": 64,
         "dv": 128, "page": 64, "block": 64, "keep": 16},
        # 4096 positions of the long document
        {"name": "sparse_b1_len131072", "op": "sparse", "B": 1, "lo": 131072, "hi": 131072, "hs": 24, "hn": 8, "d": 64,
         "dv": 128, "page": 128, "block": 64, "keep": 64},
        # wide heads, small blocks, some sequences shorter than what is kept
        {"name": "sparse_b16_d128_dv256", "op": "sparse", "B": 16, "lo": 1, "hi": 8191, "hs": 16, "hn": 4, "d": 128,
         "dv": 256, "page": 0, "block": 16, "keep": 100},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["cache", "decode", "decode", "select", "sparse", "sparse"])
    r = rng.choice([1, 2, 3, 3, 4, 5, 6])
    hn = rng.choice([1, 2, 3, 4, 4, 8]) if r <= 3 else rng.choice([1, 2, 4])
    hs, d, dv = r * hn, rng.choice([64, 64, 128]), rng.choice([128, 128, 64, 256])
    block = rng.choice([16, 32, 64, 64, 128])
    page = block * rng.choice([1, 1, 2, 3, 4])
    row = hs * (d + dv) + hn * d
    if op == "cache":
        T = _log(rng, 1, 2.0e7 / row)
        B = rng.choice([1, T, min(T, _log(rng, 1, 64))])
        return {"op": op, "B": B, "n": max(1, T // B), "held": rng.choice([0, _log(rng, 1, 300)]), "hs": hs, "hn": hn,
                "d": d, "dv": dv, "page": page, "block": block, "back": rng.choice(["new", "all"]) if T > B else "new",
                "mixed": rng.random() < 0.25}
    total = 10 ** rng.uniform(math.log10(64 * row), 8.95) / row    # positions of the batch, at most those of the listed
    B = min(_log(rng, 1, 128), max(1, int(total)))
    hi = max(1, min(131072, int(total / B)))
    c = {"op": op, "B": B, "lo": rng.choice([hi, max(1, hi // 2), 1, 0]), "hi": hi, "hs": hs, "hn": hn, "d": d,
         "page": rng.choice([0, page]), "block": block}
    if op == "select":
        keep = _log(rng, 1, max(2, -(-hi // block)))
        first = rng.choice([0, 1, min(2, keep)])
        return c | {"keep": keep, "first": first, "last": rng.choice([0, min(1, keep - first)])}
    if op == "sparse":
        return c | {"dv": dv, "keep": _log(rng, 1, max(1, hi // block))}
    return c | {"dv": dv}


# ------------------------------------------------------------------ inputs --

def _lengths(c):
    """Lengths spread evenly over [lo, hi]: their sum does not depend on the seed."""
    return torch.linspace(c["lo"], c["hi"], c["B"], dtype=torch.float64).round().to(torch.int32)


def _geometry(c):
    """Rows of a page (of a sequence, in contiguous caches) and pages of a sequence."""
    size = c["page"] or -(-c["hi"] // c["block"]) * c["block"]
    return size, -(-c["hi"] // size)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(seed)
    hs, hn, d, bl = c["hs"], c["hn"], c["d"], c["block"]
    B = c["B"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device=DEV)

    if c["op"] == "cache":
        dv, n, ps = c["dv"], c["n"], c["page"]
        start = whole(0, c["held"] + 1, B)                         # positions that a sequence holds before the call
        per = -(-(c["held"] + n) // ps)
        pages = B * per + 3
        table = torch.randperm(pages, generator=g, device=DEV)[:B * per].view(B, per)

        def slots_of(lo, hi):                                      # of positions lo <= p < hi, sequence after sequence
            p = torch.arange(per * ps, device=DEV)[None].expand(B, -1)
            b, p = torch.nonzero((p >= lo[:, None]) & (p < hi[:, None]), as_tuple=True)
            return (table[b, p // ps] * ps + p % ps).to(torch.int32)

        def rows(T):
            loud = torch.exp(0.5 * normal(T, 1, 1))                # tokens differ in size: some make a block's scale grow
            vproj = (normal(T, hs * dv + 64) * loud[:, 0]).bfloat16()   # values come out of the projection, rows apart
            return ((normal(T, hs, d) * loud).bfloat16(), (normal(T, hn, d) * loud).bfloat16(),
                    vproj[:, :hs * dv].unflatten(-1, (hs, dv)))

        dims = ((hs, d), (hn, d), (hs, dv))
        s = c | {"pools": [torch.zeros(pages, ps, h, m, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
                           for h, m in dims],
                 "scales": [torch.zeros(pages, ps // bl, h, device=DEV) for h, _ in dims],
                 "bounds": [torch.zeros(pages, ps // bl, h, 2, d, dtype=torch.int8, device=DEV) for h in (hs, hn)]}
        held = slots_of(start * 0, start)
        if held.numel():
            _append(s, rows(held.numel()), held)
        slots = slots_of(start, start + n)
        if c["mixed"]:
            slots = slots[torch.randperm(slots.numel(), generator=g, device=DEV)]
        back = slots
        if c["back"] == "all":                                     # the rows before them in their blocks too, -1 for none
            back = torch.full((B * (n + bl - 1),), -1, dtype=torch.int32, device=DEV)
            every = slots_of(start // bl * bl, start + n)
            back[:every.numel()] = every
        return s | {"rows": rows(slots.numel()), "slots": slots.contiguous(), "read": back.contiguous()}

    size, mp = _geometry(c)
    lens = _lengths(c).to(DEV)[torch.randperm(B, generator=g, device=DEV)].contiguous()
    pages = B * mp + (3 if c["page"] else 0)
    table = torch.randperm(pages, generator=g, device=DEV)[:B * mp].view(B, mp).to(torch.int32).contiguous()
    s = c | {"q1": (normal(B, hs, d) * torch.exp(0.3 * normal(B, hs, 1))).bfloat16(), "q2": normal(B, hn, d).bfloat16(),
             "lens": lens, "table": table if c["page"] else None}
    if c["op"] == "select":
        s["bounds"], s["scales"] = [], []
        for h in (hs, hn):                                         # of the rows of a block: their middle and their reach
            middle, reach = 15 * normal(pages, size // bl, h, d), 40 + 8 * normal(pages, size // bl, h, d).abs()
            s["bounds"].append(torch.stack((middle + reach, middle - reach), 3).round().clamp(-112, 112).to(torch.int8))
            s["scales"].append(torch.exp2(whole(-8, -5, pages, size // bl, h).float()))
        return s
    dv = c["dv"]
    s["pools"], s["scales"] = [], []
    for h, m in ((hs, d), (hn, d), (hs, dv)):                      # rows as a model writes them, put into 8 bits
        code = torch.empty(pages, size // bl, bl, h, m, dtype=torch.uint8, device=DEV)
        scale = torch.empty(pages, size // bl, h, device=DEV)
        step = max(1, (1 << 26) // (size * h * m))
        for a in range(0, pages, step):
            b = min(pages, a + step)
            x = (normal(b - a, size // bl, bl, h, m) * torch.exp(0.3 * normal(b - a, size // bl, 1, h, 1))).bfloat16().float()
            scale[a:b] = _scale_of(x.abs().amax((2, 4)))
            code[a:b] = (x / scale[a:b, :, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        s["pools"].append(code.view(pages, size, h, m).view(torch.float8_e4m3fn))
        s["scales"].append(scale)
    s["lam"] = 0.2 + 0.6 * torch.rand(hs, generator=g, device=DEV)
    if c["op"] == "sparse":                                        # any blocks of a sequence, the last among them
        most = -(-c["hi"] // bl)
        count = (lens.long() + bl - 1) // bl
        rank = torch.rand(B, hn, most, generator=g, device=DEV)
        at = torch.arange(most, device=DEV)[None, None]
        rank = torch.where(at == count[:, None, None] - 1, -1.0, torch.where(at < count[:, None, None], rank, 2.0))
        keep = c["keep"]
        pick = rank.argsort(-1)[..., :keep]
        if pick.shape[-1] < keep:
            pick = torch.nn.functional.pad(pick, (0, keep - pick.shape[-1]), value=most)
        kept = count.clamp(max=keep)
        pick = torch.where(torch.arange(keep, device=DEV) < kept[:, None, None], pick, most).sort(-1).values
        s["blocks"] = torch.where(pick < most, pick, -1).to(torch.int32).contiguous()
        s["counts"] = kept.to(torch.int32)
    return s


# -------------------------------------------------------------- plain forms --

def _scale_of(amax):
    """The least power of two s >= 2^-126 with amax <= 448 s."""
    m, e = torch.frexp(amax)                                       # amax = 2 m 2^(e - 1), 1 <= 2 m < 2; 448 = 1.75 2^8
    k = torch.where(amax > 0, e - 9 + (2 * m > 1.75), -126).clamp(min=-126)
    return ((k.int() + 127) << 23).view(torch.float32)


def _append(s, rows, slots):
    """Rows of K and V into the blocks of their slots, in place; bounds of the keys beside them."""
    bl = s["block"]
    at = slots.long()
    blk = at // bl
    touched, where = torch.unique(blk, return_inverse=True)
    fresh = torch.zeros(touched.numel(), dtype=torch.bool, device=DEV)
    fresh[where[at % bl == 0]] = True                              # a call that writes a block's first row starts it anew
    for i, x in enumerate(rows):
        x = x.float()
        h, n = x.shape[1:]
        codes = s["pools"][i].view(torch.uint8).view(-1, bl, h, n)
        scales = s["scales"][i].view(-1, h)
        finite = torch.where(torch.isfinite(x), x, 0.0)
        amax = torch.zeros(touched.numel(), h, device=DEV).index_reduce_(0, where, finite.abs().amax(-1), "amax")
        old = torch.where(fresh[:, None], 0.0, scales[touched])
        new = torch.maximum(old, _scale_of(amax))
        shift = torch.where(fresh[:, None], 1.0, old / new)        # rows already there
        grown = torch.nonzero((shift != 1).any(1))[:, 0]
        was = codes[touched[grown]].view(torch.float8_e4m3fn).float()
        codes[touched[grown]] = (was * shift[grown, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        code = (x * (1.0 / new)[where, :, None])
        code = torch.where(torch.isfinite(x), code, math.nan).to(torch.float8_e4m3fn)
        codes.view(-1, h, n)[at] = code.view(torch.uint8)
        scales[touched] = new
        if i == 2:
            continue
        v = code.float() / 4                                       # bounds: whole fours of the scale, outwards
        known = torch.isfinite(v)
        up = torch.where(known, v.ceil(), -128.0)
        down = torch.where(known, v.floor(), 127.0)
        bounds = s["bounds"][i].view(-1, h, 2, n)
        b = bounds[touched].float()
        f = fresh[:, None, None]
        top = torch.where(f, -128.0, (b[:, :, 0] * shift[..., None]).ceil())
        low = torch.where(f, 127.0, (b[:, :, 1] * shift[..., None]).floor())
        top = top.index_reduce(0, where, up, "amax")
        low = low.index_reduce(0, where, down, "amin")
        bounds[touched] = torch.stack((top, low), 2).to(torch.int8)


def _plain_cache(s):
    _append(s, s["rows"], s["slots"])
    live = (s["read"] >= 0)[:, None, None]
    at = s["read"].long().clamp(min=0)
    back = []
    for code, scale in zip(s["pools"], s["scales"]):
        h, n = code.shape[2:]
        v = code.view(torch.uint8).view(-1, h, n)[at].view(torch.float8_e4m3fn).float()
        back.append(torch.where(live, v * scale.view(-1, h)[at // s["block"]][..., None], 0.0).bfloat16())
    return back + s["scales"] + s["bounds"]


def _rows(s, i):
    """The cache's tensor i as float32 [B, positions, heads, n], pages in the sequence's order."""
    code, scale = s["pools"][i].view(torch.uint8), s["scales"][i]
    if s["table"] is not None:
        t = s["table"].long()
        code, scale = code[t].flatten(1, 2), scale[t].flatten(1, 2)
    return code.view(torch.float8_e4m3fn).float() * scale.repeat_interleave(s["block"], 1)[..., None]


def _softmax(x, seen):
    x = x.masked_fill(~seen, -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-3e38))
    return e / e.sum(-1, keepdim=True).clamp(min=1e-38)


def _norm(o):
    return ((1.0 - LAMBDA_INIT) * o * torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS)).bfloat16()


def _plain_decode(s):
    k1 = _rows(s, 0)
    seen = (torch.arange(k1.shape[1], device=DEV) < s["lens"][:, None])[:, None]
    a1 = _softmax(torch.einsum("bhd,bjhd->bhj", s["q1"].float(), k1) / math.sqrt(s["d"]), seen)
    del k1
    a2 = _softmax(torch.einsum("bhd,bjhd->bhj", s["q2"].float(), _rows(s, 1)) / math.sqrt(s["d"]), seen)
    w = a1 - s["lam"][None, :, None] * a2.repeat_interleave(s["hs"] // s["hn"], 1)
    return _norm(torch.einsum("bhj,bjhe->bhe", w, _rows(s, 2)))


def _by_block(s, t):
    """A tensor [pages, blocks of a page, ...] as [B, blocks of a sequence, ...]."""
    return t[s["table"].long()].flatten(1, 2) if s["table"] is not None else t


def _plain_select(s):
    B, hs, hn, bl, keep = s["B"], s["hs"], s["hn"], s["block"], s["keep"]
    most = -(-s["hi"] // bl)
    count = (s["lens"].long() + bl - 1) // bl
    there = torch.arange(most, device=DEV)[None] < count[:, None]                     # [B, most]
    score = torch.zeros(B, hn, most, device=DEV)
    unit = 4 / 127 / math.log(2) / math.sqrt(s["d"])                                  # from bounds to powers of two
    for q, bounds, scale, r in ((s["q1"], s["bounds"][0], s["scales"][0], hs // hn),
                                (s["q2"], s["bounds"][1], s["scales"][1], 1)):
        f = q.float()
        amax = f.abs().amax(-1)
        ok = torch.isfinite(amax) & (amax >= 2.0 ** -100)                             # others take no part
        q8 = torch.round(f * torch.where(ok, 127.0 / amax, 0.0)[..., None])[:, None]  # [B, 1, h, d]
        b = _by_block(s, bounds)[:, :most].float()
        dot = (torch.where(q8 > 0, q8, 0.0) * b[..., 0, :] + torch.where(q8 < 0, q8, 0.0) * b[..., 1, :]).sum(-1)
        x = dot * _by_block(s, scale)[:, :most] * amax[:, None]                       # whole numbers below 2^24: exact
        x = x.masked_fill(~there[..., None], -math.inf)
        t = ((x - x.amax(1, keepdim=True).clamp(min=-3e38)) * unit).clamp(min=-126.0)
        e = t.floor()                                                                 # 2^t, a straight line from e to e + 1
        w = (((e.int() + 127) << 23) + torch.round((t - e) * 2.0 ** 23).int()).view(torch.float32)
        w = torch.where(there[..., None] & ok[:, None], w, 0.0)
        total = (w * 2.0 ** 40).long().sum(1, keepdim=True).float() * 2.0 ** -40      # whole numbers: in any order
        share = w * torch.where(total > 0, 1.0 / total, 0.0)
        score = torch.maximum(score, share.view(B, most, hn, r).amax(-1).transpose(1, 2))
    at = torch.arange(most, device=DEV)[None]
    forced = there & ((at < s["first"]) | (at >= count[:, None] - s["last"]))
    score = score.masked_fill(forced[:, None], math.inf).masked_fill(~there[:, None], -1.0)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :keep]
    if order.shape[-1] < keep:
        order = torch.nn.functional.pad(order, (0, keep - order.shape[-1]), value=most)
    kept = count.clamp(max=keep)
    order = torch.where(torch.arange(keep, device=DEV) < kept[:, None, None], order, most).sort(-1).values
    return [torch.where(order < most, order, -1).int(), kept.int()]


def _plain_sparse(s):
    B, hs, hn, d, dv, bl = s["B"], s["hs"], s["hn"], s["d"], s["dv"], s["block"]
    r = hs // hn
    ids = s["blocks"].long()                                                          # [B, hn, keep]
    ok = (torch.arange(s["keep"], device=DEV) < s["counts"][:, None, None]) & (ids >= 0)
    pos = ids.clamp(min=0)[..., None] * bl + torch.arange(bl, device=DEV)
    seen = (ok[..., None] & (pos < s["lens"][:, None, None, None])).flatten(2)        # [B, hn, S]
    size, mp = _geometry(s)
    pos = pos.flatten(2).clamp(max=size * mp - 1)
    b = torch.arange(B, device=DEV)[:, None, None]
    page = s["table"].long()[b, pos // size] if s["table"] is not None else b.expand_as(pos)
    row = page * size + pos % size
    g = torch.arange(hn, device=DEV)[None, :, None]

    def rows(i, n, m):                                                                # [B, hn, S, n, m]
        code = s["pools"][i].view(torch.uint8).view(-1, hn, n, m)[row, g].view(torch.float8_e4m3fn).float()
        return code * s["scales"][i].view(-1, hn, n)[row // bl, g][..., None]

    x1 = torch.einsum("bgrd,bgjrd->bgrj", s["q1"].float().view(B, hn, r, d), rows(0, r, d)) / math.sqrt(d)
    x2 = torch.einsum("bgd,bgjd->bgj", s["q2"].float(), rows(1, 1, d)[:, :, :, 0]) / math.sqrt(d)
    w = _softmax(x1, seen[:, :, None]) - s["lam"].view(1, hn, r, 1) * _softmax(x2, seen)[:, :, None]
    return _norm(torch.einsum("bgrj,bgjre->bgre", w, rows(2, r, dv)).flatten(1, 2))


def run(state):
    s = state
    if own:
        import grouped_differential_attention_gb300 as gda
        if s["op"] == "cache":
            cache = (*s["pools"], *s["scales"])
            gda.gda_cache_append_fp8_block(*s["rows"], s["slots"], *cache, k_sig_bounds=s["bounds"][0],
                                           k_noise_bounds=s["bounds"][1])
            return [*gda.gda_cache_read_fp8_block(s["read"], *cache), *s["scales"], *s["bounds"]]
        if s["op"] == "select":
            return list(gda.gda_block_select(s["q1"], s["q2"], *s["bounds"], *s["scales"], s["lens"], s["block"],
                                             s["keep"], block_table=s["table"], first=s["first"], last=s["last"]))
        if s["op"] == "sparse":
            return gda.gda_attn_decode_sparse_fp8_block(s["q1"], s["q2"], *s["pools"], *s["scales"], s["blocks"],
                                                        s["counts"], s["lens"], s["lam"], LAMBDA_INIT,
                                                        block_table=s["table"], eps=EPS)
        if s["table"] is not None:
            return gda.gda_attn_decode_paged_fp8_block(s["q1"], s["q2"], *s["pools"], *s["scales"], s["table"],
                                                       s["lens"], s["lam"], LAMBDA_INIT, eps=EPS)
        return gda.gda_attn_decode_fp8_block(s["q1"], s["q2"], *s["pools"], *s["scales"], s["lens"], s["lam"],
                                             LAMBDA_INIT, eps=EPS)
    return {"cache": _plain_cache, "decode": _plain_decode, "select": _plain_select, "sparse": _plain_sparse}[s["op"]](s)


# -------------------------------------------------------------------- work --

def work(case):
    c = case
    hs, hn, d, bl = c["hs"], c["hn"], c["d"], c["block"]
    if c["op"] == "cache":
        T, row = c["B"] * c["n"], hs * (d + c["dv"]) + hn * d
        back = T if c["back"] == "new" else T + c["B"] * (bl - 1)
        blocks = max(c["B"], T // bl)
        return {"bytes": T * row * 3 + back * row * 3 + 4 * (T + back) + blocks * (4 * (2 * hs + hn) + 2 * d * (hs + hn)),
                "flops": 4 * T * row}
    lens = _lengths(c).long()
    if c["op"] == "select":
        blocks = int(((lens + bl - 1) // bl).sum())
        return {"bytes": blocks * (hs + hn) * (2 * d + 4) + c["B"] * ((hs + hn) * d * 2 + hn * c["keep"] * 4),
                "flops": 4 * blocks * (hs + hn) * d}
    row = hs * (d + c["dv"]) + hn * d
    total = int((lens if c["op"] == "decode" else lens.clamp(max=c["keep"] * bl)).sum())
    return {"bytes": total * (row + 4 * (2 * hs + hn) / bl) + c["B"] * (hs * d + hn * d + hs * c["dv"]) * 2,
            "flops": total * (2 * (hs + hn) * d + 4 * hs * c["dv"])}


# ------------------------------------------------------ from the definition --

def _nearest_e4m3(x):
    """x (float64, at most 448 in magnitude) to the nearest e4m3 value, ties to the even one: steps of 2^-9 up to
    2^-6, an eighth of the power of two below beyond."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_cache(s):
    # before the call: the values that the rows to read hold
    at, slots, bl = s["read"].long().clamp(min=0), s["slots"].long(), s["block"]
    out, scales = [], []
    first = set((slots[slots % bl == 0] // bl).tolist())
    for i, x in enumerate(s["rows"]):
        h, n = x.shape[1:]
        x = x.double()
        scale = s["scales"][i].double().view(-1, h).clone()
        before = scale.clone()
        for b in first:
            scale[b] = 0
        amax = x.abs().amax(-1)                                                       # [T, h]
        need = torch.full_like(amax, 2.0 ** -126)
        for k in range(-125, 121):
            need = torch.where(amax > TOP * need, 2.0 ** k, need)
        scale.scatter_reduce_(0, (slots // bl)[:, None].expand(-1, h), need, "amax")
        value = s["pools"][i].float().double().view(-1, h, n)
        rows = value[at] * (before / scale).nan_to_num(1.0)[at // bl][..., None]
        rows = _nearest_e4m3(rows)
        place = torch.full((value.shape[0],), -1, device=DEV)
        place[slots] = torch.arange(slots.numel(), device=DEV)
        new = place[at]
        fresh = _nearest_e4m3(x / scale[slots // bl][..., None])[new.clamp(min=0)]
        rows = torch.where((new >= 0)[:, None, None], fresh, rows) * scale[at // bl][..., None]
        out.append(torch.where((s["read"] >= 0)[:, None, None], rows, 0.0))
        scales.append(scale.view(s["scales"][i].shape))
    return out + scales + [None, None]


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "select":
        return None
    if s["op"] == "cache":
        return _exact_cache(s)
    hs, hn, d, dv, bl, B = s["hs"], s["hn"], s["d"], s["dv"], s["block"], s["B"]
    r = hs // hn
    size, _ = _geometry(s)
    outs = torch.zeros(B, hs, dv, dtype=torch.float64, device=DEV)
    for b in range(B):
        n = int(s["lens"][b])
        if n == 0:
            continue
        p = torch.arange(n, device=DEV)
        page = s["table"][b].long()[p // size] if s["table"] is not None else torch.full_like(p, b)
        for g in range(hn):
            at, rows = p, page * size + p % size
            if s["op"] == "sparse":
                kept = s["blocks"][b, g, :int(s["counts"][b])].long()
                at = at[torch.isin(p // bl, kept)]
                rows = rows[at]

            def values(i, h):
                code = s["pools"][i].view(torch.uint8).flatten(0, 1)[rows, h].view(torch.float8_e4m3fn).float().double()
                return code * s["scales"][i].double().flatten(0, 1)[rows // bl, h][:, None]

            x2 = (values(1, g) @ s["q2"][b, g].double()) / math.sqrt(d)
            p2 = torch.exp(x2 - torch.logsumexp(x2, 0))
            for h in range(g * r, g * r + r):
                x1 = (values(0, h) @ s["q1"][b, h].double()) / math.sqrt(d)
                w = torch.exp(x1 - torch.logsumexp(x1, 0)) - s["lam"][h].double() * p2
                outs[b, h] = w @ values(2, h)
    return (1.0 - LAMBDA_INIT) * outs / (outs.square().mean(-1, keepdim=True) + EPS).sqrt()
