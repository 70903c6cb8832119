"""Softmax weights of the decode over a 4-bit cache keep the digits of a float32 sum.

Tolerance.  With S the sum of absolute terms of a row's largest score (in
units of the exponent of 2), a score is off by less than 2^-20 (1 + S): its
products are exact, a dozen float32 sums and products follow.  exp2, the sums
of the weights and of the values and the norm add less than 2^-20 together.
So a weight is off by 2^-19 (1 + S) of itself, and an output element by as
much of mag, the sum of its absolute terms; the norm's factor by the row's
share of that, the bf16 result by half a step, 2^-8.  Below 2^-18 of its map's
largest, a weight is held to 2^-40 of that largest instead (two f16 numbers,
the steps of whose smallest are 2^-24 where the largest is 2^15).
"""
import math

import numpy as np
import pytest
import torch

import grouped_differential_attention_gb300 as gda
from oracle import ref_serving as R
from test_gpu_decode_fp4 import LAM0, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_differential_attention_gb300 import build
    build.build()


def held(c, b, n):
    """The float64 rows [n, heads, dim] of the three cached tensors of sequence b."""
    grid = torch.tensor(np.concatenate([R.E2M1, -R.E2M1]), device="cuda")
    out = []
    for code, block, s in zip(c["pools"], c["blocks"], c["scales"]):
        if c["table"] is None:
            code, block = code[b], block[b]
        else:
            used = c["table"][b, :-(-n // code.shape[1])].long()
            code, block = (t[used].flatten(0, 1) for t in (code, block))
        u = torch.stack((code[:n] & 15, code[:n] >> 4), -1).flatten(-2).long()
        out.append(grid[u] * block[:n].view(torch.float8_e4m3fn).double().repeat_interleave(16, -1) * s.double()[:, None])
    return out


def check(got, c, eps):
    hs, hn, d = c["q1"].shape[1], c["q2"].shape[1], c["q1"].shape[2]
    lam = c["lam"].double()[:, None]
    rms = lambda t: (t * t).mean(-1, keepdim=True).sqrt()
    for b, n in enumerate(c["lens"].tolist()):
        k1, k2, v = held(c, b, n)
        maps = []
        for q, k in ((c["q1"][b].double(), k1), (c["q2"][b].double(), k2)):
            a = torch.softmax(torch.einsum("hd,jhd->hj", q, k) / d ** 0.5, -1)
            size = torch.einsum("hd,jhd->hj", q.abs(), k.abs()).amax(-1, keepdim=True) / d ** 0.5 / math.log(2)
            maps.append([t.repeat_interleave(hs // t.shape[0], 0) for t in (a, a.amax(-1, keepdim=True), size)])
        (a1, m1, s1), (a2, m2, s2) = maps
        o = torch.einsum("hj,jhe->he", a1 - lam * a2, v)
        f = (1 - LAM0) / torch.sqrt((o * o).mean(-1, keepdim=True) + eps)
        err = (2.0 ** -19 * (1 + torch.maximum(s1, s2)) * torch.einsum("hj,jhe->he", a1 + lam.abs() * a2, v.abs())
               + 2.0 ** -40 * (m1 + lam.abs() * m2) * v.abs().sum(0))
        ref = f * o
        bound = 2.0 ** -8 * ref.abs() + f * (err + o.abs() * rms(err) / rms(o))
        off = (got[b].double() - ref).abs()
        assert (off <= bound).all(), (b, n, int((off > bound).sum()), float((off / bound).max()))


SHAPES = [(6, 2, 64, 128), (8, 4, 128, 128), (4, 1, 128, 256), (5, 5, 64, 64)]


@pytest.mark.parametrize("hs,hn,d,dv", SHAPES)
def test_short_sums(hs, hn, d, dv):
    c = make(8, 208, hs, hn, d, dv, [2, 3, 5, 16, 17, 40, 90, 208], seed=hs + dv, page=16)
    check(run(c), c, 1e-5)


@pytest.mark.parametrize("gap", [20.0, 28.0])
@pytest.mark.parametrize("hs,hn,d,dv", SHAPES)
def test_one_position_far_above_the_others_with_no_value(hs, hn, d, dv, gap):
    """A position that takes nearly all the weight (2^gap times another's) and whose value row is zero, as the first
    token of a text often is: the output is what the small weights of the others say.  eps = 0 keeps the row's size."""
    n, at = 300, 5
    c = make(2, n, hs, hn, d, dv, [n, n - 7], seed=hs + dv)
    g = torch.Generator(device="cuda").manual_seed(3)
    for q in ("q1", "q2"):
        c[q] = (torch.randint(0, 2, c[q].shape, generator=g, device="cuda") * 2 - 1).bfloat16()
    rows = [gap * math.log(2) / math.sqrt(d) * c["q1"].float(), gap * math.log(2) / math.sqrt(d) * c["q2"].float(),
            torch.zeros(2, hs, dv, device="cuda")]
    slots = torch.tensor([at, n + at], dtype=torch.int32, device="cuda")
    gda.gda_cache_append_fp4(*(t.bfloat16() for t in rows), slots, *c["pools"], *c["blocks"], *c["scales"])
    check(run(c, eps=0.0), c, 0.0)


def test_queries_and_scales_at_the_ends_of_their_ranges():
    """Queries of 2^-118 over keys with a head scale of 2^118, and the reverse: the scores are ordinary ones."""
    for up in (118, 125, -110):
        c = make(3, 100, 6, 2, 64, 128, [100, 33, 7], seed=up + 200)
        for q, s in (("q1", 0), ("q2", 1)):
            c[q] = (c[q].double() * 2.0 ** -up).bfloat16()
            c["scales"][s] = (c["scales"][s].double() * 2.0 ** up).float()
        check(run(c), c, 1e-5)
