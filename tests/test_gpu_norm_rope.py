"""gda_qk_norm_rope and its gradients on the GPU against float64.

Tolerances, in units of s = |n_a| + |n_b| (the normed pair behind an output):
float32 error of the mean (a chain of 8 fused adds and 4 shuffled ones, halved
by the root: 2^-21.4), rsqrt and the products (2^-22), the angle (2^-22.4 rad
below 2^24, 2^-21.7 above) and sincospi (2^-23): below 2^-20 s; taken as 2^-19.
A bf16 result is off by another half step, 2^-8 of its value (2^-24 float32,
inside the first term).  Gradients go through two means: 2^-18 of the sum of
their absolute terms.
"""
import pytest
import torch

import grouped_differential_attention_gb300 as gda
from oracle import ref_serving as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def device_error_word_stays_clear():
    from grouped_differential_attention_gb300 import build
    build.build()
    gda.gda_device_error(clear=True)
    yield
    assert gda.gda_device_error(clear=True) == 0


def make(lead, hs, hn, d, rot, dtype, far=0, theta=10000.0, seed=0, fused=False):
    g = torch.Generator().manual_seed(seed)
    heads = (hs, hs, hn, hn)
    if fused:       # slices of one projection, values behind them
        proj = (1.5 * torch.randn(*lead, sum(heads) * d + hs * 128, generator=g)).to(dtype).cuda()
        x, at = [], 0
        for h in heads:
            x.append(proj[..., at:at + h * d].unflatten(-1, (h, d)))
            at += h * d
    else:
        x = [(1.5 * torch.randn(*lead, h, d, generator=g)).to(dtype).cuda() for h in heads]
    w = (1 + 0.3 * torch.randn(4, d, generator=g)).cuda()
    pos = torch.randint(-5, 4096, lead, generator=g, dtype=torch.int32)
    if far:
        pos.view(-1)[::2] = far - torch.arange(pos.view(-1)[::2].numel(), dtype=torch.int32)
    freq = (theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float()
    dy = [0.3 * torch.randn(*lead, h, d, generator=g) for h in heads]
    return x, w, pos.cuda(), freq.cuda(), [t.cuda() for t in dy]


def check(got, ref, size, rel, what):
    got, ref, size = got.double().cpu(), ref.double().cpu(), size.cpu()
    half = 2.0 ** -8 if what == "bf16" else 2.0 ** -24
    bad = ~((got - ref).abs() <= half * ref.abs() + rel * size + 1e-30)
    assert not bad.any(), (int(bad.sum()), ((got - ref).abs() / (size + 1e-30)).max())


CASES = [  # tokens, h_s, h_n, d, rot, dtype, far, interleaved, fused
    ((1,), 1, 1, 64, 64, "bf16", 0, False, False),
    ((1, 1), 12, 4, 128, 128, "f32", 0, False, True),
    ((7,), 3, 1, 64, 32, "bf16", 131072, True, True),
    ((2, 65), 6, 2, 64, 64, "bf16", 131072, False, True),
    ((3, 31), 5, 5, 128, 48, "f32", 1 << 22, False, False),
    ((130,), 16, 4, 128, 128, "bf16", 1 << 22, True, True),
    ((1, 777), 12, 4, 64, 16, "f32", (1 << 31) - 1, False, True),
    ((4, 1000), 2, 1, 64, 64, "f32", (1 << 24) + 9, True, False),
    ((5003,), 1, 1, 128, 64, "bf16", 0, False, False),
    ((3,), 768, 256, 64, 64, "bf16", 0, False, True),       # as many heads as there may be
    ((2, 5), 1000, 8, 128, 16, "f32", 0, True, False),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_matches_float64(case):
    lead, hs, hn, d, rot, dt, far, inter, fused = case
    x, w, pos, freq, _ = make(lead, hs, hn, d, rot, torch.bfloat16 if dt == "bf16" else torch.float32, far,
                              seed=hs + rot, fused=fused)
    out = gda.gda_qk_norm_rope(*x, w, pos, freq, interleaved=inter)
    for i, y in enumerate(out):
        assert y.is_contiguous() and y.dtype == x[i].dtype
        ref = R.norm_rope(x[i].cpu(), w[i].cpu(), pos.cpu(), freq.cpu(), 1e-5, inter)
        check(y, ref, R.norm_rope_size(x[i].cpu(), w[i].cpu(), freq.cpu(), 1e-5, inter), 2.0 ** -19, dt)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_gradients_match_float64(case):
    lead, hs, hn, d, rot, dt, far, inter, fused = case
    x, w, pos, freq, dy = make(lead, hs, hn, d, rot, torch.bfloat16 if dt == "bf16" else torch.float32, far,
                               seed=hs + rot, fused=fused)
    grads = gda.gda_qk_norm_rope_bwd(*x, w, pos, freq, *dy, interleaved=inter)
    again = gda.gda_qk_norm_rope_bwd(*x, w, pos, freq, *dy, interleaved=inter)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    for i in range(4):
        args = (x[i].cpu(), w[i].cpu())
        dx, dw = R.norm_rope_grads(*args, pos.cpu(), freq.cpu(), dy[i].cpu(), 1e-5, inter)
        sx, sw = R.norm_rope_grad_size(*args, freq.cpu(), dy[i].cpu(), 1e-5, inter)
        check(grads[i], dx, sx, 2.0 ** -18, dt)
        check(grads[4][i], dw, sw, 2.0 ** -18, "f32")


def test_gradients_match_differences_of_the_forward():
    """float32 forward, central differences with h = 2^-6: the difference quotient of a smooth function of
    magnitude ~1 is off by h^2/6 of its third derivative (~1e-4 here) plus 2^-19 / h of rounding (~1e-4 per
    element, 64 of them at random signs: 1e-3)."""
    x, w, pos, freq, dy = make((3,), 2, 1, 64, 64, torch.float32, seed=5)
    grads = gda.gda_qk_norm_rope_bwd(*x, w, pos, freq, *dy)
    h = 2.0 ** -6
    for i in range(4):
        for at in ((0, 0, 0), (1, x[i].shape[1] - 1, 33), (2, 0, 63)):
            vals = []
            for sign in (1, -1):
                y = [t.clone() for t in x]
                y[i][at] += sign * h
                vals.append((gda.gda_qk_norm_rope(*y, w, pos, freq)[i].double() * dy[i].double()).sum().item())
            fd = (vals[0] - vals[1]) / (2 * h)
            assert abs(fd - grads[i][at].item()) <= 3e-3, (i, at, fd, grads[i][at].item())


def test_zero_rows_and_rows_of_nan_stay_alone():
    x, w, pos, freq, dy = make((9,), 3, 1, 64, 64, torch.bfloat16, seed=3)
    x[0][2, 1] = 0
    x[1][4, 0, 7] = float("nan")
    out = gda.gda_qk_norm_rope(*x, w, pos, freq)
    assert (out[0][2, 1] == 0).all()
    assert torch.isnan(out[1][4, 0]).any() and torch.isfinite(out[1][4, 1:].float()).all()
    assert torch.isfinite(out[1][:4].float()).all() and torch.isfinite(out[1][5:].float()).all()
    assert all(torch.isfinite(out[i].float()).all() for i in (0, 2, 3))
    grads = gda.gda_qk_norm_rope_bwd(*x, w, pos, freq, *dy)
    assert torch.isfinite(grads[0].float()).all() and torch.isfinite(grads[4][0]).all()


def test_in_place_and_into_slices_of_a_fused_gradient():
    x, w, pos, freq, dy = make((33,), 6, 2, 64, 64, torch.bfloat16, seed=8)
    ref = gda.gda_qk_norm_rope(*x, w, pos, freq)
    grads = gda.gda_qk_norm_rope_bwd(*x, w, pos, freq, *dy)
    fused = torch.full((33, 16 * 64 + 40), 7.0, dtype=torch.bfloat16, device="cuda")
    cuts = [0, 6, 12, 14, 16]
    views = [fused[:, a * 64:b * 64].unflatten(-1, (b - a, 64)) for a, b in zip(cuts, cuts[1:])]
    gda.gda_qk_norm_rope_bwd(*x, w, pos, freq, *dy, grads=(*views, torch.empty(4, 64, device="cuda")))
    assert all(torch.equal(a, b) for a, b in zip(views, grads))
    assert (fused[:, 16 * 64:] == 7).all()                         # the columns behind stay
    y = [t.clone() for t in x]
    gda.gda_qk_norm_rope(*y, w, pos, freq, out=tuple(y))
    assert all(torch.equal(a, b) for a, b in zip(y, ref))


def test_on_another_stream_and_in_a_graph():
    x, w, pos, freq, dy = make((300,), 6, 2, 128, 64, torch.float32, seed=9)
    ref = [t.clone() for t in gda.gda_qk_norm_rope(*x, w, pos, freq)]
    rgr = [t.clone() for t in gda.gda_qk_norm_rope_bwd(*x, w, pos, freq, *dy)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = gda.gda_qk_norm_rope(*x, w, pos, freq)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
    ws = torch.empty(gda.gda_qk_norm_rope_bwd_workspace_size(300, 6, 2, 128), dtype=torch.uint8, device="cuda")
    grads = tuple(torch.zeros_like(t) for t in rgr)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gda.gda_qk_norm_rope(*x, w, pos, freq, out=out)
        gda.gda_qk_norm_rope_bwd(*x, w, pos, freq, *dy, workspace=ws, grads=grads)
    for t in x:
        t.mul_(-1)                       # outputs and dw are odd in x, dx is even
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, -b) for a, b in zip(out, ref))
    assert all(torch.equal(a, b) for a, b in zip(grads[:4], rgr)) and torch.equal(grads[4], -rgr[4])


def test_binding_refuses():
    x, w, pos, freq, dy = make((4, 8), 6, 2, 64, 64, torch.bfloat16)
    call = lambda *a, **k: gda.gda_qk_norm_rope(*a, **k)
    for bad in [(x[0].float(), *x[1:]), (x[0], x[1][:, :7], *x[2:]), (x[0], x[1], x[2], x[3].cpu()),
                (x[0].transpose(0, 1).contiguous().transpose(0, 1), *x[1:])]:
        with pytest.raises((TypeError, ValueError)):
            call(*bad, w, pos, freq)
    for kw in (dict(w=w[:3]), dict(pos=pos.long()), dict(freq=freq.double())):
        a = dict(w=w, pos=pos, freq=freq) | kw
        with pytest.raises((TypeError, ValueError)):
            call(*x, a["w"], a["pos"], a["freq"])
    with pytest.raises(gda.GDAError):
        call(*x, w, pos, freq[:5])                                   # rot = 10
    with pytest.raises(gda.GDAError):
        call(*x, w, pos, freq, eps=-1.0)
    with pytest.raises((TypeError, ValueError)):
        gda.gda_qk_norm_rope_bwd(*x, w, pos, freq, dy[0].bfloat16(), *dy[1:])
    with pytest.raises(gda.GDAError):
        gda.gda_qk_norm_rope_bwd(*x, w, pos, freq, *dy, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
