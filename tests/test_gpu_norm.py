"""GPU parity of the norm and its gradients against the fp64 definitions.

Bounds, element by element.  A sum of n fp32 terms in lanes and then across them
is off by at most a(n) = n / 64 + 16 roundings of E32 = 2^-24 of the sum of the
terms' sizes (a lane adds n / 64 of them at most, the rest is a tree).
  mean    a E32 mean|x|; x - mu adds a rounding of its own
  squares relative 2 (a + 4) E32, half of it in r, with rsqrt's own rounding
  y       (|dmu| + E32 |x|) r |w| + |y| (a + 12) E32, and the output's rounding
  dx      u, its mean and its sum with xn are bounded alike; the three terms are
          of size r (|u| + mean|u| + |xn| mean|u xn|): that times (3 a + 24) E32,
          and what dmu does to xn (|dmu| r against every |u|)
  dw, db  sums over rows: (rows + 32) E32 sum|dy xn| at most, plus dy times what
          xn is off
"""
import numpy as np
import pytest
import torch

import test_weight_mlp_amd as ip
from block_helpers import BF16, E32, F32, HALF, TDT, generator, np64, randn, wide, within
from oracle import block as ob

pytestmark = pytest.mark.gpu
EPS = 1e-6


def pieces(x, center):
    """r, |x - mu|, and the bound of mu."""
    mu = x.mean(-1, keepdims=True) if center else 0.0 * x[:, :1]
    d = x - mu
    r = 1.0 / np.sqrt((d * d).mean(-1, keepdims=True) + EPS)
    a = x.shape[1] / 64 + 16
    dmu = a * E32 * np.abs(x).mean(-1, keepdims=True) if center else 0.0 * r
    return d, r, dmu + E32 * np.abs(x), a


def forward_bound(x, w, y, center, dt):
    d, r, off, a = pieces(x, center)
    ww = 1.0 if w is None else np.abs(w)
    return (off * r + np.abs(d) * r * (a + 12) * E32) * ww + np.abs(y) * (HALF[dt] + 2 * E32)


def check(p, x, w, b, y):
    dt, center = p.dtype, p.kind == ip.IPTTT_NORM_LAYER
    want = ob.norm(np64(x), np64(w), np64(b), center, EPS)
    within(y, want, forward_bound(np64(x), np64(w), want, center, dt))


def check_backward(p, x, w, dy, dres, dx, dw, db):
    dt, center = p.dtype, p.kind == ip.IPTTT_NORM_LAYER
    X, W, G, R = np64(x), np64(w), np64(dy), np64(dres)
    want = ob.norm_backward(X, W, G, R, center, EPS)
    d, r, off, a = pieces(X, center)
    u, xn = np.abs(G if W is None else G * W), np.abs(d) * r
    mean = lambda t: t.mean(-1, keepdims=True)  # noqa: E731
    size = r * (u + mean(u) + xn * mean(u * xn))
    shifted = r * (xn * mean(u * off * r) + off * r * mean(u * xn))
    within(dx, want[0], size * (3 * a + 24) * E32 + 2 * shifted + np.abs(want[0]) * (HALF[dt] + 2 * E32))
    n = len(X) + 32
    xn_off = off * r + xn * (a + 12) * E32
    if dw is not None:
        within(dw, want[1], (np.abs(G) * xn_off).sum(0) + n * E32 * (np.abs(G) * xn).sum(0) + E32 * np.abs(want[1]))
    if db is not None:
        within(db, want[2], n * E32 * np.abs(G).sum(0) + E32 * np.abs(want[2]))


def inputs(dt, rows, dim, seed=0, offset=0.3):
    g = generator(seed)
    size = torch.exp(0.5 * torch.randn(dim, generator=g, device="cuda"))
    x = (torch.randn(rows, dim, generator=g, device="cuda") * size + offset * size.roll(1)).to(TDT[dt])
    return x, 1 + randn(g, dt, dim, scale=0.1), randn(g, dt, dim, scale=0.1), randn(g, dt, rows, dim), randn(g, dt, rows, dim)


SHAPES = [(1, 8), (1, 2560), (3, 64), (5, 72), (7, 1000), (4, 1024), (257, 320), (2049, 64), (33, 2560), (6, 2568), (9, 4096),
          (2, 9728), (3, 16384), (1030, 16)]


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", [ip.IPTTT_NORM_RMS, ip.IPTTT_NORM_LAYER], ids=["rms", "layer"])
@pytest.mark.parametrize("rows, dim", SHAPES)
def test_norm_and_gradients(dt, kind, rows, dim):
    p = ip.NormProblem(rows, dim, dt, kind, EPS)
    x, w, b, dy, dres = inputs(dt, rows, dim, seed=rows + dim)
    g = ip.NormGrads(p)
    for ww, bb, more in ((w, b, dres), (w, None, None), (None, None, dres)):
        y = torch.empty_like(x)
        ip.ipttt_norm(p, x, ww, bb, y)
        check(p, x, ww, bb, y)
        dw = None if ww is None else g.dw.fill_(5.0)
        db = None if bb is None else g.db.fill_(5.0)
        ip.ipttt_norm_backward(p, x, ww, dy, g.dx, dw, db, g.ws if dw is not None else None, dres=more)
        check_backward(p, x, ww, dy, more, g.dx, dw, db)


# rows that share a wave, at the edges of 8, 16 and 32 lanes, in a last workgroup that is not full
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", [ip.IPTTT_NORM_RMS, ip.IPTTT_NORM_LAYER], ids=["rms", "layer"])
@pytest.mark.parametrize("rows, dim", [(1, 64), (131, 8), (131, 32), (259, 40), (67, 128), (601, 136), (45, 256), (130, 264)])
def test_narrow_rows(dt, kind, rows, dim):
    test_norm_and_gradients(dt, kind, rows, dim)


# more rows than the gradient's launch has places, for one to eight waves a row
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows, dim", [(9001, 64), (4500, 1000), (2100, 2560), (1301, 4096), (700, 9728)])
def test_several_rounds_of_rows(dt, rows, dim):
    test_norm_and_gradients(dt, ip.IPTTT_NORM_LAYER, rows, dim)


@pytest.mark.parametrize("rows, dim", [(5, 64), (37, 2560), (3, 4096)])
def test_slices_of_wider_tensors_and_in_place(rows, dim):
    for dt in (BF16, F32):
        p = ip.NormProblem(rows, dim, dt, ip.IPTTT_NORM_LAYER, EPS)
        x0, w, b, dy0, dres0 = inputs(dt, rows, dim)
        x, x_kept = wide(dt, rows, dim, 32)
        dy, dy_kept = wide(dt, rows, dim, 16)
        dres, dres_kept = wide(dt, rows, dim, 48)
        y, y_kept = wide(dt, rows, dim, 64)
        for t, v in ((x, x0), (dy, dy0), (dres, dres0)):
            t.copy_(v)
        ip.ipttt_norm(p, x, w, b, y)
        check(p, x0, w, b, y)
        plain = torch.empty_like(x0)
        ip.ipttt_norm(p, x0, w, b, plain)
        assert torch.equal(plain, y)
        g = ip.NormGrads(p)
        ip.ipttt_norm_backward(p, x0, w, dy0, g.dx, g.dw, g.db, g.ws, dres=dres0)
        want = g.dx.clone(), g.dw.clone(), g.db.clone()
        for over in (dy, dres):     # dx over its cotangent, then over the residual stream's
            over.copy_(dy0 if over is dy else dres0)
            ip.ipttt_norm_backward(p, x, w, dy if over is dy else dy0, over, g.dw, g.db, g.ws,
                                   dres=dres if over is dres else dres0)
            assert torch.equal(over, want[0]) and torch.equal(g.dw, want[1]) and torch.equal(g.db, want[2])
        ip.ipttt_norm(p, x, w, b, x)
        assert torch.equal(plain, x)
        assert x_kept() and dy_kept() and dres_kept() and y_kept()


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows, dim", [(5, 64), (2100, 320), (700, 2560), (300, 4096), (260, 9728)])
def test_gradient_over_the_input(dt, rows, dim):
    """dx over x, over columns of a wider tensor and over all of it; several rounds of rows."""
    for kind in (ip.IPTTT_NORM_RMS, ip.IPTTT_NORM_LAYER):
        p = ip.NormProblem(rows, dim, dt, kind, EPS)
        x0, w, _, dy, dres = inputs(dt, rows, dim)
        g, g2 = ip.NormGrads(p), ip.NormGrads(p)
        ip.ipttt_norm_backward(p, x0, w, dy, g.dx, g.dw, g.db, g.ws, dres=dres)
        x, x_kept = wide(dt, rows, dim, 32)
        x.copy_(x0)
        for over in (x, x0):
            ip.ipttt_norm_backward(p, over, w, dy, over, g2.dw, g2.db, g2.ws, dres=dres)
            assert torch.equal(over, g.dx) and torch.equal(g2.dw, g.dw) and torch.equal(g2.db, g.db)
        assert x_kept()


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_rows_far_from_zero_and_rows_of_nothing(dt):
    """A mean a thousand times the spread; zeros; a constant row; tiny and huge rows."""
    dim = 512
    p = ip.NormProblem(6, dim, dt, ip.IPTTT_NORM_LAYER, EPS)
    x, w, b, dy, _ = inputs(dt, 6, dim, offset=0.0)
    x[0] += 1000.0
    x[1] = 0.0
    x[2] = 3.5
    x[3] *= 1e-15
    x[4] *= 1e15
    y = torch.empty_like(x)
    ip.ipttt_norm(p, x, w, b, y)
    check(p, x, w, b, y)
    g = ip.NormGrads(p)
    ip.ipttt_norm_backward(p, x, w, dy, g.dx, g.dw, g.db, g.ws)
    check_backward(p, x, w, dy, None, g.dx, g.dw, g.db)


@pytest.mark.parametrize("dim", [64, 4096])
def test_an_infinite_row_stays_its_own(dim):
    p = ip.NormProblem(9, dim, BF16, ip.IPTTT_NORM_LAYER, EPS)
    x, w, b, dy, _ = inputs(BF16, 9, dim)
    clean, dirty = torch.empty_like(x), torch.empty_like(x)
    ip.ipttt_norm(p, x, w, b, clean)
    g = ip.NormGrads(p)
    ip.ipttt_norm_backward(p, x, w, dy, g.dx, None, None, None)
    want = g.dx.clone()
    x[4, 3], x[7, 5] = float("inf"), float("nan")
    ip.ipttt_norm(p, x, w, b, dirty)
    ip.ipttt_norm_backward(p, x, w, dy, g.dx, None, None, None)
    others = [0, 1, 2, 3, 5, 6, 8]
    assert torch.equal(clean[others], dirty[others]) and torch.equal(want[others], g.dx[others])
    assert dirty[7].isnan().all() and dirty[4].isnan().any()


def test_a_row_does_not_depend_on_the_others():
    for dim in (320, 2560, 4096):
        x, w, b, dy, _ = inputs(BF16, 700, dim)
        one, all_ = ip.NormProblem(1, dim, BF16), ip.NormProblem(700, dim, BF16)
        y, y1 = torch.empty_like(x), torch.empty_like(x[:1])
        ip.ipttt_norm(all_, x, w, b, y)
        g, g1 = ip.NormGrads(all_), ip.NormGrads(one)
        ip.ipttt_norm_backward(all_, x, w, dy, g.dx, g.dw, g.db, g.ws)
        for i in (0, 511, 699):
            ip.ipttt_norm(one, x[i:i + 1], w, b, y1)
            ip.ipttt_norm_backward(one, x[i:i + 1], w, dy[i:i + 1], g1.dx, g1.dw, g1.db, g1.ws)
            assert torch.equal(y1[0], y[i]) and torch.equal(g1.dx[0], g.dx[i])


def test_gradients_against_differences():
    """<y, dy> along a direction, in fp32: a step h moves y by h |J u|; the outputs'
    roundings give the quotient an error of 2^-22 |y| |dy| / h, the third
    derivative one of h^2: 1e-3 of |gradient| covers both at h = 1e-2."""
    p = ip.NormProblem(6, 256, F32, ip.IPTTT_NORM_LAYER, EPS)
    x, w, b, dy, _ = inputs(F32, 6, 256)
    g = ip.NormGrads(p)
    ip.ipttt_norm_backward(p, x, w, dy, g.dx, g.dw, g.db, g.ws)

    def loss():
        y = torch.empty_like(x)
        ip.ipttt_norm(p, x, w, b, y)
        return float((y.double() * dy.double()).sum())

    for t, grad in ((x, g.dx), (w, g.dw), (b, g.db)):
        u, keep, h = grad / grad.norm(), t.clone(), 1e-2
        t.copy_(keep + h * u)
        up = loss()
        t.copy_(keep - h * u)
        slope = (up - loss()) / (2 * h)
        t.copy_(keep)
        assert abs(slope - float(grad.norm())) <= 1e-3 * float(grad.norm())


def test_offsets_past_32_bits():
    rows, dim, stride = 600, 64, 1 << 22       # 2.5e9 elements from the first row to the last
    t = torch.empty(rows * stride, dtype=torch.bfloat16, device="cuda")
    x = t.as_strided((rows, dim), (stride, 1))
    p = ip.NormProblem(rows, dim, BF16, ip.IPTTT_NORM_LAYER, EPS)
    x0, w, b, dy, _ = inputs(BF16, rows, dim)
    x.copy_(x0)
    want, g, g0 = torch.empty_like(x0), ip.NormGrads(p), ip.NormGrads(p)
    ip.ipttt_norm(p, x0, w, b, want)
    ip.ipttt_norm_backward(p, x0, w, dy, g0.dx, g0.dw, g0.db, g0.ws)
    ip.ipttt_norm_backward(p, x, w, dy, g.dx, g.dw, g.db, g.ws)
    assert torch.equal(g.dx, g0.dx) and torch.equal(g.dw, g0.dw)
    ip.ipttt_norm(p, x, w, b, x)
    assert torch.equal(x, want)


def test_many_rows():
    """More rows than a launch has waves for at once, and the same bits twice."""
    rows = 70001
    p = ip.NormProblem(rows, 64, BF16, ip.IPTTT_NORM_RMS, EPS)
    x, w, b, dy, dres = inputs(BF16, rows, 64)
    y, g, g2 = torch.empty_like(x), ip.NormGrads(p), ip.NormGrads(p)
    ip.ipttt_norm(p, x, w, b, y)
    check(p, x, w, b, y)
    ip.ipttt_norm_backward(p, x, w, dy, g.dx, g.dw, g.db, g.ws, dres=dres)
    check_backward(p, x, w, dy, dres, g.dx, g.dw, g.db)
    ip.ipttt_norm_backward(p, x, w, dy, g2.dx, g2.dw, g2.db, g2.ws, dres=dres)
    assert torch.equal(g.dw, g2.dw) and torch.equal(g.db, g2.db) and torch.equal(g.dx, g2.dx)


def test_other_streams_and_graphs():
    p = ip.NormProblem(300, 1024, BF16, ip.IPTTT_NORM_LAYER, EPS)
    x, w, b, dy, dres = inputs(BF16, 300, 1024)
    y, g = torch.empty_like(x), ip.NormGrads(p)

    def both(stream=None):
        ip.ipttt_norm(p, x, w, b, y, stream=stream)
        ip.ipttt_norm_backward(p, x, w, dy, g.dx, g.dw, g.db, g.ws, dres=dres, stream=stream)

    both()
    want = [t.clone() for t in (y, g.dx, g.dw, g.db)]
    side = torch.cuda.Stream()
    for t in (y, g.dx, g.dw, g.db):
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    both(side)
    side.synchronize()
    assert all(torch.equal(a, t) for a, t in zip(want, (y, g.dx, g.dw, g.db)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for seed in (1, 2, 3):      # new values in the captured tensors
        for t, v in zip((x, w, b, dy, dres), inputs(BF16, 300, 1024, seed)):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, g.dx, g.dw, g.db)]
        both()
        assert all(torch.equal(a, t) for a, t in zip(got, (y, g.dx, g.dw, g.db)))
