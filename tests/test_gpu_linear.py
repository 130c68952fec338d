"""GPU parity of projections and their gradients against the fp64 definitions.

Bounds, element by element.  A product sums K terms in fp32, in any order: at most
K roundings of the sum of the terms' sizes, S = sum |a b|; the matrix cores may
cut instead of round, so each counts as 2 E32 = 2^-23: K 2^-23 S, at least 8
roundings.
  pre   that, one rounding for the bias and the output's
  y     the activations' slopes are at most 1.13; their own arithmetic (exp, erfc and
        a reciprocal of about 1 ulp each) is good to 32 E32 of |v|, and so is that of a
        residual sum
  dp    |dy| times 32 E32 (1 + |v|) (the slope), in dtype a rounding HALF |dp| more
  dx    the product's, and sum |dp's error| |W|; dW alike; db sums dp in fp32
The root mean square of bf16's rounding is below 2^-9: over a whole tensor an
output of one rounding is within 2^-9 of the definition's norm, of two within
1.5 2^-9.
"""
import numpy as np
import pytest
import torch

import test_weight_mlp_amd as ip
from block_helpers import BF16, E32, F32, HALF, TDT, generator, np64, randn, wide, within
from oracle import block as ob

pytestmark = pytest.mark.gpu
ACTS = {"none": ip.IPTTT_ACT_NONE, "silu": ip.IPTTT_ACT_SILU, "gelu": ip.IPTTT_ACT_GELU}
IDS = dict(argvalues=[BF16, F32], ids=["bf16", "f32"])


def rel(got, want):
    return np.linalg.norm(np64(got) - want) / max(np.linalg.norm(want), 1e-300)


def product_bound(a, b, k):
    return max(k, 8) * 2 * E32 * (np.abs(a) @ np.abs(b))


def check(p, kind, x, W, b, res, y, pre):
    X, V, B, R = (np64(t) for t in (x, W, b, res))
    want, mid = ob.linear(X, V, B, R, kind)
    off = product_bound(X, V.T, X.shape[1]) + 2 * E32 * np.abs(mid)
    if pre is not None:
        within(pre, mid, off + HALF[p.dtype] * np.abs(mid))
    within(y, want, 1.13 * off + 32 * E32 * (np.abs(mid) + np.abs(want)) + HALF[p.dtype] * np.abs(want))
    if p.dtype == BF16 and y.numel() > 4096:
        assert rel(y, want) <= 2.0 ** -9


def check_backward(p, kind, x, W, pre, dy, dx, dW, db):
    X, V, P, G = (np64(t) for t in (x, W, pre, dy))
    want = ob.linear_backward(X, V, P, G, kind)
    dp = G if kind == "none" else G * ob.slope(kind, P)
    fine = 0.0 * dp if kind == "none" else 32 * E32 * np.abs(G) * (1 + np.abs(P))
    off = fine + (HALF[p.dtype] * np.abs(dp) if kind != "none" else 0.0)
    loose = 1.5 if kind != "none" else 1.0
    if dx is not None:
        within(dx, want[0], product_bound(dp, V, len(V)) + off @ np.abs(V) + HALF[p.dtype] * np.abs(want[0]))
        if p.dtype == BF16 and dx.numel() > 4096:
            assert rel(dx, want[0]) <= loose * 2.0 ** -9
    if dW is not None:
        within(dW, want[1], product_bound(dp.T, X, len(X)) + off.T @ np.abs(X) + HALF[p.grad_dtype] * np.abs(want[1]))
        if p.grad_dtype == BF16 and dW.numel() > 4096:
            assert rel(dW, want[1]) <= loose * 2.0 ** -9
    if db is not None:
        within(db, want[2], fine.sum(0) + (len(X) + 8) * E32 * np.abs(dp).sum(0))


def inputs(dt, m, k, n, seed=0):
    g = generator(seed)
    return (randn(g, dt, m, k), randn(g, dt, n, k, scale=k ** -0.5), randn(g, dt, n, scale=0.1), randn(g, dt, m, n),
            randn(g, dt, m, n))


def forward(p, x, W, b=None, res=None, keep=False, **kw):
    y = torch.full((p.rows, p.out_dim), 5.0, dtype=x.dtype, device="cuda")
    pre = torch.full_like(y, 5.0) if keep else None
    ip.ipttt_linear(p, x, W, y, b=b, res=res, pre=pre, ws=ip.linear_workspace(p), **kw)
    return y, pre


# rows: single tokens, the sizes around the tiles' edges, and several tiles
ROWS = [1, 2, 5, 16, 17, 32, 33, 64, 65, 127, 129, 257, 1030]
DIMS = [(8, 8), (64, 64), (72, 200), (320, 448), (1024, 136), (640, 1280)]


@pytest.mark.parametrize("dt", **IDS)
@pytest.mark.parametrize("k, n", DIMS)
@pytest.mark.parametrize("m", ROWS)
def test_linear(dt, m, k, n):
    x, W, b, res, _ = inputs(dt, m, k, n, seed=m + k)
    for kind, bias, more, keep in (("none", None, None, False), ("gelu", b, res, True), ("silu", b, None, False),
                                   ("none", None, res, True)):
        p = ip.LinearProblem(m, k, n, dt, ACTS[kind])
        y, pre = forward(p, x, W, bias, more, keep)
        check(p, kind, x, W, bias, more, y, pre)


@pytest.mark.parametrize("dt", **IDS)
@pytest.mark.parametrize("k, n", DIMS)
@pytest.mark.parametrize("m", [1, 3, 16, 33, 65, 129, 260, 1030])
def test_linear_backward(dt, m, k, n):
    x, W, b, pre, dy = inputs(dt, m, k, n, seed=m + n)
    for kind, grad in (("none", F32), ("gelu", dt), ("silu", F32), ("none", dt)):
        p = ip.LinearProblem(m, k, n, dt, ACTS[kind], grad_dtype=grad)
        g = ip.LinearGrads(p)
        for t in (g.dx, g.dW, g.db):
            t.fill_(5.0)
        kept = pre if kind != "none" else None
        ip.ipttt_linear_backward(p, x, W, dy, g.dx, g.dW, g.db, g.ws, pre=kept)
        check_backward(p, kind, x, W, kept, dy, g.dx, g.dW, g.db)
        want = [t.clone() for t in (g.dx, g.dW, g.db)]
        for i in range(3):   # each on its own
            for t in (g.dx, g.dW, g.db):
                t.fill_(5.0)
            out = [t if j == i else None for j, t in enumerate((g.dx, g.dW, g.db))]
            ip.ipttt_linear_backward(p, x, W, dy, *out, g.ws, pre=kept)
            assert torch.equal(out[i], want[i])
            assert all(bool((t == 5.0).all()) for j, t in enumerate((g.dx, g.dW, g.db)) if j != i)


# (M, N, K) of a product of the large launches: in bf16 tiles of each size in more than one
# round, and those with the last ones cut along K; in fp32 the same
LARGE = [(BF16, 5688, 5504, 80), (BF16, 6040, 2744, 840), (BF16, 5432, 4048, 72), (BF16, 3296, 5064, 600),
         (BF16, 7216, 1144, 872), (BF16, 6560, 1176, 856), (BF16, 5384, 3096, 136), (BF16, 776, 5000, 1696),
         (BF16, 4624, 1712, 80), (F32, 8368, 400, 2648), (F32, 8320, 904, 168), (F32, 5456, 712, 312),
         (F32, 5600, 3288, 72)]


@pytest.mark.parametrize("which", ["y", "dx", "dW"])
@pytest.mark.parametrize("dt, M, N, K", LARGE)
def test_large_launches(dt, M, N, K, which):
    """Each product in these sizes, in 64 bits on the device; bounds as above."""
    m, k, n = {"y": (M, K, N), "dx": (M, N, K), "dW": (K, N, M)}[which]
    x, W, b, res, dy = inputs(dt, m, k, n, seed=7)
    p = ip.LinearProblem(m, k, n, dt, ip.IPTTT_ACT_SILU if which == "y" else ip.IPTTT_ACT_NONE, grad_dtype=dt)
    X, V, G = (t.double() for t in (x, W, dy))
    half = HALF[dt]

    def near(got, want, bound):
        assert bool(((got.double() - want).abs() <= bound).all())

    if which == "y":
        y, pre = forward(p, x, W, b, res, True)
        mid = X @ V.T + b.double()
        off = K * 2 * E32 * (X.abs() @ V.abs().T) + 2 * E32 * mid.abs()
        near(pre, mid, off + half * mid.abs())
        want = mid * torch.sigmoid(mid) + res.double()
        near(y, want, 1.13 * off + 32 * E32 * (mid.abs() + want.abs()) + half * want.abs())
        return
    g = ip.LinearGrads(p)
    for t in (g.dx, g.dW):
        t.fill_(5.0)
    if which == "dx":
        ip.ipttt_linear_backward(p, x, W, dy, g.dx, None, None, g.ws)
        want = G @ V
        near(g.dx, want, K * 2 * E32 * (G.abs() @ V.abs()) + half * want.abs())
    else:
        ip.ipttt_linear_backward(p, x, W, dy, None, g.dW, g.db, g.ws)
        want = G.T @ X
        near(g.dW, want, K * 2 * E32 * (G.abs().T @ X.abs()) + half * want.abs())
        near(g.db, G.sum(0), (K + 8) * E32 * G.abs().sum(0))


def test_two_calls_at_once_and_two_graphs():
    """Calls side by side on two streams, each with its own workspace, and two captured
    graphs that share one, replayed in turn."""
    shapes = [(1500, 256, 320), (700, 512, 256)]
    made = []
    for i, (m, k, n) in enumerate(shapes):
        p = ip.LinearProblem(m, k, n, BF16, ip.IPTTT_ACT_SILU)
        x, W, b, res, dy = inputs(BF16, m, k, n, seed=20 + i)
        made.append((p, x, W, b, res, dy, torch.empty_like(res), torch.empty_like(res), ip.LinearGrads(p)))

    def call(c, ws, gws, stream=None):
        p, x, W, b, res, dy, y, pre, g = c
        ip.ipttt_linear(p, x, W, y, b=b, res=res, pre=pre, ws=ws, stream=stream)
        ip.ipttt_linear_backward(p, x, W, dy, g.dx, g.dW, g.db, gws, pre=pre, stream=stream)

    own = [(ip.linear_workspace(c[0]), c[8].ws) for c in made]
    outs = [(c[6], c[7], c[8].dx, c[8].dW, c[8].db) for c in made]
    want = []
    for c, w, o in zip(made, own, outs):
        call(c, *w)
        want.append([t.clone() for t in o])
        for t in o:
            t.zero_()
    streams = [torch.cuda.Stream() for _ in made]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for c, w, s in zip(made, own, streams):
            call(c, *w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, t) for w, o in zip(want, outs) for a, t in zip(w, o))
    shared = torch.empty(max(t.numel() for w in own for t in w if t is not None), dtype=torch.uint8, device="cuda")
    graphs = []
    for c in made:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(c, shared, shared)
    for _ in range(3):
        for g, w, o in zip(graphs, want, outs):
            for t in o:
                t.zero_()
            shared.fill_(0xFF)
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, t) for a, t in zip(w, o))


@pytest.mark.parametrize("m, k, n", [(3, 128, 192), (40, 192, 64), (300, 256, 512), (70, 72, 104)])
def test_columns_of_wider_tensors_and_in_place(m, k, n):
    for dt in (BF16, F32):
        x0, W, b, res0, dy0 = inputs(dt, m, k, n)
        (x, x_kept), (res, res_kept), (y, y_kept), (pre, pre_kept), (dy, dy_kept), (dx, dx_kept) = (
            wide(dt, m, c, e) for c, e in ((k, 48), (n, 16), (n, 32), (n, 64), (n, 112), (k, 8)))
        for t, v in ((x, x0), (res, res0), (dy, dy0)):
            t.copy_(v)
        p = ip.LinearProblem(m, k, n, dt, ip.IPTTT_ACT_SILU)
        ws = ip.linear_workspace(p)
        want, want_pre = forward(p, x0, W, b, res0, True)
        check(p, "silu", x0, W, b, res0, want, want_pre)
        ip.ipttt_linear(p, x, W, y, b=b, res=res, pre=pre, ws=ws)
        assert torch.equal(y, want) and torch.equal(pre, want_pre)
        ip.ipttt_linear(p, x, W, res, b=b, res=res, ws=ws)     # y over the residual stream
        assert torch.equal(res, want)
        g, g2 = ip.LinearGrads(p), ip.LinearGrads(p)
        ip.ipttt_linear_backward(p, x0, W, dy0, g.dx, g.dW, g.db, g.ws, pre=want_pre)
        ip.ipttt_linear_backward(p, x, W, dy, dx, g2.dW, g2.db, g2.ws, pre=pre)
        assert torch.equal(dx, g.dx) and torch.equal(g2.dW, g.dW) and torch.equal(g2.db, g.db)
        assert x_kept() and res_kept() and y_kept() and pre_kept() and dy_kept() and dx_kept()


@pytest.mark.parametrize("m, k, n", [(3, 64, 72), (40, 192, 64), (300, 256, 520)])
@pytest.mark.parametrize("kind", ["none", "gelu"])
def test_tensors_that_start_at_16_bytes(m, k, n, kind):
    """fp32 tensors whose rows of 8 elements start in the middle of 32 bytes."""
    p = ip.LinearProblem(m, k, n, F32, ACTS[kind])
    x0, W, b, pre0, dy0 = inputs(F32, m, k, n)

    def placed(rows, cols, values=None):
        t = torch.full((rows, cols + 8), 7.0, device="cuda")[:, 4:4 + cols]
        assert t.data_ptr() % 32 == 16
        return t if values is None else t.copy_(values)

    x, dy, dx, y, res = placed(m, k, x0), placed(m, n, dy0), placed(m, k), placed(m, n), placed(m, n, pre0)
    pre = placed(m, n, pre0) if kind != "none" else None
    want, _ = forward(p, x0, W, b, pre0)
    ip.ipttt_linear(p, x, W, y, b=b, res=res, ws=ip.linear_workspace(p))
    assert torch.equal(y, want)
    g, g2 = ip.LinearGrads(p), ip.LinearGrads(p)
    ip.ipttt_linear_backward(p, x0, W, dy0, g.dx, g.dW, g.db, g.ws, pre=None if pre is None else pre0)
    ip.ipttt_linear_backward(p, x, W, dy, dx, g2.dW, g2.db, g2.ws, pre=pre)
    check_backward(p, kind, x, W, pre, dy, dx, g2.dW, g2.db)
    assert torch.equal(dx, g.dx) and torch.equal(g2.dW, g.dW) and torch.equal(g2.db, g.db)


@pytest.mark.parametrize("m", [1, 20, 100, 513])
def test_rows_with_infinities_stay_their_own(m):
    k, n = 256, 320
    x, W, _, res, dy = inputs(BF16, m, k, n)
    p = ip.LinearProblem(m, k, n)
    clean, _ = forward(p, x, W, None, res)
    g = ip.LinearGrads(p)
    ip.ipttt_linear_backward(p, x, W, dy, g.dx, None, None, g.ws)
    want = g.dx.clone()
    bad = m // 2
    x[bad, 7], dy[bad, 3] = float("inf"), float("nan")
    dirty, _ = forward(p, x, W, None, res)
    ip.ipttt_linear_backward(p, x, W, dy, g.dx, None, None, g.ws)
    others = [i for i in range(m) if i != bad]
    assert torch.equal(clean[others], dirty[others]) and torch.equal(want[others], g.dx[others])
    assert not dirty[bad].isfinite().any() and g.dx[bad].isnan().all()


def test_activations_of_extreme_values():
    """W = the unit matrix: y = act(x) for values far out, infinite and NaN."""
    v = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 5.0, -5.0, 12.0, -12.0, 90.0, -90.0, 1e4, -1e4, 3e38, -3e38] + [1.0] * 50)
    for dt in (F32, BF16):
        x = v.to(TDT[dt]).cuda()[None].contiguous()
        W = torch.eye(64).to(TDT[dt]).cuda()
        for kind in ("silu", "gelu"):
            p = ip.LinearProblem(1, 64, 64, dt, ACTS[kind])
            y, pre = forward(p, x, W, keep=True)
            want = ob.act(kind, np64(x))
            within(y, want, 64 * E32 * np.abs(np64(x)) + HALF[dt] * np.abs(want) + 1e-37)
            dy = torch.ones_like(x)
            g = ip.LinearGrads(p)
            ip.ipttt_linear_backward(p, x, W, dy, g.dx, g.dW, g.db, g.ws, pre=pre)
            slope = ob.slope(kind, np64(x))
            # |v| up to 90 in an exponent of fp32
            within(g.dx, slope, 64 * E32 * (1 + np.minimum(np.abs(np64(x)), 100)) + 2 * HALF[dt] * np.abs(slope))


@pytest.mark.parametrize("dt", **IDS)
@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
@pytest.mark.parametrize("m", [3, 100])   # one pass over the weights; tiles
def test_infinite_and_nan_values_before_an_activation(m, kind, dt):
    """Infinities and a NaN come in through the bias, and through pre in the gradient:
    where the definition has a number or an infinity so has the call, where it has a NaN
    (0 times an infinity) the call has one, and the other outputs are those without them."""
    k = n = 64
    x, W, b, pre, dy = inputs(dt, m, k, n)
    p = ip.LinearProblem(m, k, n, dt, ACTS[kind], grad_dtype=dt)
    clean, _ = forward(p, x, W, b)
    odd = {3: float("inf"), 17: float("-inf"), 40: float("nan")}
    for at, v in odd.items():
        b[at] = v
    y, kept = forward(p, x, W, b, keep=True)
    rest = [i for i in range(n) if i not in odd]
    assert torch.equal(y[:, rest], clean[:, rest])
    with np.errstate(invalid="ignore", over="ignore"):
        v = np.array(list(odd.values()))
        act, slope = ob.act(kind, v), ob.slope(kind, v)
    got, mid = np64(y)[:, list(odd)], np64(kept)[:, list(odd)]
    assert np.array_equal(mid, np.broadcast_to(v, mid.shape), equal_nan=True)
    assert np.array_equal(got, np.broadcast_to(act, got.shape), equal_nan=True)
    g, g2 = ip.LinearGrads(p), ip.LinearGrads(p)
    none = kind == "none"
    ip.ipttt_linear_backward(p, x, W, dy, g.dx, g.dW, g.db, g.ws, pre=None if none else pre)
    dirty = pre.clone()
    dirty[m // 2, list(odd)] = torch.tensor(v, device="cuda").to(dirty.dtype)
    ip.ipttt_linear_backward(p, x, W, dy, g2.dx, g2.dW, g2.db, g2.ws, pre=None if none else dirty)
    others = [i for i in range(m) if none or i != m // 2]
    assert torch.equal(g2.dx[others], g.dx[others]) and torch.equal(g2.dW[rest], g.dW[rest])
    assert torch.equal(g2.db[rest], g.db[rest])
    finite = [at for at, s in zip(odd, slope) if np.isfinite(s)]
    bad = [at for at, s in zip(odd, slope) if not np.isfinite(s)]
    assert g2.db[finite].isfinite().all() and g2.db[bad].isnan().all() and g2.dW[bad].isnan().all()
    assert g2.dx[m // 2].isnan().all() if bad else g2.dx.isfinite().all()


@pytest.mark.parametrize("m", [2, 130])   # one pass over the weights; tiles
def test_gelu_of_negative_values_keeps_their_bits(m):
    """Relative to the value, through the unit matrix (exact).  The tail's polynomial is
    off by 0.5 roundings, its evaluation by up to 8 (an emulation of the fp32 steps), the
    reciprocal and the exponential by an ulp each (2 + 2), the product with v by one: 14,
    bounded by 16.  The slope's second term, v times the density, is the larger: the tail's
    and the density's errors, 16 and 8, add to less than 28 of their difference."""
    g = generator(5)
    v = -3 - 9 * torch.rand(m, 64, generator=g, device="cuda")
    W = torch.eye(64, device="cuda")
    p = ip.LinearProblem(m, 64, 64, F32, ACTS["gelu"])
    y, pre = forward(p, v, W, keep=True)
    want = ob.act("gelu", np64(v))
    assert torch.equal(pre, v)
    within(y, want, 16 * E32 * np.abs(want))
    grads = ip.LinearGrads(p)
    ip.ipttt_linear_backward(p, v, W, torch.ones_like(v), grads.dx, None, None, grads.ws, pre=pre)
    slope = ob.slope("gelu", np64(v))
    within(grads.dx, slope, 28 * E32 * np.abs(slope))


@pytest.mark.parametrize("m", [1, 31, 200, 700])
def test_a_row_does_not_depend_on_the_others(m):
    """The same row at other places of a call of the same size."""
    k, n = 320, 256
    x, W, b, res, dy = inputs(BF16, m, k, n)
    p = ip.LinearProblem(m, k, n, act=ip.IPTTT_ACT_GELU)
    y, pre = forward(p, x, W, b, res, True)
    turn = torch.roll(torch.arange(m), m // 3).cuda()
    y2, pre2 = forward(p, x[turn].contiguous(), W, b, res[turn].contiguous(), True)
    assert torch.equal(y[turn], y2) and torch.equal(pre[turn], pre2)
    g, g2 = ip.LinearGrads(p), ip.LinearGrads(p)
    ip.ipttt_linear_backward(p, x, W, dy, g.dx, g.dW, g.db, g.ws, pre=pre)
    ip.ipttt_linear_backward(p, x[turn].contiguous(), W, dy[turn].contiguous(), g2.dx, None, None, g2.ws, pre=pre2)
    assert torch.equal(g.dx[turn], g2.dx)
    keep = g.dW.clone()
    ip.ipttt_linear_backward(p, x, W, dy, g.dx, g.dW, g.db, g.ws, pre=pre)
    assert torch.equal(keep, g.dW)


def test_gradients_against_differences():
    """<y, dy> along each gradient, in fp32; the bound as for the norm's."""
    m, k, n = 40, 64, 72
    x, W, b, res, dy = inputs(F32, m, k, n)
    for kind in ACTS:
        p = ip.LinearProblem(m, k, n, F32, ACTS[kind])
        _, pre = forward(p, x, W, b, res, True)
        g = ip.LinearGrads(p)
        ip.ipttt_linear_backward(p, x, W, dy, g.dx, g.dW, g.db, g.ws, pre=pre)
        for t, grad in ((x, g.dx), (W, g.dW), (b, g.db)):
            u, keep, h = grad / grad.norm(), t.clone(), 1e-2

            def loss():
                y, _ = forward(p, x, W, b, res)
                return float((y.double() * dy.double()).sum())

            t.copy_(keep + h * u)
            up = loss()
            t.copy_(keep - h * u)
            slope = (up - loss()) / (2 * h)
            t.copy_(keep)
            assert abs(slope - float(grad.norm())) <= 2e-3 * float(grad.norm())


@pytest.mark.parametrize("dt", **IDS)
@pytest.mark.parametrize("m", [3, 100, 600])
def test_offsets_past_32_bits(dt, m):
    """Rows 2^22 apart: the last starts up to 2.5e9 elements after the first."""
    k, n, stride = 64, 128, 1 << 22
    x0, W, b, res0, dy0 = inputs(dt, m, k, n)
    room = [torch.empty((m - 1) * stride + 256, dtype=TDT[dt], device="cuda") for _ in "ab"]
    x, res, y, pre = (room[i].as_strided((m, c), (stride, 1), o) for i, c, o in ((0, k, 0), (0, n, 128), (1, n, 0), (1, n, 128)))
    x.copy_(x0)
    res.copy_(res0)
    p = ip.LinearProblem(m, k, n, dt, ip.IPTTT_ACT_SILU)
    want, want_pre = forward(p, x0, W, b, res0, True)
    ip.ipttt_linear(p, x, W, y, b=b, res=res, pre=pre, ws=ip.linear_workspace(p))
    assert torch.equal(y, want) and torch.equal(pre, want_pre)
    g, g2 = ip.LinearGrads(p), ip.LinearGrads(p)
    ip.ipttt_linear_backward(p, x0, W, dy0, g.dx, g.dW, g.db, g.ws, pre=want_pre)
    y.copy_(dy0)
    ip.ipttt_linear_backward(p, x, W, y, res[:, :k], g2.dW, g2.db, g2.ws, pre=pre)
    assert torch.equal(res[:, :k], g.dx) and torch.equal(g2.dW, g.dW) and torch.equal(g2.db, g.db)


@pytest.mark.parametrize("m, k, n", [(1, 512, 256), (30, 256, 512), (200, 512, 256), (1500, 256, 320)])
def test_other_streams_and_graphs(m, k, n):
    p = ip.LinearProblem(m, k, n, BF16, ip.IPTTT_ACT_GELU)
    x, W, b, res, dy = inputs(BF16, m, k, n)
    y, pre, ws, g = torch.empty_like(res), torch.empty_like(res), ip.linear_workspace(p), ip.LinearGrads(p)
    outs = (y, pre, g.dx, g.dW, g.db)

    def both(stream=None):
        ip.ipttt_linear(p, x, W, y, b=b, res=res, pre=pre, ws=ws, stream=stream)
        ip.ipttt_linear_backward(p, x, W, dy, g.dx, g.dW, g.db, g.ws, pre=pre, stream=stream)

    both()
    want = [t.clone() for t in outs]
    for t in outs:
        t.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    both(side)
    side.synchronize()
    assert all(torch.equal(a, t) for a, t in zip(want, outs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for seed in (1, 2, 3):
        for t, v in zip((x, W, b, res, dy), inputs(BF16, m, k, n, seed)):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        both()
        assert all(torch.equal(a, t) for a, t in zip(got, outs))
