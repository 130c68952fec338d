"""GPU parity of the gated products kept in 8 bits against the fp64 definitions.

What is kept is checked through the gradients' linearity: with dZ one where a
feature is asked for and zero elsewhere dU = SiLU(G) dZ and dG = U SiLU'(G) dZ come
out in dH through weights of the unit matrix, so the kept values can be read
back.  Bounds: a kept value is a multiple of max / 127, so it is off by at most half
of that, plus the bf16 rounding of the product (2^-8 of its size) and, where that
or fp32's own rounding moves a value across a tie, nothing more than those again.
"""
import numpy as np
import pytest
import torch

import test_weight_mlp_amd as ip
from block_helpers import HALF, BF16, generator, np64, randn
from oracle import block as ob

pytestmark = pytest.mark.gpu


def rel(got, want):
    return np.linalg.norm(np64(got) - want) / np.linalg.norm(want)


def inputs(t, d, f, seed=0):
    g = generator(seed)
    return randn(g, BF16, t, d), randn(g, BF16, f, d, scale=d ** -0.5), randn(g, BF16, f, d, scale=d ** -0.5), randn(g, BF16, t, f)


def run(p, H, Wg, Wu, dZ, kept=None, stream=None):
    Z = torch.full((p.tokens, p.d_ff), 5.0, dtype=torch.bfloat16, device="cuda")
    kept = torch.full((ip.ipttt_saved8_bytes(p),), 0x55, dtype=torch.uint8, device="cuda") if kept is None else kept
    g = ip.Grads(p)
    ip.ipttt_z_save8(p, H, Wg, Wu, Z, kept, stream)
    ip.ipttt_z_backward_saved8(p, H, Wg, Wu, kept, dZ, g.dH, g.dW_gate, g.dW_up, g.ws, stream)
    return Z, kept, g


def definition(H, Wg, Wu, dZ):
    H, Wg, Wu, dZ = (np64(x) for x in (H, Wg, Wu, dZ))
    G, U = H @ Wg.T, H @ Wu.T
    Z = ob.act("silu", G) * U
    as_bf16 = lambda x: torch.from_numpy(x).bfloat16().double().numpy()  # noqa: E731
    G, U = ob.kept8(as_bf16(G)), ob.kept8(as_bf16(U))
    dG, dU = dZ * U * ob.slope("silu", G), dZ * ob.act("silu", G)
    return Z, dG @ Wg + dU @ Wu, dG.T @ H, dU.T @ H


# d and f of the 8-wave kernels (multiples of 64) and of the general ones; a last
# block of 8, 16, 56 features; one token; several tiles
SHAPES = [(1, 64, 64), (5, 64, 256), (200, 128, 320), (130, 72, 200), (257, 320, 448), (33, 64, 72), (70, 200, 520),
          (129, 64, 120), (600, 256, 640)]


@pytest.mark.parametrize("t, d, f", SHAPES)
def test_gradients_from_kept_values(t, d, f):
    p = ip.Problem(1, t, d, f, 64)
    H, Wg, Wu, dZ = inputs(t, d, f, seed=t)
    Z, _, g = run(p, H, Wg, Wu, dZ)
    want = definition(H, Wg, Wu, dZ)
    plain = torch.empty_like(Z)
    ip.ipttt_z(p, H, Wg, Wu, plain)
    assert torch.equal(Z, plain)
    # two roundings (dG, dU as operands, and dH's own) of 2^-9 each, and what a
    # value pushed across a tie changes: a step of 2 / 127 of its block's largest
    # in some 1e-3 of the values, below 2^-10
    for got, w in zip((g.dH, g.dW_gate, g.dW_up), want[1:]):
        assert rel(got, w) <= 1.5 * 2.0 ** -9 + 2.0 ** -10


# tiles of 8 waves in the forward; the large launches of the gradients: dH of 8 waves, of 4
# and of small tiles, with the last tiles cut along K; the weights' gradients of 8 waves in
# several rounds, with the last ones cut, and of 4
@pytest.mark.parametrize("t, d, f", [(20000, 64, 640), (5000, 320, 1096), (3480, 4776, 464), (7248, 1088, 336),
                                     (3080, 1296, 744), (72, 3824, 4056), (856, 5600, 1520), (872, 1000, 8304),
                                     (752, 5424, 672)])
def test_large_launches(t, d, f):
    test_gradients_from_kept_values(t, d, f)


@pytest.mark.parametrize("d, f", [(64, 64), (64, 192), (72, 72)])
def test_kept_values_themselves(d, f):
    """H = rows of the unit matrix reads W's columns: G[t, j] = W_gate[j, t], exact in
    bf16.  dW_up = dU^T H = (dZ SiLU(kept G))^T, one token a column."""
    p = ip.Problem(1, d, d, f, 64)
    g = generator(3)
    H = torch.eye(d).bfloat16().cuda()
    Wg, Wu = randn(g, BF16, f, d, scale=2.0), randn(g, BF16, f, d)
    dZ = torch.ones(d, f, dtype=torch.bfloat16, device="cuda")
    _, _, grads = run(p, H, Wg, Wu, dZ)
    G, U = ob.kept8(np64(Wg).T), ob.kept8(np64(Wu).T)
    silu, gate = ob.act("silu", G), U * ob.slope("silu", G)
    # the operands' rounding, and 2^-20 for the fp32 arithmetic of SiLU and the scale
    for got, w in ((grads.dW_up, silu), (grads.dW_gate, gate)):
        assert (np.abs(np64(got).T - w) <= (HALF[BF16] + 2.0 ** -20) * np.abs(w) + 1e-6 * np.abs(w).max()).all()


def kept_parts(kept, t, f):
    """G's integers and scales."""
    room = lambda n: -(-n // 256) * 256  # noqa: E731
    n, blocks = room(t * f), -(-f // 64)
    q = kept[:t * f].view(torch.int8).view(t, f).cpu().numpy().astype(np.float64)
    scale = kept[2 * n:2 * n + t * blocks * 4].view(torch.float32).view(t, blocks).cpu().numpy().astype(np.float64)
    return q, scale


def unit_rows(d, Wg):
    """Tokens that read W_gate's columns (0 times an infinity is a NaN, so the
    feature of one that is not finite has no finite token)."""
    p = ip.Problem(1, d, d, d, 64)
    Wu = torch.ones(d, d, dtype=torch.bfloat16, device="cuda")
    dZ = torch.ones(d, d, dtype=torch.bfloat16, device="cuda")
    _, kept, grads = run(p, torch.eye(d).bfloat16().cuda(), Wg, Wu, dZ)
    return kept_parts(kept, d, d), grads


def check_blocks(q, scale, W):
    """Finite blocks: multiples to 127 of the scale, off by half a scale at most."""
    d = len(W)
    top = np.abs(W).reshape(d, -1, 64).max(-1).repeat(64, 1)
    values = q * np.repeat(scale, 64, 1)
    assert (np.abs(q) <= 127).all() and (np.abs(values - W) <= top * (0.5 / 127 + 2.0 ** -22) + 2.0 ** -100).all()


def test_blocks_of_infinities_and_nans_are_nans():
    d = 256
    Wg = randn(generator(4), BF16, d, d)
    Wg[70, 1], Wg[130, 2] = float("inf"), float("nan")
    (q, scale), grads = unit_rows(d, Wg)
    assert np.isnan(scale[:, 1:3]).all() and np.isfinite(scale[:, [0, 3]]).all() and not q[:, 64:192].any()
    keep = np.r_[0:64, 192:256]
    check_blocks(q[:, keep], scale[:, [0, 3]], np64(Wg).T[:, keep])
    # the features of a NaN block have NaN gradients, the others do not
    dW = np64(grads.dW_up)
    assert np.isnan(dW[64:192]).all() and np.isfinite(dW[keep]).all()


def test_blocks_of_zeros_and_of_the_types_ends():
    d = 256
    Wg = randn(generator(4), BF16, d, d)
    Wg[0:64, 0] = 0.0
    Wg[64:128, 0] *= 1e-35                      # below 2^-100: zeros
    Wg[128:192, 0] *= 2.0 ** -90
    Wg[0:64, 1] *= 2.0 ** 100
    Wg[64:128, 1] = torch.finfo(torch.bfloat16).max
    Wg[64, 1] = -Wg[64, 1]
    Wg[128:192, 1] = 1e-38                      # one large value beside values that vanish next to it
    Wg[130, 1] = 1.0
    (q, scale), _ = unit_rows(d, Wg)
    assert not q[0, :128].any() and not scale[0, :2].any() and np.isfinite(scale).all()
    assert (np.abs(q[1, 64:128]) == 127).all() and q[1, 64] == -127 and q[1, 130] == 127 and np.abs(q[1, 128:192]).sum() == 127
    check_blocks(q, scale, np64(Wg).T)


def test_a_token_does_not_depend_on_the_others():
    t, d, f = 300, 128, 192
    H, Wg, Wu, _ = inputs(t, d, f)
    p, one = ip.Problem(1, t, d, f, 64), ip.Problem(1, 1, d, f, 64)
    kept, alone = (torch.empty(ip.ipttt_saved8_bytes(x), dtype=torch.uint8, device="cuda") for x in (p, one))
    Z, Z1 = torch.empty(t, f, dtype=torch.bfloat16, device="cuda"), torch.empty(1, f, dtype=torch.bfloat16, device="cuda")
    ip.ipttt_z_save8(p, H, Wg, Wu, Z, kept)
    for i in (0, 77, 299):
        ip.ipttt_z_save8(one, H[i:i + 1], Wg, Wu, Z1, alone)
        assert torch.equal(kept[i * f:(i + 1) * f], alone[:f]) and torch.equal(Z[i], Z1[0])


def test_whole_layer_through_forward_and_backward():
    """allocate(keep8=True): the layer's outputs are those of the products kept whole;
    the gate's and up's gradients differ by what 8 bits lose: rounding errors of
    1 / sqrt(12) steps of max / 127, some 0.6 % of each value's root mean square in
    normal blocks of 64, through slopes of order one: 2 %."""
    t, d, f = 400, 128, 320
    g = generator(9)
    H, X0 = randn(g, BF16, t, d), randn(g, BF16, t, d)
    W = [randn(g, BF16, f, d, scale=d ** -0.5), randn(g, BF16, f, d, scale=d ** -0.5), randn(g, BF16, d, f, scale=f ** -0.5),
         randn(g, BF16, d, 5, scale=0.2), randn(g, BF16, d, d, scale=d ** -0.5)]
    p = ip.Problem(2, 200, d, f, 32, doc_starts=[70, 250])
    dO = randn(g, BF16, t, d)
    got = []
    for keep8 in (False, True):
        buf = ip.allocate(p, save=True, keep8=keep8)
        ip.forward(p, H, X0, *W, 0.01, 1.0, buf)
        got.append((buf.O.clone(), ip.backward(p, buf, H, X0, *W, 0.01, 1.0, dO)))
    assert torch.equal(got[0][0], got[1][0])
    a, b = got[0][1], got[1][1]
    for name in ("dX0", "dW_down", "dconv_w", "dW_target"):
        assert torch.equal(getattr(a, name), getattr(b, name))
    for name in ("dH", "dW_gate", "dW_up"):
        assert 0 < rel(getattr(b, name), np64(getattr(a, name))) <= 0.02


def test_bytes_behind_the_buffer_and_inputs_stay():
    t, d, f = 70, 64, 200
    p = ip.Problem(1, t, d, f, 64)
    H, Wg, Wu, dZ = inputs(t, d, f)
    n = ip.ipttt_saved8_bytes(p)
    room = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    run(p, H, Wg, Wu, dZ, kept=room[:n])
    assert bool((room[n:] == 0x5A).all())


def test_streams_and_graphs():
    t, d, f = 300, 128, 192
    p = ip.Problem(1, t, d, f, 64).prepare_segments()
    H, Wg, Wu, dZ = inputs(t, d, f)
    Z, kept, g = run(p, H, Wg, Wu, dZ)
    want = [x.clone() for x in (Z, g.dH, g.dW_gate, g.dW_up)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Z2, _, g2 = run(p, H, Wg, Wu, dZ, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (Z2, g2.dH, g2.dW_gate, g2.dW_up)))
    graph = torch.cuda.CUDAGraph()

    def both():
        ip.ipttt_z_save8(p, H, Wg, Wu, Z, kept)
        ip.ipttt_z_backward_saved8(p, H, Wg, Wu, kept, dZ, g.dH, g.dW_gate, g.dW_up, g.ws)

    with torch.cuda.graph(graph):
        both()
    for seed in (1, 2, 3):
        for x, v in zip((H, Wg, Wu, dZ), inputs(t, d, f, seed)):
            x.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (Z, g.dH, g.dW_gate, g.dW_up)]
        both()
        assert all(torch.equal(a, b) for a, b in zip(got, (Z, g.dH, g.dW_gate, g.dW_up)))


def unit_kept(W):
    """The integers and scales of G = W^T [tokens = inputs, features], U = W^T beside it."""
    f, d = W.shape
    p = ip.Problem(1, d, d, f, 64)
    Z = torch.empty(d, f, dtype=torch.bfloat16, device="cuda")
    kept = torch.empty(ip.ipttt_saved8_bytes(p), dtype=torch.uint8, device="cuda")
    ip.ipttt_z_save8(p, torch.eye(d).bfloat16().cuda(), W, W, Z, kept)
    return kept_parts(kept, d, f)


def nearest(W):
    """The definition's integers of G = W^T."""
    g = np64(W).T
    top = np.repeat(np.abs(g).reshape(len(g), -1, 64).max(-1), 64, 1)
    return np.rint(g * 127.0 / np.where(top > 0, top, 1.0))


@pytest.mark.parametrize("d", [256, 4096])   # tiles of 4 and of 8 waves
def test_every_integer_is_the_nearest_and_ties_are_even(d):
    W = randn(generator(6), BF16, d, d)
    half = torch.arange(64, device="cuda") + 0.5
    n = d // 64
    for t in range(128):       # token t: a largest of each significand, halves of its steps beside it
        top = 1 + t / 128
        step = 2.0 ** (t % 40 - 20)
        block = W[64 * (t % n):64 * (t % n) + 64, t]
        block.copy_((torch.where(half.long() % 3 == 0, -1, 1) * half * (top / 127 if t == 126 else top / 128) * step).bfloat16())
        block[0], block[1], block[2] = top * step, top / 2 * step, -top / 2 * step
    q, scale = unit_kept(W)
    want = nearest(W)
    assert np.isfinite(scale).all() and np.array_equal(q, want)
    values = np64(W).T * 127 / np.repeat(np.abs(np64(W).T).reshape(d, -1, 64).max(-1), 64, 1)
    assert (np.abs(values[126]) % 1 == 0.5).sum() >= 60    # the ties are there
