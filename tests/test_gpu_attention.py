"""GPU parity of the attention half against the fp64 definitions.

Tolerances (relative, over a whole tensor), derived from the roundings:
  bf16  an output's rounding and that of the probabilities (or their gradients)
        are each at most 2^-8 of the value they round, and below 2^-9 of a whole
        tensor's norm (their root mean square); the backward adds that of the
        stored O in delta.  Twice 2^-9 for the forward, four times 2^-9 for
        gradients bound their sums.
  fp32  fp32 sums of products of O(1) and exponents up to about 30, each
        rounded to 2^-24 of its size: 30 * 2^-24 in the exponent, times 4 for
        what else adds up: 1e-5 forward; the gradients' differences dP - delta
        lose another factor 2.
  lse   absolute: exponents up to 30 in fp32 give 30 * 2^-23 = 4e-6, times 4.
"""
import numpy as np
import pytest
import torch

import test_weight_mlp_amd as ip
from oracle import attention as oa

pytestmark = pytest.mark.gpu

BF16, F32 = ip.IPTTT_BF16, ip.IPTTT_F32
TDT = {BF16: torch.bfloat16, F32: torch.float32}
FWD = {BF16: 2 * 2.0 ** -9, F32: 1e-5}
BWD = {BF16: 4 * 2.0 ** -9, F32: 2e-5}
LSE = 1.6e-5


def rel(a, b):
    n = np.linalg.norm(b)
    return np.linalg.norm(a - b) / (n if n > 0 else 1.0)


def np64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def starts(lens):
    return np.concatenate([[0], np.cumsum(lens)[:-1]]).astype(int)


def draw(dt, heads, kv, dim, ql, kl, seed=0, layout="plain"):
    """q, k, v, do of a case.  layout: plain; fused (slices of one projection);
    heads (cache with the tokens of a head together)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(TDT[dt])

    nq, nk = sum(ql), sum(kl)
    if layout == "fused":
        x = randn(max(nq, nk), heads + 2 * kv, dim)
        return x[:nq, :heads], x[:nk, heads:heads + kv], x[:nk, heads + kv:], randn(nq, heads, dim)
    if layout == "heads":
        return (randn(heads, nq, dim).transpose(0, 1), randn(kv, nk, dim).transpose(0, 1),
                randn(kv, nk, dim).transpose(0, 1), randn(nq, heads, dim))
    return randn(nq, heads, dim) * 2, randn(nk, kv, dim), randn(nk, kv, dim), randn(nq, heads, dim)


def seqs_of(ql, kl):
    return list(zip(starts(ql), ql, starts(kl), kl))


def check_forward(dt, plan, q, k, v, ql, kl, buf):
    o, lse = oa.attention(np64(q), np64(k), np64(v), seqs_of(ql, kl), plan.scale)
    assert rel(np64(buf.o), o) <= FWD[dt]
    got = np64(buf.lse)
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(got), empty) and np.all(np64(buf.o)[empty] == 0)
    assert np.abs(got[~empty] - lse[~empty]).max(initial=0.0) <= LSE
    # every row on its own too: none hides behind the others' norm
    rows = np.linalg.norm(np64(buf.o) - o, axis=-1) / np.maximum(np.linalg.norm(o, axis=-1), 1e-30)
    assert rows[~empty].max(initial=0.0) <= 2 * FWD[dt]


SHAPES = [
    # heads, key heads, head width, query lengths, key lengths
    (1, 1, 8, [1], [1]),
    (4, 4, 64, [1, 2, 31], [1, 2, 31]),
    (8, 2, 128, [64, 65, 1, 127], [64, 65, 1, 127]),
    (6, 2, 80, [33, 130], [33, 130]),                # group of 3: tiles that cut a token's heads
    (5, 1, 40, [77], [77]),
    (7, 1, 72, [19, 200], [19, 200]),
    (12, 4, 96, [129], [300]),                       # a piece over what came before
    (4, 2, 120, [50, 9, 3], [20, 9, 70]),            # rows that see nothing
    (32, 8, 128, [1, 1, 5, 1], [1, 700, 1333, 5000]),  # single tokens, a few tokens; long axis split
    (32, 1, 64, [1, 3], [2500, 64]),
    (16, 8, 24, [4, 0, 6], [0, 5, 6]),               # no keys; no queries
    (3, 3, 104, [256], [256]),
    (8, 1, 64, [900, 3], [900, 3]),                  # dK, dV summed from several parts
    (128, 1, 32, [3, 41], [3, 90]),                  # a token's heads fill several tiles
    (2, 2, 128, [1, 300], [40, 300]),                # few rows over few keys beside many
    (4, 1, 128, [600], [600]),                       # delta from the keys and from O
]


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads,kv,dim,ql,kl", SHAPES)
def test_forward(dt, heads, kv, dim, ql, kl):
    q, k, v, _ = draw(dt, heads, kv, dim, ql, kl)
    plan = ip.AttentionPlan(heads, kv, dim, ql, kl, dt)
    buf = ip.AttentionBuffers(plan)
    ip.ipttt_attention(plan, q, k, v, buf.o, buf.lse, buf.ws)
    torch.cuda.synchronize()
    check_forward(dt, plan, q, k, v, ql, kl, buf)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads,kv,dim,ql,kl", SHAPES)
def test_backward(dt, heads, kv, dim, ql, kl):
    q, k, v, do = draw(dt, heads, kv, dim, ql, kl, seed=1)
    plan = ip.AttentionPlan(heads, kv, dim, ql, kl, dt)
    buf = ip.AttentionBuffers(plan, grads=True)
    ip.ipttt_attention(plan, q, k, v, buf.o, buf.lse, buf.ws)
    ip.ipttt_attention_backward(plan, q, k, v, buf.o, buf.lse, do, buf.dq, buf.dk, buf.dv, buf.ws)
    torch.cuda.synchronize()
    want = oa.attention_backward(np64(q), np64(k), np64(v), np64(do), seqs_of(ql, kl), plan.scale)
    for name, got, w in zip(("dq", "dk", "dv"), (buf.dq, buf.dk, buf.dv), want):
        got = np64(got)
        assert np.isfinite(got).all(), name
        assert rel(got, w) <= BWD[dt], name
        assert np.all(got[np.abs(w).max(-1) == 0] == 0), name   # rows without a gradient are exactly 0


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("layout", ["fused", "heads"])
def test_strided_layouts_give_the_same_bits(dt, layout):
    heads, kv, dim, ql, kl = 8, 2, 64, [70, 1, 130], [70, 1, 130]
    q, k, v, do = draw(dt, heads, kv, dim, ql, kl, seed=2, layout=layout)
    assert not q.is_contiguous()
    plan = ip.AttentionPlan(heads, kv, dim, ql, kl, dt)
    outs = []
    for x in ((q, k, v), tuple(t.contiguous() for t in (q, k, v))):
        b = ip.AttentionBuffers(plan, grads=True)
        ip.ipttt_attention(plan, *x, b.o, b.lse, b.ws)
        ip.ipttt_attention_backward(plan, *x, b.o, b.lse, do, b.dq, b.dk, b.dv, b.ws)
        torch.cuda.synchronize()
        outs.append((b.o, b.lse, b.dq, b.dk, b.dv))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    check = ip.AttentionBuffers(plan)
    check.o, check.lse = outs[0][:2]
    check_forward(dt, plan, q, k, v, ql, kl, check)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("q_len", [1, 40])
def test_a_cache_is_read_only_where_it_is_filled(dt, q_len):
    """Slots of a cache in any order, the rest of each slot NaN: nothing past
    k_len, between the slots or of another sequence reaches an output; a shared
    prefix is read by two sequences."""
    heads, kv, dim, kl = 8, 2, 128, [130, 1000, 63, 1000]
    ql, at = [q_len] * 4, [2000, 100, 1300, 100]
    q, k0, v0, _ = draw(dt, heads, kv, dim, ql, [3300], seed=3)
    k, v = torch.full_like(k0, float("nan")), torch.full_like(v0, float("nan"))
    for s, n in zip(at, kl):
        k[s:s + n], v[s:s + n] = k0[s:s + n], v0[s:s + n]
    plan = ip.AttentionPlan(heads, kv, dim, ql, kl, dt, k_starts=at, k_rows=3300)
    b = ip.AttentionBuffers(plan)
    ip.ipttt_attention(plan, q, k, v, b.o, b.lse, b.ws)
    torch.cuda.synchronize()
    seqs = list(zip(starts(ql), ql, at, kl))
    o, lse = oa.attention(np64(q), np64(k0), np64(v0), seqs, plan.scale)
    assert rel(np64(b.o), o) <= FWD[dt]
    assert np.abs(np64(b.lse) - lse).max() <= LSE


def test_rows_of_no_sequence_are_left_alone():
    heads, kv, dim = 4, 2, 64
    q, k, v, do = draw(BF16, heads, kv, dim, [40], [60], seed=4)
    plan = ip.AttentionPlan(heads, kv, dim, [5, 9], [7, 9], BF16, q_starts=[3, 20], k_starts=[30, 2], q_rows=40,
                            k_rows=60)
    b = ip.AttentionBuffers(plan, grads=True)
    for t in (b.o, b.lse, b.dq, b.dk, b.dv):
        t.fill_(7.0)
    ip.ipttt_attention(plan, q, k, v, b.o, b.lse, b.ws)
    ip.ipttt_attention_backward(plan, q, k, v, b.o, b.lse, do, b.dq, b.dk, b.dv, b.ws)
    torch.cuda.synchronize()
    seqs = [(3, 5, 30, 7), (20, 9, 2, 9)]
    want = (oa.attention(*(np64(t) for t in (q, k, v)), seqs, plan.scale) +
            oa.attention_backward(*(np64(t) for t in (q, k, v, do)), seqs, plan.scale))
    for got, w in zip((b.o, b.lse, b.dq, b.dk, b.dv), want):
        got, out = np64(got), np.isnan(w)
        assert np.all(got[out] == 7.0) and rel(got[~out], w[~out]) <= BWD[BF16]


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_extreme_scores(dt):
    """Scores of hundreds (one key takes all), equal scores, keys of -inf and of
    the type's lowest value in masked places, and a key whose score is -inf."""
    heads, kv, dim, ql, kl = 2, 1, 64, [70], [70]
    q, k, v, _ = draw(dt, heads, kv, dim, ql, kl, seed=5)
    big = (q * 16, k * 4, v)
    flat = (q * 0, k, v)
    for x in (big, flat):
        plan = ip.AttentionPlan(heads, kv, dim, ql, kl, dt)
        b = ip.AttentionBuffers(plan)
        ip.ipttt_attention(plan, *x, b.o, b.lse, b.ws)
        torch.cuda.synchronize()
        o, lse = oa.attention(*(np64(t) for t in x), seqs_of(ql, kl), plan.scale)
        # the exponents reach 1000 here: their fp32 rounding is 1000 * 2^-24 each way
        assert rel(np64(b.o), o) <= FWD[dt] + 1000 * 2.0 ** -23
        assert np.abs(np64(b.lse) - lse).max() <= 1000 * 2.0 ** -22
    # the last rows' keys are masked for all earlier rows
    for value in (float("-inf"), torch.finfo(TDT[dt]).min, float("nan")):
        kk = k.clone()
        kk[50:] = value
        b2 = ip.AttentionBuffers(plan)
        ip.ipttt_attention(plan, q, kk, v, b2.o, b2.lse, b2.ws)
        ref = ip.AttentionBuffers(plan)
        ip.ipttt_attention(plan, q, k, v, ref.o, ref.lse, ref.ws)
        torch.cuda.synchronize()
        assert torch.equal(b2.o[:50], ref.o[:50]) and torch.equal(b2.lse[:50], ref.lse[:50])
    # q.k = -inf for one visible key: it has no weight
    kk, qq = k.clone(), q.abs() + 0.1
    kk[3] = float("-inf")
    ip.ipttt_attention(plan, qq, kk, v, b.o, b.lse, b.ws)
    torch.cuda.synchronize()
    keep = [i for i in range(70) if i != 3]
    s = [(0, 66, 0, 69)]
    o, _ = oa.attention(np64(qq[4:]), np64(kk[keep]), np64(v[keep]), s, plan.scale)
    assert rel(np64(b.o[4:]), o) <= FWD[dt]


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_pieces_and_single_tokens_equal_the_prompt(dt):
    """A prompt read whole, in pieces and token by token gives the same outputs."""
    heads, kv, dim, n = 8, 2, 128, 300
    q, k, v, _ = draw(dt, heads, kv, dim, [n], [n], seed=6)

    def run(pieces):
        out = []
        end = 0
        for m in pieces:
            plan = ip.AttentionPlan(heads, kv, dim, [m], [end + m], dt, k_rows=n)
            b = ip.AttentionBuffers(plan)
            ip.ipttt_attention(plan, q[end:end + m], k, v, b.o, b.lse, b.ws)
            out.append(b.o)
            end += m
        torch.cuda.synchronize()
        return np64(torch.cat(out))

    whole = run([n])
    assert rel(run([128, 1, 100, 71]), whole) <= FWD[dt]
    assert rel(run([1] * n), whole) <= FWD[dt]


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_same_bits_every_run_and_on_any_stream(dt):
    heads, kv, dim, ql, kl = 8, 2, 64, [300, 1, 77], [300, 3000, 400]
    q, k, v, do = draw(dt, heads, kv, dim, ql, kl, seed=7)
    plan = ip.AttentionPlan(heads, kv, dim, ql, kl, dt)
    side, outs = torch.cuda.Stream(), []
    torch.cuda.synchronize()
    for st in (None, None, side):
        b = ip.AttentionBuffers(plan, grads=True)
        torch.cuda.synchronize()
        ip.ipttt_attention(plan, q, k, v, b.o, b.lse, b.ws, stream=st)
        ip.ipttt_attention_backward(plan, q, k, v, b.o, b.lse, do, b.dq, b.dk, b.dv, b.ws, stream=st)
        torch.cuda.synchronize()
        outs.append((b.o, b.lse, b.dq, b.dk, b.dv))
    for other in outs[1:]:
        for a, b in zip(outs[0], other):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """The last rows of a cache of 4.5 GB, read by a token and by a piece."""
    heads, kv, dim, rows = 16, 8, 128, 2_200_000
    cache = torch.zeros(rows, kv, dim, dtype=torch.bfloat16, device="cuda")
    n = 700
    q, k, v, _ = draw(BF16, heads, kv, dim, [41], [n], seed=8)
    cache[-2 * n:-n], cache[-n:] = k, v
    values = cache.view(-1)[n * kv * dim:].view(rows - n, kv, dim)     # row i of it is row i + n of the cache
    plan = ip.AttentionPlan(heads, kv, dim, [1, 40], [n - 200, n], BF16, k_starts=[rows - 2 * n] * 2,
                            k_rows=rows - n)
    b = ip.AttentionBuffers(plan)
    ip.ipttt_attention(plan, q, cache[:rows - n], values, b.o, b.lse, b.ws)
    torch.cuda.synchronize()
    o, lse = oa.attention(np64(q), np64(k), np64(v), [(0, 1, 0, n - 200), (1, 40, 0, n)], plan.scale)
    assert rel(np64(b.o), o) <= FWD[BF16]
    assert np.abs(np64(b.lse) - lse).max() <= LSE


def test_gradients_against_differences():
    """fp32: <dx, u> equals the central difference of <O, dO> along u, within the
    difference's own error: h^2 of third derivatives (h = 1e-2: about 1e-4 of the
    slope) plus the forward's rounding over h (1e-5 / 1e-2 of |O||dO|, a
    random sum of it)."""
    heads, kv, dim, ql, kl = 4, 2, 32, [37, 5], [37, 50]
    q, k, v, do = draw(F32, heads, kv, dim, ql, kl, seed=9)
    plan = ip.AttentionPlan(heads, kv, dim, ql, kl, F32)
    b = ip.AttentionBuffers(plan, grads=True)

    def loss(x):
        ip.ipttt_attention(plan, *x, b.o, b.lse, b.ws)
        return float((b.o.double() * do.double()).sum())

    base = [q, k, v]
    loss(base)
    ip.ipttt_attention_backward(plan, q, k, v, b.o, b.lse, do, b.dq, b.dk, b.dv, b.ws)
    grads = [t.double().clone() for t in (b.dq, b.dk, b.dv)]
    h = 1e-2
    for i, g in enumerate(grads):
        u = g.float() / g.float().norm()       # the steepest direction: the slope is |g|
        a = [t + h * u if j == i else t for j, t in enumerate(base)]
        c = [t - h * u if j == i else t for j, t in enumerate(base)]
        slope = (loss(a) - loss(c)) / (2 * h)
        assert abs(slope - float((g * u).sum())) <= 3e-3 * float(g.norm())


def test_graph_replays_equal_the_eager_calls():
    heads, kv, dim, ql, kl = 8, 2, 64, [33, 1], [33, 2000]
    q, k, v, do = draw(BF16, heads, kv, dim, ql, kl, seed=10)
    plan = ip.AttentionPlan(heads, kv, dim, ql, kl, BF16)
    b = ip.AttentionBuffers(plan, grads=True)

    def step():
        ip.ipttt_attention(plan, q, k, v, b.o, b.lse, b.ws)
        ip.ipttt_attention_backward(plan, q, k, v, b.o, b.lse, do, b.dq, b.dk, b.dv, b.ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (11, 12, 13):
        q2, k2, v2, do2 = draw(BF16, heads, kv, dim, ql, kl, seed=seed)
        for dst, src in zip((q, k, v, do), (q2, k2, v2, do2)):
            dst.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (b.o, b.lse, b.dq, b.dk, b.dv)]
        for t in (b.o, b.lse, b.dq, b.dk, b.dv):
            t.zero_()
        step()
        torch.cuda.synchronize()
        for x, y in zip(got, (b.o, b.lse, b.dq, b.dk, b.dv)):
            assert torch.equal(x, y)


# ------------------------------------------------------- norm and rotation

QK_SHAPES = [(1, 32, 8, 128), (5, 2, 1, 8), (37, 6, 6, 80), (130, 12, 4, 96), (9, 5, 5, 64), (63, 3, 1, 40),
             (1000, 16, 8, 64), (4099, 4, 2, 24), (2, 7, 7, 120)]


def draw_qk(dt, n, hq, hk, d, seed=0, positions=None):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = (torch.randn(n, hq + 2 * hk, d, generator=g, device="cuda") * 3).to(TDT[dt])
    w = [(1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(TDT[dt]) for _ in "qk"]
    table = ip.rotation_table(5000, d, 10000.0)
    pos = torch.randint(0, 5000, (n,), generator=g, device="cuda").to(torch.int32) if positions is None else positions
    dz = [torch.randn(n, h, d, generator=g, device="cuda").to(TDT[dt]) for h in (hq, hk)]
    return x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], w, table, pos, dz


# fp32: a sum of D squares and a few products, each 2^-24: 2e-6 of the head's
# norm.  bf16: one rounding more, at most 2^-8 of each value.
QK = {BF16: 2.0 ** -9, F32: 2e-6}


def check_rounded(dt, got, want):
    """Every value is its definition's, rounded once: within the rounding of that
    value and fp32's error on the scale of its head."""
    scale = np.linalg.norm(want, axis=-1, keepdims=True)
    once = 2.0 ** -8 if dt == BF16 else 0.0
    assert np.all(np.abs(got - want) <= once * np.abs(want) + QK[F32] * scale)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,hq,hk,d", QK_SHAPES)
def test_norm_rope(dt, n, hq, hk, d):
    q, k, v, w, table, pos, dz = draw_qk(dt, n, hq, hk, d)
    p = ip.QKProblem(n, hq, hk, d, dt, eps=1e-5, table_rows=5000)
    qo, ko = torch.empty(n, hq, d, dtype=TDT[dt], device="cuda"), torch.empty(n, hk, d, dtype=TDT[dt], device="cuda")
    ip.ipttt_qk_norm_rope(p, q, k, w[0], w[1], pos, table, qo, ko)
    torch.cuda.synchronize()
    at, tb = pos.cpu().numpy(), np64(table)
    for x, wx, got in ((q, w[0], qo), (k, w[1], ko)):
        want = oa.norm_rope(np64(x), np64(wx), at, tb, 1e-5)
        check_rounded(dt, np64(got), want)
    # in place, and on another stream: the same bits
    q2, k2 = q.clone(), k.clone()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    ip.ipttt_qk_norm_rope(p, q2, k2, w[0], w[1], pos, table, q2, k2, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(q2, qo) and torch.equal(k2, ko)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,hq,hk,d", QK_SHAPES)
def test_norm_rope_backward(dt, n, hq, hk, d):
    q, k, v, w, table, pos, dz = draw_qk(dt, n, hq, hk, d, seed=1)
    p = ip.QKProblem(n, hq, hk, d, dt, eps=1e-5, table_rows=5000)
    outs = []
    for _ in "ab":
        g = ip.QKGrads(p)
        ip.ipttt_qk_norm_rope_backward(p, q, k, w[0], w[1], pos, table, dz[0], dz[1], g.dq, g.dk, g.dw_q, g.dw_k, g.ws)
        torch.cuda.synchronize()
        outs.append((g.dq, g.dk, g.dw_q, g.dw_k))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    at, tb = pos.cpu().numpy(), np64(table)
    dq, dk, dw_q, dw_k = outs[0]
    for x, wx, z, dx, dw in ((q, w[0], dz[0], dq, dw_q), (k, w[1], dz[1], dk, dw_k)):
        want, want_w = oa.norm_rope_backward(np64(x), np64(wx), np64(z), at, tb, 1e-5)
        assert rel(np64(dx), want) <= 2 * QK[dt]
        assert rel(np64(dw), want_w) <= 2 * QK[F32]


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_norm_rope_into_a_cache(dt):
    """Keys and values go to their tokens' rows; a row outside the cache drops the
    token; every other row of the cache keeps its bits."""
    n, hq, hk, d, rows = 6, 4, 2, 64, 50
    q, k, v, w, table, pos, _ = draw_qk(dt, n, hq, hk, d, seed=2)
    at = torch.tensor([3, 49, 0, -1, 50, 17], dtype=torch.int32, device="cuda")
    p = ip.QKProblem(n, hq, hk, d, dt, table_rows=5000, out_rows=rows)
    kc, vc = (torch.full((rows, hk, d), 5.0, dtype=TDT[dt], device="cuda") for _ in "kv")
    qo = torch.empty(n, hq, d, dtype=TDT[dt], device="cuda")
    ip.ipttt_qk_norm_rope(p, q, k, w[0], w[1], pos, table, qo, kc, v=v, v_out=vc, rows=at)
    torch.cuda.synchronize()
    plain = ip.QKProblem(n, hq, hk, d, dt, table_rows=5000)
    qo2, ko2 = torch.empty_like(qo), torch.empty(n, hk, d, dtype=TDT[dt], device="cuda")
    ip.ipttt_qk_norm_rope(plain, q, k, w[0], w[1], pos, table, qo2, ko2)
    torch.cuda.synchronize()
    kept = [0, 1, 2, 5]
    to = at[kept].long()
    assert torch.equal(qo, qo2) and torch.equal(kc[to], ko2[kept]) and torch.equal(vc[to], v[kept])
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[to] = False
    assert bool((kc[rest] == 5.0).all()) and bool((vc[rest] == 5.0).all())


def test_norm_rope_position_outside_the_table_is_nan():
    pos = torch.tensor([0, 5000, -1, 4999], dtype=torch.int32, device="cuda")
    q, k, v, w, table, _, _ = draw_qk(BF16, 4, 2, 1, 64, positions=pos)
    p = ip.QKProblem(4, 2, 1, 64, BF16, table_rows=5000)
    qo, ko = torch.empty(4, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(4, 1, 64, dtype=torch.bfloat16,
                                                                                     device="cuda")
    ip.ipttt_qk_norm_rope(p, q, k, w[0], w[1], pos, table, qo, ko)
    torch.cuda.synchronize()
    for t in (qo, ko):
        assert bool(torch.isnan(t[1:3]).all()) and bool(torch.isfinite(t[[0, 3]]).all())


@pytest.mark.parametrize("heads,kv,dim,lens", [(6, 6, 80, [17, 3]), (32, 8, 128, [9]), (16, 8, 64, [40, 5]),
                                               (8, 2, 128, [120]), (16, 8, 64, [300, 30]), (8, 1, 96, [700])])
def test_fp32_gradients_are_as_near_as_the_plain_form(heads, kv, dim, lens):
    """fp32 gradients, against the definition in 64 bits, are no more than twice as
    far off (in the Frobenius norm) as the formulas in 32-bit torch operations: the
    same roundings in another order differ by less, one rounding at a larger
    magnitude by more."""
    plan = ip.AttentionPlan(heads, kv, dim, lens, lens, dtype=ip.IPTTT_F32)
    gen = torch.Generator(device="cuda").manual_seed(sum(lens) + dim)
    n, G = sum(lens), heads // kv
    q, do = (torch.randn(n, heads, dim, device="cuda", generator=gen) for _ in "ab")
    k, v = (torch.randn(n, kv, dim, device="cuda", generator=gen) for _ in "ab")
    b = ip.AttentionBuffers(plan, grads=True)
    ip.ipttt_attention(plan, q, k, v, b.o, b.lse, b.ws)
    ip.ipttt_attention_backward(plan, q, k, v, b.o, b.lse, do, b.dq, b.dk, b.dv, b.ws)

    def plain(dtype):
        dq, dk, dv = torch.zeros_like(q, dtype=dtype), torch.zeros_like(k, dtype=dtype), torch.zeros_like(v, dtype=dtype)
        t0 = 0
        for length in lens:
            at = slice(t0, t0 + length)
            t0 += length
            hidden = torch.ones(length, length, dtype=torch.bool, device="cuda").triu(1)
            for head in range(heads):
                x, y, z, d = (t[at, i].to(dtype) for t, i in ((q, head), (k, head // G), (v, head // G), (do, head)))
                w = torch.softmax((x @ y.T * plan.scale).masked_fill(hidden, -float("inf")), -1)
                dw = d @ z.T
                ds = w * (dw - (w * dw).sum(-1, keepdim=True)) * plan.scale
                dq[at, head] = ds @ y
                dk[at, head // G] += ds.T @ x
                dv[at, head // G] += w.T @ d
        return dq, dk, dv

    for name, got, near, want in zip(("dq", "dk", "dv"), (b.dq, b.dk, b.dv), plain(torch.float32), plain(torch.float64)):
        ours, theirs = ((t.double() - want).norm().item() for t in (got, near))
        print(f"{name} {ours / want.norm().item():.2e} plain {theirs / want.norm().item():.2e}")
        assert ours <= 2 * theirs, name


@pytest.mark.parametrize("heads,kv,dim,lens", [(2, 1, 32, [3]), (32, 8, 128, [9]), (16, 8, 64, [2, 5, 1]), (5, 5, 64, [30]),
                                               (8, 1, 128, [4, 32]), (6, 6, 80, [12])])
def test_bf16_gradients_of_short_sequences(heads, kv, dim, lens):
    """Few probabilities do not average their roundings, so calls of short sequences
    round P and dS to 16 bits: what is left, in the Frobenius norm, is the gradients'
    own rounding to bf16, here within a quarter of it."""
    q, k, v, do = draw(BF16, heads, kv, dim, lens, lens, seed=sum(lens))
    plan = ip.AttentionPlan(heads, kv, dim, lens, lens)
    b = ip.AttentionBuffers(plan, grads=True)
    ip.ipttt_attention(plan, q, k, v, b.o, b.lse, b.ws)
    ip.ipttt_attention_backward(plan, q, k, v, b.o, b.lse, do, b.dq, b.dk, b.dv, b.ws)
    torch.cuda.synchronize()
    want = oa.attention_backward(*(np64(t) for t in (q, k, v, do)), seqs_of(lens, lens), plan.scale)
    for name, got, w in zip(("dq", "dk", "dv"), (b.dq, b.dk, b.dv), want):
        own = np64(torch.from_numpy(w).to(torch.bfloat16)) - w
        ratio = np.linalg.norm(np64(got) - w) / np.linalg.norm(own)
        print(f"{name} {ratio:.3f}")
        assert ratio <= 1.25, name


# ------------------------------------------------------------------ binding

def _without(t, how):
    """t with one thing about it made wrong."""
    return {"shape": lambda: t[:-1], "type": lambda: t.double(), "host": lambda: t.cpu(), "kind": lambda: [0.0],
            "rank": lambda: t[None], "strides": lambda: torch.stack([t, t], -1)[..., 0]}[how]()


@pytest.mark.parametrize("how", ["shape", "type", "host", "kind", "rank", "strides"])
def test_binding_refuses_tensors(how):
    """Every tensor of every call is checked: nothing is launched, and the message
    names the tensor."""
    T, H, KV, D, bf, dev = 4, 4, 2, 64, torch.bfloat16, "cuda"
    z = lambda *s, t=bf: torch.zeros(s, dtype=t, device=dev)
    p = ip.QKProblem(T, H, KV, D, table_rows=6)
    plan = ip.AttentionPlan(H, KV, D, [T], [T])
    base = dict(q=z(T, H, D), k=z(T, KV, D), w_q=z(D), w_k=z(D), positions=z(T, t=torch.int32),
                table=z(6, D, t=torch.float32))
    qk = dict(base, q_out=z(T, H, D), k_out=z(T, KV, D), v=z(T, KV, D), v_out=z(T, KV, D),
              rows=torch.arange(T, dtype=torch.int32, device=dev))
    g = ip.QKGrads(p)
    back = dict(base, dq_out=z(T, H, D), dk_out=z(T, KV, D), dq=g.dq, dk=g.dk, dw_q=g.dw_q, dw_k=g.dw_k, ws=g.ws)
    fwd = dict(q=z(T, H, D), k=z(T, KV, D), v=z(T, KV, D), o=z(T, H, D), lse=z(T, H, t=torch.float32))
    b = ip.AttentionBuffers(plan, grads=True)
    bwd = dict(fwd, dO=z(T, H, D), dq=b.dq, dk=b.dk, dv=b.dv, ws=b.ws)
    here = torch.cuda.current_stream()
    for call, args in ((lambda **a: ip.ipttt_qk_norm_rope(p, **a, stream=here), qk),
                       (lambda **a: ip.ipttt_qk_norm_rope_backward(p, **a, stream=here), back),
                       (lambda **a: ip.ipttt_attention(plan, **a, stream=here), fwd),
                       (lambda **a: ip.ipttt_attention_backward(plan, **a, stream=here), bwd)):
        call(**args)
        for name, t in args.items():
            if t is None or (name == "ws" and how in ("shape", "type", "rank")):   # any memory of enough bytes will do
                continue
            with pytest.raises(TypeError if how == "kind" else ValueError, match=rf"^{name} must be"):
                call(**dict(args, **{name: _without(t, how)}))
    torch.cuda.synchronize()
