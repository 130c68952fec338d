"""GPU parity of the attention half where a call's company, its size or its values
choose another path than test_gpu_attention.py's shapes do; draws, definitions and
tolerances are those of that file."""
import numpy as np
import pytest
import torch

import test_weight_mlp_amd as ip
from oracle import attention as oa
from test_attention_host import Plan
from test_gpu_attention import BF16, F32, check_forward, draw, draw_qk, np64, rel, seqs_of, starts

pytestmark = pytest.mark.gpu


def step(plan, q, k, v, do):
    b = ip.AttentionBuffers(plan, grads=True)
    ip.ipttt_attention(plan, q, k, v, b.o, b.lse, b.ws)
    ip.ipttt_attention_backward(plan, q, k, v, b.o, b.lse, do, b.dq, b.dk, b.dv, b.ws)
    torch.cuda.synchronize()
    return b


@pytest.mark.parametrize("heads,kv,dim,lens,idle", [
    (32, 8, 128, [9] * 20, 0),              # more workgroups than CUs
    (16, 8, 64, [3, 12] * 30, 0),
    (2, 1, 32, [5, 40], 0),                 # beside sequences of more keys
    (32, 8, 128, [9, 700, 3, 33], 0),
    (8, 1, 96, [20, 300, 2], 0),
    (16, 8, 64, [7, 4], 500),               # beside keys without queries
])
def test_bf16_gradients_of_short_sequences_do_not_depend_on_their_company(heads, kv, dim, lens, idle):
    """What is left of a short sequence's gradients' errors, in the Frobenius norm, is
    their own rounding to bf16, here within a quarter of it, whatever it is packed
    with: sequences of up to 32 keys round P and dS to 16 bits."""
    ql, kl = lens + [0] * bool(idle), lens + [idle] * bool(idle)
    q, k, v, do = draw(BF16, heads, kv, dim, ql, kl, seed=sum(lens))
    b = step(ip.AttentionPlan(heads, kv, dim, ql, kl), q, k, v, do)
    want = oa.attention_backward(*(np64(t) for t in (q, k, v, do)), seqs_of(ql, kl), dim ** -0.5)
    short = np.concatenate([np.arange(s, s + n) for s, n in zip(starts(lens), lens) if n <= 32])
    for name, got, w in zip(("dq", "dk", "dv"), (b.dq, b.dk, b.dv), want):
        own = np64(torch.from_numpy(w).to(torch.bfloat16)) - w
        ratio = np.linalg.norm((np64(got) - w)[short]) / np.linalg.norm(own[short])
        print(f"{name} {ratio:.3f}")
        assert ratio <= 1.25, name


def test_norm_rope_into_no_rows():
    """A cache of no rows drops every key and value; the queries are as ever."""
    n, hq, hk, d = 5, 4, 2, 64
    q, k, v, w, table, pos, _ = draw_qk(BF16, n, hq, hk, d)
    none, at = torch.empty(0, hk, d, dtype=q.dtype, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    out, want = (torch.empty(n, hq, d, dtype=q.dtype, device="cuda") for _ in "ab")
    ip.ipttt_qk_norm_rope(ip.QKProblem(n, hq, hk, d, BF16, table_rows=5000), q, k, w[0], w[1], pos, table, want,
                          torch.empty(n, hk, d, dtype=q.dtype, device="cuda"))
    ip.ipttt_qk_norm_rope(ip.QKProblem(n, hq, hk, d, BF16, table_rows=5000, out_rows=0), q, k, w[0], w[1], pos, table, out,
                          none, v=v, v_out=none, rows=at)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# heads, key heads, width, query and key lengths, and what the plan does with them:
# a backward of 512 tiles and more (tiles of rows whole, those of keys cut), a forward
# of two workgroups a CU (folded order), tiles of many rows cut at narrow widths
REGIMES = [
    (32, 8, 64, [1800], [1800], "many folded"),
    (16, 16, 128, [2050], [2050], "many"),
    (32, 8, 128, [700, 600, 500], [700, 600, 500], "many"),
    (16, 8, 64, [300, 700], [4000, 700], "cut"),
    (16, 8, 32, [300], [5000], "cut"),
]
# Rounding to bf16 is off by 1.7e-3 of a tensor's norm.  O is rounded once and made of
# rounded P: sqrt(2) times that.  A gradient the same, of dS or P, and bf16's O goes
# into delta of rows of many keys.  A quarter more than sqrt(2) times 1.7e-3.
NEAR = {BF16: 3.0e-3, F32: 2e-5}


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads,kv,dim,ql,kl,regime", REGIMES)
def test_regimes_of_large_calls(dt, heads, kv, dim, ql, kl, regime):
    plan = ip.AttentionPlan(heads, kv, dim, ql, kl, dt)
    pl = Plan(plan)
    if "many" in regime:
        assert pl.h["n_dq_join"] == 0 and pl.h["n_key_join"] > 0
    if "folded" in regime:
        assert 256 < len(pl.rows) * kv <= 512
    if "cut" in regime:
        assert any(x["part"] >= 0 for x in pl.rows)
    q, k, v, do = draw(dt, heads, kv, dim, ql, kl, seed=21)
    b = step(plan, q, k, v, do)
    check_forward(dt, plan, q, k, v, ql, kl, b)
    want = oa.attention_backward(*(np64(t) for t in (q, k, v, do)), seqs_of(ql, kl), plan.scale)
    for name, got, w in zip(("dq", "dk", "dv"), (b.dq, b.dk, b.dv), want):
        print(f"{name} {rel(np64(got), w):.2e}")
        assert rel(np64(got), w) <= NEAR[dt], name


@pytest.mark.parametrize("heads,kv,dim,lens", [(8, 2, 64, [40] * 12), (4, 1, 128, [64, 50, 33]), (8, 8, 64, [130, 48])])
def test_delta_of_few_keys_does_not_take_the_rounding_of_o(heads, kv, dim, lens):
    """dQ of bf16 sequences of 33 keys and more: dS's rounding and its own, sqrt(2)
    times the latter, and a tenth more; with bf16's O in delta it is twice the latter."""
    q, k, v, do = draw(BF16, heads, kv, dim, lens, lens, seed=22)
    b = step(ip.AttentionPlan(heads, kv, dim, lens, lens), q, k, v, do)
    want = oa.attention_backward(*(np64(t) for t in (q, k, v, do)), seqs_of(lens, lens), dim ** -0.5)[0]
    own = np64(torch.from_numpy(want).to(torch.bfloat16)) - want
    ratio = np.linalg.norm(np64(b.dq) - want) / np.linalg.norm(own)
    print(f"dq {ratio:.3f}")
    assert ratio <= 1.1 * 2 ** 0.5


def test_graph_replays_of_short_and_long_sequences_equal_the_eager_calls():
    heads, kv, dim, lens = 8, 2, 128, [9, 300, 1, 32]
    q, k, v, do = draw(BF16, heads, kv, dim, lens, lens, seed=30)
    plan = ip.AttentionPlan(heads, kv, dim, lens, lens)
    b = step(plan, q, k, v, do)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ip.ipttt_attention(plan, q, k, v, b.o, b.lse, b.ws)
        ip.ipttt_attention_backward(plan, q, k, v, b.o, b.lse, do, b.dq, b.dk, b.dv, b.ws)
    for seed in (31, 32, 33):
        for dst, src in zip((q, k, v, do), draw(BF16, heads, kv, dim, lens, lens, seed=seed)):
            dst.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        want = step(plan, q, k, v, do)
        for x in ("o", "lse", "dq", "dk", "dv"):
            assert torch.equal(getattr(b, x), getattr(want, x)), x
