"""GPU parity of the attention half where a call's company, its size or its values
choose another path than test_gpu_attention.py's shapes do; draws, definitions and
tolerances are those of that file."""
import numpy as np
import pytest
import torch

import test_weight_mlp_amd as ip
from oracle import attention as oa
from test_gpu_attention import BF16, draw, draw_qk, np64, seqs_of, starts

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
