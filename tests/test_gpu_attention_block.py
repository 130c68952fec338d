"""The example block: the attention half and the In-Place TTT layer together,
as a prompt, in pieces, token by token and as a training step."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


@pytest.fixture(scope="module")
def small():
    import attention_block as ab
    return ab, ab.Block(d=128, f=256, heads=8, kv_heads=2, head_dim=32, chunk=16, positions=512, dtype=torch.float32)


def plain(block, x, docs):
    """The block's attention half in 64 bits, up to the layer's input."""
    from oracle import attention as oa
    import attention_block as ab
    x64 = x.double()
    n = x64 * torch.rsqrt(x64.square().mean(-1, keepdim=True) + ab.EPS)
    t = len(x)
    qkv = (n @ block.W_qkv.double().T).view(t, block.hq + 2 * block.hk, block.D).cpu().numpy()
    pos = torch.cat([torch.arange(m) for m in docs]).numpy()
    table = block.table.double().cpu().numpy()
    q = oa.norm_rope(qkv[:, :block.hq], block.w_q.double().cpu().numpy(), pos, table, ab.EPS)
    k = oa.norm_rope(qkv[:, block.hq:block.hq + block.hk], block.w_k.double().cpu().numpy(), pos, table, ab.EPS)
    s = ab.starts(docs)
    o, _ = oa.attention(q, k, qkv[:, block.hq + block.hk:], list(zip(s, docs, s, docs)), block.D ** -0.5)
    return torch.from_numpy(o).cuda().view(t, -1)


def test_attention_half_equals_the_definition(small):
    ab, block = small
    x = torch.randn(96, block.d, device="cuda")
    docs = [40, 1, 55]
    plan = ab.ip.AttentionPlan(block.hq, block.hk, block.D, docs, docs, block.code)
    pos = torch.cat([torch.arange(n, dtype=torch.int32, device="cuda") for n in docs])
    a = ab.AttentionHalf.apply(ab.norm(x) @ block.W_qkv.T, block.w_q, block.w_k, pos, block.table, plan,
                               block.qk_problem(96))
    # fp32 throughout, library products included: a few 1e-6, an order to spare
    assert rel(a, plain(block, x, docs)) <= 5e-5


def test_pieces_and_tokens_equal_the_prompt(small):
    ab, block = small
    c = block.chunk
    x = torch.randn(6 * c, block.d, device="cuda")
    with torch.no_grad():
        whole = block.prompt(x, [len(x)])
    cache = block.cache(len(x) + 5)
    pieces = torch.cat([block.step(p, cache) for p in (x[:c], x[c:4 * c], x[4 * c:])])
    assert rel(pieces, whole) <= 5e-5
    cache = block.cache(len(x) + 5)
    block.step(x[:5 * c], cache)
    tail = torch.cat([block.step(x[i:i + 1], cache, fold=False) for i in range(5 * c, 5 * c + 7)])
    assert rel(tail, whole[5 * c:5 * c + 7]) <= 5e-5


def test_documents_do_not_mix(small):
    ab, block = small
    x = torch.randn(5 * block.chunk, block.d, device="cuda")
    docs = [33, 30, 17]
    with torch.no_grad():
        a = block.prompt(x, docs)
        y = x.clone()
        y[33:63] = torch.randn(30, block.d, device="cuda")
        b = block.prompt(y, docs)
    assert torch.equal(a[:33], b[:33]) and not torch.equal(a[33:63], b[33:63])


def test_training_step_against_differences(small):
    """<gradient, u> against the block's output along u (fp32: the difference of a
    sum of 96 * 128 terms at a step of 1e-2 is good to a few 1e-3 of |gradient|)."""
    ab, block = small
    x, dy = torch.randn(96, block.d, device="cuda"), torch.randn(96, block.d, device="cuda")
    docs = [50, 46]
    _, grads = ab.train_step(block, x, docs, dy)

    def loss():
        with torch.no_grad():
            return float((block.prompt(x, docs).double() * dy.double()).sum())

    leaves = block.weights() + [x]
    for i in (0, 1, 2, 3, 6, len(leaves) - 1):     # the projections, norms, W_down and the input
        w, g = leaves[i], grads[i]
        u = (g / g.norm()).to(w.dtype)
        h = 1e-2 * float(w.norm()) / w.numel() ** 0.5
        keep = w.clone()
        w.copy_(keep + h * u)
        up = loss()
        w.copy_(keep - h * u)
        down = loss()
        w.copy_(keep)
        slope, want = (up - down) / (2 * h), float((g.double() * u.double()).sum())
        assert abs(slope - want) <= 1e-2 * float(g.norm()), i
