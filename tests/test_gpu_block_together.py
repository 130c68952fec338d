"""Norms, projections and the kept 8 bits as a decoder block uses them together, with
the attention between them and the layer behind, against the same block in 64 bits.

Bounds in bf16, as parts of each tensor's norm.  The root mean square of a rounding is
below 2^-9 of the values'.  The half has eight of them forward (n, qkv, q and k twice
each, o, y) and as many backward, and every step between has a gain of order one on
these inputs (normal weights of unit gain, scores of order one): 16 2^-9 = 2^-5 if all
of them lined up."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def block_of(dtype, **kw):
    import attention_block as ab
    sizes = dict(d=256, f=640, heads=8, kv_heads=2, head_dim=32, chunk=32, positions=512)
    return ab, ab.Block(**{**sizes, **kw}, dtype=dtype)


def norm64(x, w, eps):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w


def half64(block, x, docs, weights, eps):
    """The attention half in torch's 64 bits."""
    W_qkv, W_o, w_q, w_k, w_in = weights
    t, D = len(x), block.D
    qkv = (norm64(x, w_in, eps) @ W_qkv.T).view(t, -1, D)
    pos = torch.cat([torch.arange(m) for m in docs]).cuda()
    cs = block.table.double()[pos]
    c, s = cs[:, None, :D // 2], cs[:, None, D // 2:]

    def rotated(v, w):
        v = norm64(v, w, eps)
        a, b = v[..., :D // 2], v[..., D // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    q, k, v = qkv[:, :block.hq], qkv[:, block.hq:block.hq + block.hk], qkv[:, block.hq + block.hk:]
    q, k = rotated(q, w_q), rotated(k, w_k)
    group, out = block.hq // block.hk, []
    at = 0
    for n in docs:
        later = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
        heads = []
        for h in range(block.hq):
            score = q[at:at + n, h] @ k[at:at + n, h // group].T * D ** -0.5
            heads.append(torch.softmax(score.masked_fill(later, float("-inf")), -1) @ v[at:at + n, h // group])
        out.append(torch.stack(heads, 1))
        at += n
    return x + torch.cat(out).reshape(t, -1) @ W_o.T


# one token; a few rows (one pass over the weights); documents over several tiles
@pytest.mark.parametrize("dtype, limit", [(torch.bfloat16, 2.0 ** -5), (torch.float32, 2e-5)], ids=["bf16", "f32"])
@pytest.mark.parametrize("docs", [[1], [5, 1, 20], [100, 1, 200, 31]])
def test_half_and_its_gradients(docs, dtype, limit):
    """fp32: sums of up to 330 terms, some 1e-6 each step."""
    ab, block = block_of(dtype)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x, dy = (torch.randn(sum(docs), block.d, generator=gen, device="cuda").to(dtype) for _ in "xy")
    leaves = [x] + [block.W_qkv, block.W_o, block.w_q, block.w_k, block.w_in]
    for t in leaves:
        t.requires_grad_(True)
    y = block.half(x, docs)
    grads = torch.autograd.grad(y, leaves, dy)
    wide = [t.detach().double().requires_grad_(True) for t in leaves]
    want = half64(block, wide[0], docs, wide[1:], ab.EPS)
    want_grads = torch.autograd.grad(want, wide, dy.double())
    assert rel(y.detach(), want.detach()) <= limit
    for i, (a, b) in enumerate(zip(grads, want_grads)):
        if docs == [1] and i in (3, 4):     # one key: the scores' gradients are rounding alone
            continue
        assert rel(a, b) <= limit, i


def test_training_step_with_8_bits_kept():
    """The whole block: the same output, and gradients that 8 bits move by 2 % at most
    (some 0.6 % of each kept value, through slopes of order one)."""
    ab, block = block_of(torch.bfloat16)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    docs = [130, 64, 70]
    x, dy = (torch.randn(sum(docs), block.d, generator=gen, device="cuda").bfloat16() for _ in "xy")
    y, grads = ab.train_step(block, x, docs, dy)
    block.keep8 = False
    y_whole, whole = ab.train_step(block, x, docs, dy)
    assert torch.equal(y, y_whole)
    for a, b in zip(grads, whole):
        assert rel(a, b) <= 0.02
    assert any(not torch.equal(a, b) for a, b in zip(grads, whole))


def test_tokens_equal_the_prompt_in_bf16():
    """Single tokens take the projections' few-row form; two more roundings of each
    intermediate than the 64-bit block has, so twice its bound apart."""
    ab, block = block_of(torch.bfloat16)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    c = block.chunk
    x = torch.randn(3 * c, block.d, generator=gen, device="cuda").bfloat16()
    with torch.no_grad():
        whole = block.prompt(x, [len(x)])
    cache = block.cache(len(x))
    block.step(x[:2 * c], cache)
    tail = torch.cat([block.step(x[i:i + 1], cache, fold=False) for i in range(2 * c, 2 * c + 6)])
    assert rel(tail, whole[2 * c:2 * c + 6]) <= 2.0 ** -4
