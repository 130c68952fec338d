"""A decoder block around the In-Place TTT layer: packed documents, a document
read in pieces, single tokens and a training step.

    x -> norm -> q, k, v -> per-head norm and rotation -> attention -> + x
      -> norm -> In-Place TTT layer -> +

The projections are plain library products; the per-head norm and rotation,
the attention and the layer run in libipttt.so.  What a program keeps: the
rotation table, one attention plan for the sequences of a step (every layer of
a model shares it) and, for serving, a cache of keys and values.

    python examples/attention_block.py            # runs all four, prints agreement and times
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import test_weight_mlp_amd as ip  # noqa: E402

ETA, TAU, EPS = 1e-3, 1e-5, 1e-6


def norm(x):
    return x * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + EPS).to(x.dtype)


def starts(lens):
    return [sum(lens[:i]) for i in range(len(lens))]


class AttentionHalf(torch.autograd.Function):
    """Fused q, k, v [tokens, (heads + 2 kv_heads) D] -> attention output, with its
    backward: one document a sequence of the plan, positions from each start."""

    @staticmethod
    def forward(ctx, qkv, w_q, w_k, positions, table, plan, p):
        n, hq, hk = p.tokens, p.heads, p.kv_heads
        x = qkv.view(n, hq + 2 * hk, p.head_dim)
        q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
        qr, kr = torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty_like(
            k, memory_format=torch.contiguous_format)
        ip.ipttt_qk_norm_rope(p, q, k, w_q, w_k, positions, table, qr, kr)
        b = ip.AttentionBuffers(plan, device=qkv.device)
        ip.ipttt_attention(plan, qr, kr, v, b.o, b.lse, b.ws)
        ctx.save_for_backward(qkv, w_q, w_k, positions, table, qr, kr, b.o, b.lse)
        ctx.plan, ctx.p = plan, p
        return b.o.view(n, -1)

    @staticmethod
    def backward(ctx, do):
        qkv, w_q, w_k, positions, table, qr, kr, o, lse = ctx.saved_tensors
        plan, p = ctx.plan, ctx.p
        n, hq, hk = p.tokens, p.heads, p.kv_heads
        x, dx = qkv.view(n, hq + 2 * hk, p.head_dim), torch.empty_like(qkv).view(n, hq + 2 * hk, p.head_dim)
        q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
        dq, dk, dv = dx[:, :hq], dx[:, hq:hq + hk], dx[:, hq + hk:]
        ws = torch.empty(plan.backward_workspace_bytes, dtype=torch.uint8, device=qkv.device)
        ip.ipttt_attention_backward(plan, qr, kr, v, o, lse, do.contiguous().view(o.shape), dq, dk, dv, ws)
        g = ip.QKGrads(p, device=qkv.device)
        ip.ipttt_qk_norm_rope_backward(p, q, k, w_q, w_k, positions, table, dq, dk, dq, dk, g.dw_q, g.dw_k, g.ws)
        return dx.view(n, -1), g.dw_q.to(w_q.dtype), g.dw_k.to(w_k.dtype), None, None, None, None


class TTTLayer(torch.autograd.Function):
    """The In-Place TTT layer over one step's tokens."""

    @staticmethod
    def forward(ctx, H, X0, W_gate, W_up, W_down, conv_w, W_target, p):
        buf = ip.allocate(p, H.device, save=True)
        ip.forward(p, H, X0, W_gate, W_up, W_down, conv_w, W_target, ETA, TAU, buf)
        ctx.save_for_backward(H, X0, W_gate, W_up, W_down, conv_w, W_target)
        ctx.p, ctx.buf = p, buf
        return buf.O

    @staticmethod
    def backward(ctx, dO):
        t = ctx.saved_tensors
        g = ip.backward(ctx.p, ctx.buf, *t, ETA, TAU, dO.contiguous())
        return (g.dH, g.dX0) + tuple(x.to(w.dtype) for x, w in zip(
            (g.dW_gate, g.dW_up, g.dW_down, g.dconv_w, g.dW_target), t[2:])) + (None,)


class Block:
    def __init__(self, d=1024, f=4096, heads=16, kv_heads=8, head_dim=64, chunk=128, positions=4096, seed=0,
                 dtype=torch.bfloat16):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def w(*shape, var):
            return (torch.randn(*shape, generator=gen, device="cuda") * var ** 0.5).to(dtype)

        self.d, self.f, self.hq, self.hk, self.D, self.chunk, self.dtype = d, f, heads, kv_heads, head_dim, chunk, dtype
        self.code = ip.IPTTT_BF16 if dtype == torch.bfloat16 else ip.IPTTT_F32
        self.W_qkv = w((heads + 2 * kv_heads) * head_dim, d, var=1 / d)
        self.W_o = w(d, heads * head_dim, var=1 / (heads * head_dim))
        self.w_q, self.w_k = 1 + w(head_dim, var=0.01), 1 + w(head_dim, var=0.01)
        self.ttt = [w(f, d, var=1 / d), w(f, d, var=1 / d), w(d, f, var=1 / f), w(d, 5, var=0.05), w(d, d, var=1 / d)]
        self.table = ip.rotation_table(positions, head_dim, 1e6)

    def weights(self):
        return [self.W_qkv, self.W_o, self.w_q, self.w_k] + self.ttt

    def qk_problem(self, tokens, out_rows=None):
        return ip.QKProblem(tokens, self.hq, self.hk, self.D, self.code, EPS, self.table.shape[0], out_rows)

    def prompt(self, x, docs):
        """Packed documents; differentiable."""
        plan = ip.AttentionPlan(self.hq, self.hk, self.D, docs, docs, self.code)
        pos = torch.cat([torch.arange(n, dtype=torch.int32, device="cuda") for n in docs])
        a = AttentionHalf.apply(norm(x) @ self.W_qkv.T, self.w_q, self.w_k, pos, self.table, plan,
                                self.qk_problem(len(x)))
        y = x + a @ self.W_o.T
        p = ip.Problem(1, len(x), self.d, self.f, self.chunk, self.code, starts(docs)).prepare_segments()
        return y + TTTLayer.apply(norm(y), x, *self.ttt, p)

    def cache(self, rows):
        return Cache(self, rows)

    @torch.no_grad()
    def step(self, x, cache, fold=True):
        """The next tokens of the cache's document: a piece of whole chunks, or
        (fold=False) tokens of a chunk that is not complete yet."""
        n, end = len(x), cache.end
        rows = torch.arange(end, end + n, dtype=torch.int32, device="cuda")
        qkv = (norm(x) @ self.W_qkv.T).view(n, self.hq + 2 * self.hk, self.D)
        q, k, v = qkv[:, :self.hq], qkv[:, self.hq:self.hq + self.hk], qkv[:, self.hq + self.hk:]
        ip.ipttt_qk_norm_rope(self.qk_problem(n, len(cache.k)), q, k, self.w_q, self.w_k, rows, self.table, q, cache.k,
                              v=v, v_out=cache.v, rows=rows)
        plan = ip.AttentionPlan(self.hq, self.hk, self.D, [n], [end + n], self.code, k_rows=len(cache.k))
        b = ip.AttentionBuffers(plan)
        ip.ipttt_attention(plan, q, cache.k, cache.v, b.o, b.lse, b.ws)
        y = x + b.o.view(n, -1) @ self.W_o.T
        p = ip.Problem(1, n, self.d, self.f, self.chunk, self.code, continues=[end > 0])
        buf = ip.forward(p, norm(y), x, *self.ttt, ETA, TAU, carry=True, S_in=cache.S if end else None,
                         S_out=cache.S if fold else None)
        cache.end += n
        return y + buf.O


class Cache:
    """One document's keys, values and fast-weight state."""

    def __init__(self, block, rows):
        self.k, self.v = (torch.empty(rows, block.hk, block.D, dtype=block.dtype, device="cuda") for _ in "kv")
        self.S = torch.zeros(1, block.d, block.f, dtype=torch.float32, device="cuda")
        self.end = 0


def train_step(block, x, docs, dy):
    """Gradients of <y, dy> with respect to every weight and the input."""
    leaves = [w.requires_grad_(True) for w in block.weights()]
    x = x.detach().requires_grad_(True)
    try:
        y = block.prompt(x, docs)
        grads = torch.autograd.grad(y, leaves + [x], dy)
    finally:
        for w in leaves:
            w.requires_grad_(False)
    return y.detach(), grads


def main():
    block = Block()
    c = block.chunk
    x = torch.randn(8 * c, block.d, device="cuda").to(block.dtype)

    def rel(a, b):
        return float((a.float() - b.float()).norm() / b.float().norm())

    with torch.no_grad():
        whole = block.prompt(x, [len(x)])
    cache = block.cache(len(x) + 16)
    pieces = torch.cat([block.step(p, cache) for p in (x[:3 * c], x[3 * c:4 * c], x[4 * c:])])
    print(f"a document of {len(x)} tokens in three pieces against one call: {rel(pieces, whole):.1e}")
    cache = block.cache(len(x) + 16)
    head = block.step(x[:7 * c], cache)
    tail = torch.cat([block.step(x[i:i + 1], cache, fold=False) for i in range(7 * c, 7 * c + 16)])
    print(f"its last chunk's first 16 tokens one at a time: {rel(tail, whole[7 * c:7 * c + 16]):.1e}")
    docs = [300, 1, 500, len(x) - 801]
    for what, f in (("packed documents", lambda: block.prompt(x, docs)),
                    ("training step", lambda: train_step(block, x, docs, x))):
        for _ in range(3):
            f()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(10):
            f()
        torch.cuda.synchronize()
        print(f"{what}: {(time.perf_counter() - t) * 100:.2f} ms")
    del head
    return 0


if __name__ == "__main__":
    sys.exit(main())
