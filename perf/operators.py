"""What is measured of the attention half of a block: the per-head norm and
position rotation of queries and keys, and causal attention over packed
sequences, each forward and backward.

A case is one pass through one of them:

  qk       ipttt_qk_norm_rope: q, k [tokens, heads, D] -> normed, rotated; with
           a cache, k and v go to the cache rows of their tokens
  qk_grad  ipttt_qk_norm_rope_backward: cotangents -> dq, dk, dw_q, dw_k
  attend   ipttt_attention: o and the rows' log-sum-exp
  train    ipttt_attention, then ipttt_attention_backward: o, dq, dk, dv

Sequences are given as comma-separated lengths; sequence i's queries are the
last q[i] positions of its k[i] keys.  The layouts are those of use: prompts
and training read q, k, v as slices of one fused projection, single tokens
and streamed pieces read a cache of equal slots.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
THETA = 1e6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# (query heads, key heads, head width): the block of the framework's 4B shape
# (d_model 2560), of its small one (d_model 1024), of its tiny one (d_model 64),
# and generic ones: one key head, a key head for each query head, odd widths.
HEADS = [(32, 8, 128), (16, 8, 64), (2, 1, 32), (8, 1, 128), (6, 6, 80), (12, 4, 96), (5, 5, 64)]


def listed():
    return [
        # one token of one sequence being decoded, into its cache row: latency
        dict(name="qk 1 token", op="qk", tokens=1, heads=32, kv=8, dim=128, dtype="bf16", cache=4097),
        # the fp32 configuration's heads over an odd number of tokens
        dict(name="qk f32 1021 tokens", op="qk", tokens=1021, heads=16, kv=8, dim=64, dtype="f32", cache=0),
        # the 4B shape's 32k prompt
        dict(name="qk 32768 tokens", op="qk", tokens=32768, heads=32, kv=8, dim=128, dtype="bf16", cache=0),
        # a training step over packed rows
        dict(name="qk_grad 16384 tokens", op="qk_grad", tokens=16384, heads=32, kv=8, dim=128, dtype="bf16", cache=0),
        # the next token of one sequence: latency, and one long axis to split
        dict(name="attend 1 over 4097", op="attend", q="1", k="4097", heads=32, kv=8, dim=128, dtype="bf16", cache=1),
        # the next token of 32 sequences of a serving batch, lengths of all kinds
        dict(name="attend 32 x 1 over caches", op="attend", q=",".join(["1"] * 32),
             k=",".join(str(1 + (i * i * 5167) % 16000) for i in range(1, 33)), heads=32, kv=8, dim=128, dtype="bf16",
             cache=1),
        # one piece of a long document read in pieces, over what it read before
        dict(name="attend 2048 over 30721", op="attend", q="2048", k="30721", heads=32, kv=8, dim=128, dtype="bf16",
             cache=1),
        # packed documents of a prompt batch, a document of one token among them
        dict(name="attend packed 8192", op="attend", q="2311,1,640,3500,257,1483", k="2311,1,640,3500,257,1483",
             heads=32, kv=8, dim=128, dtype="bf16", cache=0),
        # the 4B shape's 32k prompt, one document
        dict(name="attend 32768", op="attend", q="32768", k="32768", heads=32, kv=8, dim=128, dtype="bf16", cache=0),
        # fp32 data, odd lengths, a sequence with more queries than keys (its first rows see nothing)
        dict(name="attend f32 packed", op="attend", q="700,97,300", k="700,1025,255", heads=16, kv=8, dim=64,
             dtype="f32", cache=1),
        # a training step over one long document
        dict(name="train 8192", op="train", q="8192", k="8192", heads=32, kv=8, dim=128, dtype="bf16", cache=0),
        # a training step of the small shape over packed documents
        dict(name="train packed 4096", op="train", q="1025,333,1999,739", k="1025,333,1999,739", heads=16, kv=8,
             dim=64, dtype="bf16", cache=0),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n + 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["qk", "qk_grad", "attend", "attend", "attend", "train", "train"])
    heads, kv, dim = rng.choice(HEADS)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    c = dict(op=op, heads=heads, kv=kv, dim=dim, dtype=dtype)
    if op in ("qk", "qk_grad"):
        c["tokens"] = _log(rng, 1, 16384)
        c["cache"] = c["tokens"] + _log(rng, 1, 4096) if op == "qk" and rng.random() < 0.5 else 0
        return c
    if op == "train":
        q = [_log(rng, 1, 2500) for _ in range(rng.randint(1, 4))]
        k = list(q)
        c["cache"] = 0
    else:
        form = rng.choice(["single", "piece", "prompt"])
        if form == "single":      # the next token, or a few, of many sequences
            k = [_log(rng, 1, 16384) for _ in range(_log(rng, 1, 32))]
            q = [rng.choice([1, 1, 1, 2, 5]) for _ in k]
        elif form == "piece":     # pieces over what came before
            k = [_log(rng, 64, 16384) for _ in range(rng.randint(1, 3))]
            q = [_log(rng, 1, 2048) for _ in k]
        else:
            q = [_log(rng, 1, 5000) for _ in range(rng.randint(1, 5))]
            k = list(q)
        c["cache"] = 0 if form == "prompt" else 1
    c["q"], c["k"] = (",".join(str(3073 if n == 3072 else n) for n in x) for x in (q, k))
    return c


def _lens(text):
    return [int(n) for n in text.split(",")]


def _starts(lens):
    return [int(n) for n in np.concatenate([[0], np.cumsum(lens)[:-1]])]


def prepare(case, seed):
    dev, dt = "cuda", DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dt)

    hq, hk, d = case["heads"], case["kv"], case["dim"]
    s = dict(case=dict(case))
    if case["op"] in ("qk", "qk_grad"):
        n = case["tokens"]
        rows = max(case["cache"], n)
        # a fused projection's output, channels of unequal size
        fused = randn(n, hq + 2 * hk, d) * torch.exp(0.5 * torch.randn(d, generator=gen, device=dev)).to(dt)
        s.update(q=fused[:, :hq], k=fused[:, hq:hq + hk], v=fused[:, hq + hk:])
        s.update(w_q=1 + randn(d, scale=0.1), w_k=1 + randn(d, scale=0.1))
        inv = THETA ** (-np.arange(0, d, 2, dtype=np.float64) / d)
        ang = np.arange(rows, dtype=np.float64)[:, None] * inv
        s["table"] = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).to(dev)
        # the last n positions; several documents restart them
        pos = torch.arange(n, device=dev) + (rows - n if case["cache"] else 0)
        if n > 64 and not case["cache"]:
            cut = torch.randint(1, n, (3,), generator=gen, device=dev)
            start = torch.where(torch.arange(n, device=dev)[:, None] >= cut, cut, 0).amax(1)
            pos = pos - start
        s["pos"] = pos.to(torch.int32)
        s["q_out"] = torch.empty(n, hq, d, dtype=dt, device=dev)
        s["rows"] = None
        if case["cache"]:
            s["k_out"], s["v_out"] = randn(rows, hk, d), randn(rows, hk, d)
            s["rows"] = torch.randperm(rows, generator=gen, device=dev)[:n].to(torch.int32)  # slots as a pool hands them out
        else:
            s["k_out"], s["v_out"] = torch.empty(n, hk, d, dtype=dt, device=dev), None
        if case["op"] == "qk_grad":
            s["dq_out"], s["dk_out"] = randn(n, hq, d), randn(n, hk, d)
    else:
        ql, kl = _lens(case["q"]), _lens(case["k"])
        qs = _starts(ql)
        nq = sum(ql)
        if case["cache"]:
            cap = max(kl) + 13
            ks, nk = [i * cap for i in range(len(kl))], cap * len(kl)
            q, k, v = randn(nq, hq, d, scale=2.0), randn(nk, hk, d), randn(nk, hk, d)
        else:
            ks, nk = _starts(kl), sum(kl)
            fused = randn(nq, hq + 2 * hk, d)
            fused[:, :hq] *= 2
            q, k, v = fused[:, :hq], fused[:, hq:hq + hk], fused[:, hq + hk:]
        s.update(q=q, k=k, v=v, ql=ql, kl=kl, qs=qs, ks=ks, nq=nq, nk=nk, scale=1 / math.sqrt(d))
        s["seqs"] = torch.tensor([qs, ql, ks, kl], device=dev)
        if case["op"] == "train":
            s["do"] = randn(nq, hq, d)
    if own:
        _prepare_own(s, case, dt)
    return s


def _prepare_own(s, case, dt):
    import test_weight_mlp_amd as ip
    code = ip.IPTTT_F32 if dt == torch.float32 else ip.IPTTT_BF16
    if case["op"] in ("qk", "qk_grad"):
        s["p"] = ip.QKProblem(case["tokens"], case["heads"], case["kv"], case["dim"], code, eps=EPS,
                              table_rows=s["table"].shape[0], out_rows=s["k_out"].shape[0])
        if case["op"] == "qk_grad":
            s["grads"] = ip.QKGrads(s["p"])
    else:
        s["plan"] = ip.AttentionPlan(case["heads"], case["kv"], case["dim"], s["ql"], s["kl"], code, k_starts=s["ks"],
                                     k_rows=s["nk"], scale=s["scale"])
        s["buf"] = ip.AttentionBuffers(s["plan"], grads=case["op"] == "train")


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        return _run_own(s, op)
    if op == "qk":
        return _plain_qk(s)
    if op == "qk_grad":
        return _plain_qk_grad(s)
    return _plain_attention(s, op == "train")


def _run_own(s, op):
    import test_weight_mlp_amd as ip
    if op == "qk":
        ip.ipttt_qk_norm_rope(s["p"], s["q"], s["k"], s["w_q"], s["w_k"], s["pos"], s["table"], s["q_out"], s["k_out"],
                              v=s["v"] if s["rows"] is not None else None, v_out=s["v_out"], rows=s["rows"])
        return (s["q_out"], s["k_out"]) if s["rows"] is None else (s["q_out"], s["k_out"], s["v_out"])
    if op == "qk_grad":
        g = s["grads"]
        ip.ipttt_qk_norm_rope_backward(s["p"], s["q"], s["k"], s["w_q"], s["w_k"], s["pos"], s["table"], s["dq_out"],
                                       s["dk_out"], g.dq, g.dk, g.dw_q, g.dw_k, g.ws)
        return g.dq, g.dk, g.dw_q, g.dw_k
    b = s["buf"]
    ip.ipttt_attention(s["plan"], s["q"], s["k"], s["v"], b.o, b.lse, b.ws)
    if op == "attend":
        return b.o, b.lse
    ip.ipttt_attention_backward(s["plan"], s["q"], s["k"], s["v"], b.o, b.lse, s["do"], b.dq, b.dk, b.dv, b.ws)
    return b.o, b.dq, b.dk, b.dv


# ------------------------------------------------------------- plain forms

def _norm(x):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x, r


def _plain_qk(s):
    h = s["case"]["dim"] // 2
    cs = s["table"][s["pos"].long()][:, None, :]
    c, sn = cs[..., :h], cs[..., h:]

    def turn(x, w):
        x, r = _norm(x)
        y = x * r * w.float()
        a, b = y[..., :h], y[..., h:]
        return torch.cat([a * c - b * sn, b * c + a * sn], -1)

    s["q_out"].copy_(turn(s["q"], s["w_q"]))
    k = turn(s["k"], s["w_k"]).to(s["k_out"].dtype)
    if s["rows"] is None:
        s["k_out"].copy_(k)
        return s["q_out"], s["k_out"]
    at = s["rows"].long()
    s["k_out"][at] = k
    s["v_out"][at] = s["v"]
    return s["q_out"], s["k_out"], s["v_out"]


def _plain_qk_grad(s):
    h = s["case"]["dim"] // 2
    cs = s["table"][s["pos"].long()][:, None, :]
    c, sn = cs[..., :h], cs[..., h:]

    def back(x, w, dz):
        x, r = _norm(x)
        dz = dz.float()
        a, b = dz[..., :h], dz[..., h:]
        dy = torch.cat([a * c + b * sn, b * c - a * sn], -1)
        xn, u = x * r, dy * w.float()
        dx = r * (u - xn * (u * xn).mean(-1, keepdim=True))
        return dx.to(s["q"].dtype), (dy * xn).sum((0, 1))

    dq, dw_q = back(s["q"], s["w_q"], s["dq_out"])
    dk, dw_k = back(s["k"], s["w_k"], s["dk_out"])
    return dq, dk, dw_q, dw_k


def _plain_attention(s, grads):
    """Every sequence padded to the longest, all scores of a group of heads at once."""
    hk, g, d = s["case"]["kv"], s["case"]["heads"] // s["case"]["kv"], s["case"]["dim"]
    qs, ql, ks, kl = s["seqs"]
    n, mq, mk, dt = len(s["ql"]), max(s["ql"]), max(s["kl"]), s["q"].dtype
    iq, ik = (torch.arange(m, device=qs.device) for m in (mq, mk))
    at_q = torch.minimum(qs[:, None] + iq, qs[:, None] + ql[:, None] - 1)
    at_k = torch.minimum(ks[:, None] + ik, ks[:, None] + kl[:, None] - 1)

    # a group's heads share one product, unless its scores reach 2^31 elements:
    # the library's batched product is wrong from there on
    b = 1 if g * mq * mk < 1 << 31 else g

    def rows(x, at):  # [rows, hq, d] -> [n, hk, b, (g / b) * mq, d]
        return x[at].float().view(n, mq, hk, g, d).permute(0, 2, 3, 1, 4).reshape(n, hk, b, g // b * mq, d)

    def keys(x):      # [rows, hk, d] -> [n, hk, 1, mk, d]
        return x[at_k].float().permute(0, 2, 1, 3).contiguous()[:, :, None]

    def packed(x):    # [n, hk, b, (g / b) * mq, ...] -> [rows, hq, ...]
        seq = torch.repeat_interleave(torch.arange(n, device=qs.device), ql, output_size=s["nq"])
        pos = torch.arange(s["nq"], device=qs.device) - qs[seq]
        x = x.reshape(n, hk, g, mq, -1).permute(0, 3, 1, 2, 4)
        return x[seq, pos].reshape(s["nq"], hk * g, -1)

    q, k, v = rows(s["q"], at_q), keys(s["k"]), keys(s["v"])
    sees = ik < torch.minimum((kl - ql)[:, None] + iq + 1, kl[:, None])[..., None]     # [n, mq, mk]
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
    p.view(n, hk, g, mq, mk).masked_fill_(~sees[:, None, None], -math.inf)
    m = p.amax(-1, keepdim=True)
    p.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    l = p.sum(-1, keepdim=True)
    some = torch.where(l == 0, 1.0, l)
    o = torch.matmul(p, v) / some
    out = packed(o).to(dt)
    if not grads:
        return out, packed(m + torch.log(l))[..., 0]
    p /= some
    do = rows(torch.cat([s["do"], s["do"].new_zeros(1, hk * g, d)]), torch.where(iq < ql[:, None], at_q, s["nq"]))
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2)
    ds = torch.matmul(do, v.transpose(-1, -2))
    ds.sub_((ds * p).sum(-1, keepdim=True)).mul_(p).mul_(s["scale"])
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2)
    seq = torch.repeat_interleave(torch.arange(n, device=qs.device), kl, output_size=s["nk"])
    pos = torch.arange(s["nk"], device=qs.device) - ks[seq]
    dk, dv = (x.permute(0, 2, 1, 3)[seq, pos].to(dt) for x in (dk, dv))
    return out, packed(dq).to(dt), dk, dv


# ------------------------------------------------------------------- work

def work(case):
    hq, hk, d = case["heads"], case["kv"], case["dim"]
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "qk":
        n, moved = case["tokens"], hq + hk + (hk if case["cache"] else 0)
        return dict(bytes=2 * n * moved * d * e + n * (4 * d + 4) + 2 * d * e, flops=n * (hq + hk) * d * 8)
    if case["op"] == "qk_grad":
        n = case["tokens"]
        return dict(bytes=3 * n * (hq + hk) * d * e + n * (4 * d + 4) + 2 * d * (e + 4), flops=n * (hq + hk) * d * 16)
    ql, kl = _lens(case["q"]), _lens(case["k"])
    nq = sum(ql)
    nk = sum(k for q, k in zip(ql, kl) if q)
    pairs = 0
    for q, k in zip(ql, kl):        # row t sees max(0, k - q + t + 1) keys
        first = max(0, q - k)       # rows that see nothing
        n, a = q - first, k - q + first + 1
        pairs += n * a + n * (n - 1) // 2
    if case["op"] == "attend":
        return dict(bytes=(2 * nq * hq + 2 * nk * hk) * d * e + 4 * nq * hq, flops=4 * pairs * d * hq)
    # q, k, v, do read; o, dq, dk, dv written; two products forward and five backward
    return dict(bytes=(4 * nq * hq + 4 * nk * hk) * d * e, flops=14 * pairs * d * hq)


# ------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "qk":
        return _exact_qk(s, case)
    if case["op"] == "qk_grad":
        return _exact_qk_grad(s, case)
    return _exact_attention(s, case)


def _halves(case, s):
    t = s["table"].double().index_select(0, s["pos"].long())
    h = case["dim"] // 2
    return t[:, None, :h], t[:, None, h:], h


def _exact_qk(s, case):
    c, sn, h = _halves(case, s)
    out = []
    for x, w in ((s["q"], s["w_q"]), (s["k"], s["w_k"])):
        y = x.double()
        y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / case["dim"] + EPS) * w.double()
        z = torch.complex(y[..., :h], y[..., h:]) * torch.complex(c, sn)
        out.append(torch.cat([z.real, z.imag], -1))
    if s["rows"] is None:
        return tuple(out)
    k, v = s["k_out"].double(), s["v_out"].double()
    k.index_copy_(0, s["rows"].long(), out[1])
    v.index_copy_(0, s["rows"].long(), s["v"].double())
    return out[0], k, v


def _exact_qk_grad(s, case):
    c, sn, h = _halves(case, s)
    dx, dw = [], []
    for x, w, dz in ((s["q"], s["w_q"], s["dq_out"]), (s["k"], s["w_k"], s["dk_out"])):
        x, w, dz = x.double(), w.double(), dz.double()
        y = torch.complex(dz[..., :h], dz[..., h:]) * torch.complex(c, -sn)
        y = torch.cat([y.real, y.imag], -1)
        n = torch.sqrt(x.pow(2).sum(-1, keepdim=True) / case["dim"] + EPS)
        u = y * w
        dx.append(u / n - x * (u * x).sum(-1, keepdim=True) / (case["dim"] * n.pow(3)))
        dw.append((y * x / n).sum(1).sum(0))
    return dx[0], dx[1], dw[0], dw[1]


def _exact_attention(s, case):
    hq, g, train = case["heads"], case["heads"] // case["kv"], case["op"] == "train"
    o = torch.zeros(s["nq"], hq, case["dim"], dtype=torch.float64, device=s["q"].device)
    lse = torch.full((s["nq"], hq), -math.inf, dtype=torch.float64, device=s["q"].device)
    if train:
        dq = torch.zeros_like(o)
        dk, dv = (torch.zeros(s["nk"], case["kv"], case["dim"], dtype=torch.float64, device=o.device) for _ in "kv")
    for q0, ql, k0, kl in zip(s["qs"], s["ql"], s["ks"], s["kl"]):
        for head in range(hq):
            k, v = (s[x][k0:k0 + kl, head // g].double() for x in "kv")
            for t0 in range(max(0, ql - kl), ql, 8192):      # rows before see nothing
                t1 = min(ql, t0 + 8192)
                q = s["q"][q0 + t0:q0 + t1, head].double()
                last = torch.arange(t0, t1, device=o.device)[:, None] + (kl - ql)
                x = (q @ k.T) * s["scale"]
                x = torch.where(torch.arange(kl, device=o.device)[None] <= last, x, -math.inf)
                z = torch.logsumexp(x, -1)
                w = torch.exp(x - z[:, None])
                o[q0 + t0:q0 + t1, head] = w @ v
                lse[q0 + t0:q0 + t1, head] = z
                if train:
                    do = s["do"][q0 + t0:q0 + t1, head].double()
                    dv[k0:k0 + kl, head // g] += w.T @ do
                    dw = do @ v.T
                    dx = w * (dw - (w * dw).sum(-1, keepdim=True)) * s["scale"]
                    dq[q0 + t0:q0 + t1, head] = dx @ k
                    dk[k0:k0 + kl, head // g] += dx.T @ q
    return (o, dq, dk, dv) if train else (o, lse)
