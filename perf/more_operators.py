"""What is measured of the rest of a block around the layer and its attention
half: the norm in front of each half, the projections of the attention half,
and the layer's gated products kept in 8 bits for the backward.

A case is one pass through one of them:

  norm         ipttt_norm: rows -> normed rows (layer norm or RMS norm)
  norm_grad    ipttt_norm_backward: cotangents (and those of the residual
               stream) -> dx, dw, db
  linear       ipttt_linear: act(x W^T + b) + residual; with pre, the product
               before the activation too
  linear_grad  ipttt_linear_backward: cotangents -> dx, dW, db
  keep8        ipttt_z_save8, then ipttt_z_backward_saved8: Z and, from gate
               and up products kept as 8-bit integers with a scale for each 64
               of a token, dH, dW_gate, dW_up
"""
import math

import torch

own = False

EPS = 1e-6
BLOCK = 64   # values of a token that share a scale in 8 bits
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# (inputs, outputs) of a projection: the 4B shape's fused q, k, v, its output
# projection and feed-forward pair (d_model 2560, d_ff 9728, 32 and 8 heads of
# width 128), the small shape's (d_model 1024, d_ff 4096, 16 and 8 heads of width
# 64), the tiny one's, and generic ones of odd multiples of 8.
LINEAR = [(2560, 6144), (4096, 2560), (2560, 9728), (9728, 2560), (1024, 2048), (1024, 4096), (4096, 1024), (1024, 1024),
          (64, 256), (200, 1000), (1288, 520), (320, 448)]
NORM = [64, 320, 1000, 1024, 2560, 2568, 4096, 9728]
LAYER = [(2560, 9728), (1024, 4096), (1024, 4096), (320, 448), (200, 520), (64, 256)]


def listed():
    return [
        # the next token of one sequence: latency
        dict(name="norm 1 row", op="norm", rows=1, dim=2560, kind="rms", dtype="bf16", affine="w"),
        # the 4B shape's 32k prompt
        dict(name="norm 32768 rows", op="norm", rows=32768, dim=2560, kind="layer", dtype="bf16", affine="wb"),
        # a training step of packed documents, with the residual stream's cotangent
        dict(name="norm_grad 16384 rows", op="norm_grad", rows=16384, dim=2560, kind="layer", dtype="bf16",
             affine="wb", res=True),
        # the small shape in fp32, an odd number of tokens
        dict(name="norm_grad f32 1021 rows", op="norm_grad", rows=1021, dim=1024, kind="rms", dtype="f32", affine="w",
             res=False),
        # the next token of one sequence through the fused q, k, v projection: latency, the weights' bytes
        dict(name="linear 1 token", op="linear", rows=1, k=2560, n=6144, act="none", bias=False, res=False, pre=False,
             dtype="bf16", wide=0),
        # the next token of 32 sequences through the output projection, added to the residual stream
        dict(name="linear 32 tokens", op="linear", rows=32, k=4096, n=2560, act="none", bias=False, res=True, pre=False,
             dtype="bf16", wide=0),
        # a feed-forward's first product in training, fp32, an odd number of tokens, kept for the backward
        dict(name="linear f32 1021 tokens", op="linear", rows=1021, k=1024, n=4096, act="gelu", bias=True, res=False,
             pre=True, dtype="f32", wide=0),
        # the output projection of the 4B shape's 32k prompt
        dict(name="linear 32768 tokens", op="linear", rows=32768, k=4096, n=2560, act="none", bias=False, res=True,
             pre=False, dtype="bf16", wide=0),
        # a training step's fused projection, gradients kept in 32 bits
        dict(name="linear_grad 8192 tokens", op="linear_grad", rows=8192, k=2560, n=6144, act="none", bias=True,
             dtype="bf16", grad="f32", wide=0),
        # a feed-forward's first product of the small shape over ragged documents
        dict(name="linear_grad 1999 tokens", op="linear_grad", rows=1999, k=1024, n=4096, act="gelu", bias=True,
             dtype="bf16", grad="bf16", wide=0),
        # a training step of the small shape
        dict(name="keep8 2049 tokens", op="keep8", tokens=2049, d=1024, f=4096),
        # a training step of the 4B shape
        dict(name="keep8 16384 tokens", op="keep8", tokens=16384, d=2560, f=9728),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "linear", "linear", "linear", "linear_grad", "linear_grad", "keep8"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("norm", "norm_grad"):
        c = dict(op=op, rows=_log(rng, 1, 20000), dim=rng.choice(NORM), kind=rng.choice(["rms", "layer"]), dtype=dtype,
                 affine=rng.choice(["w", "w", "wb", ""]))
        if op == "norm_grad":
            c["res"] = rng.random() < 0.5
        return c
    if op == "keep8":
        d, f = rng.choice(LAYER)
        return dict(op=op, tokens=_log(rng, 1, 8192), d=d, f=f)
    k, n = rng.choice(LINEAR)
    c = dict(op=op, rows=_log(rng, 1, 16384), k=k, n=n, act=rng.choice(["none", "none", "silu", "gelu"]),
             bias=rng.random() < 0.5, dtype=dtype, wide=rng.choice([0, 0, 8, 1024]))
    if op == "linear":
        c["res"] = rng.random() < 0.5
        c["pre"] = c["act"] != "none" and rng.random() < 0.5
    else:
        c["grad"] = "f32" if dtype == "f32" or c["act"] == "none" and rng.random() < 0.5 else "bf16"
    return c


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt = DTYPES[case.get("dtype", "bf16")]

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dt)

    s = dict(case=dict(case))
    if case["op"] in ("norm", "norm_grad"):
        n, d = case["rows"], case["dim"]
        # a residual stream: channels of unequal size and mean
        size = torch.exp(0.5 * torch.randn(d, generator=gen, device=dev))
        s["x"] = (torch.randn(n, d, generator=gen, device=dev) * size + 0.3 * size.roll(1)).to(dt)
        s["w"] = 1 + randn(d, scale=0.1) if "w" in case["affine"] else None
        s["b"] = randn(d, scale=0.1) if "b" in case["affine"] else None
        s["out"] = torch.empty(n, d, dtype=dt, device=dev)
        if case["op"] == "norm_grad":
            s["dy"] = randn(n, d)
            s["dres"] = randn(n, d) if case["res"] else None
    elif case["op"] in ("linear", "linear_grad"):
        m, k, n = case["rows"], case["k"], case["n"]
        s["x"] = randn(m, k + case["wide"])[:, :k]     # wide: columns of a wider tensor
        s["W"] = randn(n, k, scale=k ** -0.5)
        s["b"] = randn(n, scale=0.1) if case["bias"] else None
        if case["op"] == "linear":
            s["res"] = randn(m, n) if case["res"] else None
            s["y"] = torch.empty(m, n, dtype=dt, device=dev)
            s["pre"] = torch.empty(m, n, dtype=dt, device=dev) if case["pre"] else None
        else:
            s["dy"] = randn(m, n)
            # what the forward kept: the product before the activation
            s["pre"] = None if case["act"] == "none" else (
                s["x"].float() @ s["W"].float().T + (0.0 if s["b"] is None else s["b"].float())).to(dt)
    else:
        t, d, f = case["tokens"], case["d"], case["f"]
        s["H"] = randn(t, d)
        s["Wg"], s["Wu"] = randn(f, d, scale=d ** -0.5), randn(f, d, scale=d ** -0.5)
        s["dZ"] = randn(t, f)
    if own:
        _prepare_own(s, case, dt)
    return s


def _prepare_own(s, case, dt):
    import test_weight_mlp_amd as ip
    code = ip.IPTTT_F32 if dt == torch.float32 else ip.IPTTT_BF16
    if case["op"] in ("norm", "norm_grad"):
        kind = ip.IPTTT_NORM_LAYER if case["kind"] == "layer" else ip.IPTTT_NORM_RMS
        s["p"] = ip.NormProblem(case["rows"], case["dim"], code, kind, EPS)
        if case["op"] == "norm_grad":
            s["grads"] = ip.NormGrads(s["p"])
    elif case["op"] in ("linear", "linear_grad"):
        act = {"none": ip.IPTTT_ACT_NONE, "silu": ip.IPTTT_ACT_SILU, "gelu": ip.IPTTT_ACT_GELU}[case["act"]]
        grad = ip.IPTTT_F32 if case.get("grad") == "f32" else code
        s["p"] = ip.LinearProblem(case["rows"], case["k"], case["n"], code, act, grad_dtype=grad)
        if case["op"] == "linear":
            s["ws"] = ip.linear_workspace(s["p"])
        else:
            s["grads"] = ip.LinearGrads(s["p"])
    else:
        s["p"] = ip.Problem(1, case["tokens"], case["d"], case["f"], 512, code)
        s["Z"] = torch.empty_like(s["dZ"])
        s["GU8"] = torch.empty(ip.ipttt_saved8_bytes(s["p"]), dtype=torch.uint8, device="cuda")
        s["grads"] = ip.Grads(s["p"])


def run(state):
    s = state
    return (_OWN if own else _PLAIN)[s["case"]["op"]](s)


def _own_norm(s):
    import test_weight_mlp_amd as ip
    ip.ipttt_norm(s["p"], s["x"], s["w"], s["b"], s["out"])
    return s["out"]


def _own_norm_grad(s):
    import test_weight_mlp_amd as ip
    g = s["grads"]
    dw, db = (None if s[x] is None else y for x, y in (("w", g.dw), ("b", g.db)))
    ip.ipttt_norm_backward(s["p"], s["x"], s["w"], s["dy"], g.dx, dw, db, g.ws, dres=s["dres"])
    return g.dx, dw, db


def _own_linear(s):
    import test_weight_mlp_amd as ip
    ip.ipttt_linear(s["p"], s["x"], s["W"], s["y"], b=s["b"], res=s["res"], pre=s["pre"], ws=s["ws"])
    return s["y"], s["pre"]


def _own_linear_grad(s):
    import test_weight_mlp_amd as ip
    g = s["grads"]
    db = None if s["b"] is None else g.db
    ip.ipttt_linear_backward(s["p"], s["x"], s["W"], s["dy"], g.dx, g.dW, db, g.ws, pre=s["pre"])
    return g.dx, g.dW, db


def _own_keep8(s):
    import test_weight_mlp_amd as ip
    p, g, dt = s["p"], s["grads"], s["H"].dtype
    ip.ipttt_z_save8(p, s["H"], s["Wg"], s["Wu"], s["Z"], s["GU8"])
    ip.ipttt_z_backward_saved8(p, s["H"], s["Wg"], s["Wu"], s["GU8"], s["dZ"], g.dH, g.dW_gate, g.dW_up, g.ws)
    return s["Z"], g.dH, g.dW_gate.to(dt), g.dW_up.to(dt)   # as an optimizer of weights of that type takes them


# ------------------------------------------------------------- plain forms

def _normed(s):
    x = s["x"].float()
    if s["case"]["kind"] == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _plain_norm(s):
    y, _ = _normed(s)
    if s["w"] is not None:
        y = y * s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    return y.to(s["x"].dtype)


def _plain_norm_grad(s):
    xn, r = _normed(s)
    dy = s["dy"].float()
    u = dy if s["w"] is None else dy * s["w"].float()
    dx = u - xn * (u * xn).mean(-1, keepdim=True)
    if s["case"]["kind"] == "layer":
        dx = dx - u.mean(-1, keepdim=True)
    dx = dx * r
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    dw = None if s["w"] is None else (dy * xn).sum(0)
    db = None if s["b"] is None else dy.sum(0)
    return dx.to(s["x"].dtype), dw, db


def _cdf(x):
    return 0.5 * torch.erfc(x * -math.sqrt(0.5))


def _plain_linear(s):
    dt, act = s["x"].dtype, s["case"]["act"]
    y = s["x"].float() @ s["W"].float().T
    if s["b"] is not None:
        y = y + s["b"].float()
    pre = y.to(dt) if s["pre"] is not None else None
    if act == "silu":
        y = y / (1 + torch.exp(-y))
    elif act == "gelu":
        y = y * _cdf(y)
    if s["res"] is not None:
        y = y + s["res"].float()
    return y.to(dt), pre


def _slope(act, x):
    if act == "silu":
        e = 1 / (1 + torch.exp(-x))
        return e * (1 + x * (1 - e))
    return _cdf(x) + x * torch.exp(-0.5 * x * x) * (0.5 / math.pi) ** 0.5


def _plain_linear_grad(s):
    dt, act = s["x"].dtype, s["case"]["act"]
    dp = s["dy"].float()
    if act != "none":
        dp = dp * _slope(act, s["pre"].float())
    dx = dp @ s["W"].float()
    dW = dp.T @ s["x"].float()
    return dx.to(dt), dW.to(DTYPES[s["case"]["grad"]]), dp.sum(0) if s["b"] is not None else None


def _kept(g):
    """What 8 bits keep of g [tokens, f], rounded to bf16 before: integers to 127, a scale for each block."""
    t, f = g.shape
    g = torch.nn.functional.pad(g.to(torch.bfloat16).to(g.dtype), (0, -f % BLOCK)).view(t, -1, BLOCK)
    scale = g.abs().amax(-1, keepdim=True) / 127
    q = torch.round(g / torch.where(scale == 0, 1.0, scale))
    return (q * scale).view(t, -1)[:, :f]


def _plain_keep8(s):
    dt = s["H"].dtype
    H, Wg, Wu, dZ = (s[x].float() for x in ("H", "Wg", "Wu", "dZ"))
    g, u = H @ Wg.T, H @ Wu.T
    Z = (g / (1 + torch.exp(-g)) * u).to(dt)
    g, u = _kept(g), _kept(u)
    e = 1 / (1 + torch.exp(-g))
    dg, du = dZ * u * (e * (1 + g * (1 - e))), dZ * (g * e)
    dH = dg @ Wg + du @ Wu
    return Z, dH.to(dt), (dg.T @ H).to(dt), (du.T @ H).to(dt)


_OWN = dict(norm=_own_norm, norm_grad=_own_norm_grad, linear=_own_linear, linear_grad=_own_linear_grad,
            keep8=_own_keep8)
_PLAIN = dict(norm=_plain_norm, norm_grad=_plain_norm_grad, linear=_plain_linear, linear_grad=_plain_linear_grad,
              keep8=_plain_keep8)


# ------------------------------------------------------------------- work

def work(case):
    e = 2 if case.get("dtype", "bf16") == "bf16" else 4
    if case["op"] in ("norm", "norm_grad"):
        n, d, vectors = case["rows"], case["dim"], len(case["affine"])
        if case["op"] == "norm":
            return dict(bytes=(2 * n * d + vectors * d) * e, flops=8 * n * d)
        return dict(bytes=(3 + bool(case["res"])) * n * d * e + vectors * d * (e + 4), flops=16 * n * d)
    if case["op"] == "linear":
        m, k, n = case["rows"], case["k"], case["n"]
        return dict(bytes=(m * k + n * k + m * n * (1 + case["res"] + case["pre"]) + n * case["bias"]) * e,
                    flops=2 * m * n * k)
    if case["op"] == "linear_grad":
        m, k, n = case["rows"], case["k"], case["n"]
        g = 4 if case["grad"] == "f32" else 2
        return dict(bytes=(2 * m * k + n * k + m * n * (1 + (case["act"] != "none"))) * e + n * k * g +
                    4 * n * case["bias"], flops=4 * m * n * k)
    t, d, f = case["tokens"], case["d"], case["f"]
    # H, the weights and dZ read; Z, dH and the weights' gradients written; what is kept, written and read
    kept = 2 * t * f + 8 * t * -(-f // BLOCK)
    return dict(bytes=(2 * t * d + 4 * d * f + 2 * t * f) * 2 + 2 * kept, flops=12 * t * d * f)


# ------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if case["op"] in ("norm", "norm_grad"):
        return _exact_norm(s, case)
    if case["op"] in ("linear", "linear_grad"):
        return _exact_linear(s, case)
    return _exact_keep8(s)


def _exact_norm(s, case):
    d = case["dim"]
    x = s["x"]
    mean = x.sum(1, keepdim=True) / d if case["kind"] == "layer" else torch.zeros_like(x[:, :1])
    std = torch.sqrt((x - mean).pow(2).sum(1, keepdim=True) / d + EPS)
    one, zero = torch.ones(d, dtype=torch.float64, device=x.device), 0.0
    w = one if s["w"] is None else s["w"]
    if case["op"] == "norm":
        return torch.addcmul(zero * one if s["b"] is None else s["b"], (x - mean) / std, w)
    dy = s["dy"]
    along = (dy * w * (x - mean)).sum(1, keepdim=True) / d
    dx = (dy * w) / std - (x - mean) * along / std.pow(3)
    if case["kind"] == "layer":
        dx -= (dy @ w)[:, None] / (d * std)
    if s["dres"] is not None:
        dx += s["dres"]
    return (dx, None if s["w"] is None else torch.einsum("td,td->d", dy, (x - mean) / std),
            None if s["b"] is None else torch.einsum("td->d", dy))


def _exact_linear(s, case):
    act, m = case["act"], case["rows"]
    step = 4096
    if case["op"] == "linear":
        y = torch.cat([torch.mm(s["x"][i:i + step], s["W"].t()) for i in range(0, m, step)])
        if s["b"] is not None:
            y += s["b"]
        pre = y.clone() if s["pre"] is not None else None
        if act == "silu":
            y = y * torch.sigmoid(y)
        elif act == "gelu":
            y = y * torch.special.ndtr(y)
        return (y if s["res"] is None else y + s["res"]), pre
    dp = s["dy"]
    if act != "none":
        z = s["pre"].detach().requires_grad_(True)
        with torch.enable_grad():
            a = z * torch.sigmoid(z) if act == "silu" else z * torch.special.ndtr(z)
            dp, = torch.autograd.grad(a, z, dp)
    return (torch.mm(dp, s["W"]), torch.mm(dp.t(), s["x"]),
            None if s["b"] is None else torch.mv(dp.t(), torch.ones(m, dtype=torch.float64, device=dp.device)))


def _exact_keep8(s):
    H, Wg, Wu, dZ = s["H"], s["Wg"], s["Wu"], s["dZ"]
    g, u = torch.mm(H, Wg.t()), torch.mm(H, Wu.t())
    Z = g * torch.sigmoid(g) * u
    for x in (g, u):       # in place: the values that 8 bits hold
        x.copy_(x.bfloat16())
        for c in range(0, x.shape[1], BLOCK):
            b = x[:, c:c + BLOCK]
            top = b.abs().max(1, keepdim=True).values
            b.copy_(torch.where(top > 0, torch.round(b * 127 / top.clamp_min(1e-300)) * top / 127, b))
    e = torch.sigmoid(g)
    du = dZ * g * e
    dg = dZ * u * e * (1 + g - g * e)
    return Z, torch.addmm(torch.mm(du, Wu), dg, Wg), torch.mm(dg.t(), H), torch.mm(du.t(), H)
