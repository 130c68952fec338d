"""fp64 numpy definitions of the rest of a block, written from the formulas; the
reference of its tests: the norm of rows, a projection with its activation and
residual sum, each with its backward, and the values that 8 bits keep."""
import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def _centred(x, center, eps):
    d = x - x.mean(-1, keepdims=True) if center else x
    return d, 1.0 / np.sqrt((d * d).mean(-1, keepdims=True) + eps)


def norm(x, w, b, center, eps):
    d, r = _centred(x, center, eps)
    y = d * r
    y = y if w is None else y * w
    return y if b is None else y + b


def norm_backward(x, w, dy, dres, center, eps):
    """dx, dw, db."""
    d, r = _centred(x, center, eps)
    xn, u = d * r, dy if w is None else dy * w
    dx = u - xn * (u * xn).mean(-1, keepdims=True)
    if center:
        dx = dx - u.mean(-1, keepdims=True)
    dx = r * dx
    return dx if dres is None else dx + dres, (dy * xn).sum(0), dy.sum(0)


def _sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def act(kind, v):
    """kind: none, silu, gelu."""
    if kind == "silu":
        return v * _sigmoid(v)
    return v * 0.5 * _erfc(-v / math.sqrt(2.0)) if kind == "gelu" else v


def slope(kind, v):
    """The activation's derivative."""
    if kind == "silu":
        s = _sigmoid(v)
        return s * (1.0 + v * (1.0 - s))
    if kind == "gelu":
        return 0.5 * _erfc(-v / math.sqrt(2.0)) + v * np.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
    return np.ones_like(v)


def linear(x, W, b, res, kind):
    """y and what stands before the activation."""
    pre = x @ W.T if b is None else x @ W.T + b
    y = act(kind, pre)
    return y if res is None else y + res, pre


def linear_backward(x, W, pre, dy, kind):
    """dx, dW, db; pre is not looked at without an activation."""
    dp = dy if kind == "none" else dy * slope(kind, pre)
    return dp @ W, dp.T @ x, dp.sum(0)


def kept8(g, block=64):
    """The values that 8 bits keep of g [tokens, features]: each token's blocks of
    features as multiples, to 127, of 1/127 of the block's largest."""
    out = np.zeros_like(g)
    for c in range(0, g.shape[1], block):
        b = g[:, c:c + block]
        top = np.abs(b).max(1, keepdims=True)
        top = np.where(top > 0, top, 1.0)
        # bf16 values times 127 are exact, so ties are met exactly; they go to the even integer
        q = np.rint(b * 127.0 / top)
        out[:, c:c + block] = q * (top / 127.0)
    return out
