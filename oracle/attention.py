"""fp64 numpy definitions of the attention half, written from the formulas; the
reference of its tests.

attention(): causal attention over packed sequences with grouped heads, the
queries of sequence i being the last q_len[i] positions of its k_len[i] keys.
qk_norm_rope(): RMS norm of each head, then the rotation of its halves.
Each has its backward (the chain rule through exactly that forward).
"""
import numpy as np


def visible(q_len, k_len):
    """[q_len, k_len] truth values: query t sees keys below k_len - q_len + t + 1."""
    return np.arange(k_len)[None, :] < (k_len - q_len + np.arange(q_len) + 1)[:, None]


def _softmax(s, see):
    s = np.where(see, s, -np.inf)
    m = s.max(-1, keepdims=True, initial=-np.inf)
    e = np.where(see, np.exp(s - np.where(np.isfinite(m), m, 0.0)), 0.0)
    l = e.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (np.where(np.isfinite(m), m, 0.0) + np.log(l))[..., 0]
    return e / np.where(l > 0, l, 1.0), lse


def _blocks(q, k, seqs):
    hq, hk = q.shape[1], k.shape[1]
    for qs, ql, ks, kl in seqs:
        for h in range(hq):
            yield slice(qs, qs + ql), slice(ks, ks + kl), h, h // (hq // hk), visible(ql, kl)


def attention(q, k, v, seqs, scale):
    """o [rows, heads, D] and lse [rows, heads]; rows of no sequence are NaN."""
    o, lse = np.full(q.shape, np.nan), np.full(q.shape[:2], np.nan)
    for rq, rk, h, g, see in _blocks(q, k, seqs):
        p, lse[rq, h] = _softmax(scale * (q[rq, h] @ k[rk, g].T), see)
        o[rq, h] = p @ np.where(np.isfinite(v[rk, g]), v[rk, g], 0.0)
    return o, lse


def attention_backward(q, k, v, do, seqs, scale):
    """dq, dk, dv; rows of no sequence are NaN."""
    dq, dk, dv = np.full(q.shape, np.nan), np.full(k.shape, np.nan), np.full(v.shape, np.nan)
    for qs, ql, ks, kl in seqs:
        dk[ks:ks + kl], dv[ks:ks + kl] = 0.0, 0.0
    for rq, rk, h, g, see in _blocks(q, k, seqs):
        p, _ = _softmax(scale * (q[rq, h] @ k[rk, g].T), see)
        dp = do[rq, h] @ v[rk, g].T
        ds = scale * p * (dp - (dp * p).sum(-1, keepdims=True))
        dq[rq, h] = ds @ k[rk, g]
        dk[rk, g] += ds.T @ q[rq, h]
        dv[rk, g] += p.T @ do[rq, h]
    return dq, dk, dv


def _angles(table, positions):
    h = table.shape[1] // 2
    t = table[positions][:, None, :]
    return t[..., :h], t[..., h:], h


def norm_rope(x, w, positions, table, eps):
    """One of q, k: [tokens, heads, D]."""
    c, s, h = _angles(table, positions)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return np.concatenate([y[..., :h] * c - y[..., h:] * s, y[..., h:] * c + y[..., :h] * s], -1)


def norm_rope_backward(x, w, dz, positions, table, eps):
    """dx and dw (summed over tokens and heads)."""
    c, s, h = _angles(table, positions)
    dy = np.concatenate([dz[..., :h] * c + dz[..., h:] * s, dz[..., h:] * c - dz[..., :h] * s], -1)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xn, u = x * r, dy * w
    return r * (u - xn * (u * xn).mean(-1, keepdims=True)), (dy * xn).sum((0, 1))
