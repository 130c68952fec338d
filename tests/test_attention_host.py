"""Host checks of the attention half (no GPU): the fp64 definitions against
finite differences, the plan's tiles against the definition of what each query
sees, and every refusal before anything is launched."""
import ctypes
import os
import struct

import numpy as np
import pytest

import test_weight_mlp_amd as ip
from oracle import attention as oa
from test_weight_mlp_amd import attention as at

needs_lib = pytest.mark.skipif(not os.path.exists(ip.library_path), reason="libipttt.so not built")


# ------------------------------------------------------------ definitions

def _difference(f, x, u, eps=1e-6):
    return (f(x + eps * u) - f(x - eps * u)) / (2 * eps)


def test_attention_gradients_are_those_of_the_forward():
    rng = np.random.default_rng(0)
    seqs = [(0, 5, 0, 5), (5, 4, 5, 9), (9, 6, 14, 3), (15, 1, 17, 1)]
    q, do = (rng.standard_normal((16, 4, 8)) for _ in "ab")
    k, v = (rng.standard_normal((18, 2, 8)) for _ in "ab")
    grads = oa.attention_backward(q, k, v, do, seqs, 0.3)
    for i, g in enumerate(grads):
        u = rng.standard_normal(g.shape)

        def f(x):
            a = [q, k, v]
            a[i] = x
            return (oa.attention(*a, seqs, 0.3)[0] * do).sum()

        d = _difference(f, [q, k, v][i], u)
        assert abs(d - (g * u).sum()) <= 1e-6 * max(1.0, abs(d))
    assert np.all(grads[0][15] == 0)            # a softmax over one key


def test_norm_rope_gradients_are_those_of_the_forward():
    rng = np.random.default_rng(1)
    x, dz, w = rng.standard_normal((7, 3, 8)), rng.standard_normal((7, 3, 8)), rng.standard_normal(8)
    ang = rng.standard_normal((11, 4))
    table, pos = np.concatenate([np.cos(ang), np.sin(ang)], 1), rng.integers(0, 11, 7)
    dx, dw = oa.norm_rope_backward(x, w, dz, pos, table, 1e-3)
    for g, at_, f in ((dx, x, lambda y: (oa.norm_rope(y, w, pos, table, 1e-3) * dz).sum()),
                      (dw, w, lambda y: (oa.norm_rope(x, y, pos, table, 1e-3) * dz).sum())):
        u = rng.standard_normal(g.shape)
        assert abs(_difference(f, at_, u) - (g * u).sum()) <= 1e-6 * abs((g * u).sum())


def test_rotation_table_holds_64_bit_angles():
    t = ip.rotation_table(1000, 16, 10000.0, device="cpu").numpy()
    ang = 999 * 10000.0 ** (-np.arange(8) / 8)
    assert t.shape == (1000, 16)
    assert np.array_equal(t[999], np.concatenate([np.cos(ang), np.sin(ang)]).astype(np.float32))


# ------------------------------------------------------------------- plan

class Plan:
    """The plan's items, read back from the host table."""

    def __init__(self, p):
        raw = p._host.view(np.int32)
        names = ["magic", "dtype", "heads", "kv_heads", "head_dim", "n_seqs", "q_rows", "k_rows", "n_rows", "n_join",
                 "n_dq", "n_key", "o_rows", "o_join", "o_dq", "o_key", "parts", "overlap", "bytes", "n_key_join",
                 "o_key_join", "key_parts", "n_few", "o_few", "join_rows",
                 "n_tiles", "o_tiles", "n_dq_join", "o_dq_join", "dq_parts"]
        self.h = dict(zip(names, raw[:len(names)].tolist()))

        def items(o, n, fields):
            x = raw[o // 4:o // 4 + n * len(fields)].reshape(n, len(fields))
            return [dict(zip(fields, r.tolist())) for r in x]

        row = ["q_start", "q_len", "r0", "k_start", "off", "k_begin", "k_end", "part"]
        self.rows = items(self.h["o_rows"], self.h["n_rows"], row)
        self.dq = items(self.h["o_dq"], self.h["n_dq"], row)
        self.few = items(self.h["o_few"], self.h["n_few"], row)
        self.tiles = items(self.h["o_tiles"], self.h["n_tiles"], row)
        self.join, self.dq_join = (items(self.h["o" + w], self.h["n" + w], ["q_start", "q_len", "r0", "part", "n", "step"])
                                   for w in ("_join", "_dq_join"))
        self.key = items(self.h["o_key"], self.h["n_key"],
                         ["q_start", "q_len", "r_begin", "r_end", "k_start", "off", "key0", "part"])
        self.key_join = items(self.h["o_key_join"], self.h["n_key_join"], ["k_row", "n_keys", "part", "n"])


CASES = [
    (4, 4, [1], [1]),
    (4, 1, [3, 0, 257, 1], [3, 9, 257, 5000]),
    (6, 2, [100, 31], [40, 0]),
    (32, 8, [1] * 5, [1, 64, 4097, 300, 16000]),
    (8, 8, [700, 1], [2100, 130]),
    (32, 8, [3000], [3001]),
]


@needs_lib
@pytest.mark.parametrize("heads,kv,ql,kl", CASES)
def test_plan_tiles_cover_what_each_query_sees(heads, kv, ql, kl):
    p = ip.AttentionPlan(heads, kv, 64, ql, kl, device="cpu")
    pl, G = Plan(p), heads // kv
    qs, ks = np.concatenate([[0], np.cumsum(ql)]), np.concatenate([[0], np.cumsum(kl)])
    assert all(x["q_len"] * G <= 32 for x in pl.few)
    for items, joined, slots in ((pl.rows + pl.few, pl.join, "parts"), (pl.tiles, [], None),
                                 (pl.dq, pl.dq_join, "dq_parts")):
        got, seen = {(int(qs[i]), r0): [] for i, n in enumerate(ql) for r0 in range(0, n * G, 128)}, {}
        for x in items:
            got[(x["q_start"], x["r0"])].append(x)
        for (q0, r0), parts in got.items():
            i = next(i for i, n in enumerate(ql) if n and qs[i] == q0)
            last = min(r0 + 128, ql[i] * G) - 1
            sees = max(0, kl[i] - ql[i] + last // G + 1)
            parts.sort(key=lambda x: x["k_begin"])
            assert parts[0]["k_begin"] == 0 and parts[-1]["k_end"] == sees
            assert all(a["k_end"] == b["k_begin"] and b["k_begin"] % 64 == 0 for a, b in zip(parts, parts[1:]))
            assert all(x["k_start"] == ks[i] and x["off"] == kl[i] - ql[i] and x["q_len"] == ql[i] for x in parts)
            if len(parts) > 1:
                seen[(q0, r0)] = [x["part"] for x in parts]
            else:
                assert parts[0]["part"] == -1
        assert {(j["q_start"], j["r0"]): [j["part"] + x * j["step"] for x in range(j["n"])] for j in joined} == seen
        few = {x["q_start"] for x in pl.few} if slots == "parts" else set()
        assert all(j["step"] == (1 if j["q_start"] in few else 4) for j in joined)
        used = sorted(j["part"] + x for j in joined for x in range(j["n"] * j["step"]))
        assert used == list(range(pl.h[slots] if slots else 0))
    assert all(min(32 * j["step"], j["q_len"] * G - j["r0"]) <= pl.h["join_rows"] for j in pl.join)
    # keys: every tile of every sequence, over all rows from the first that sees its first key
    want = {(int(ks[i]), k0): (i, min(n, max(0, k0 - (m - n))) * G)
            for i, (n, m) in enumerate(zip(ql, kl)) for k0 in range(0, m, 128)}
    got = {key: [] for key in want}
    for x in pl.key:
        got[(x["k_start"], x["key0"])].append(x)
    joins = {}
    for (k0, key0), parts in got.items():
        i, first = want[(k0, key0)]
        parts.sort(key=lambda x: x["r_begin"])
        assert parts[0]["r_begin"] == first and parts[-1]["r_end"] == ql[i] * G
        assert all(a["r_end"] == b["r_begin"] and (b["r_begin"] - first) % 32 == 0 for a, b in zip(parts, parts[1:]))
        assert all(x["off"] == kl[i] - ql[i] and x["q_start"] == qs[i] for x in parts)
        if len(parts) > 1:
            joins[(k0 + key0, min(128, kl[i] - key0))] = [x["part"] for x in parts]
        else:
            assert parts[0]["part"] == -1
    assert {(j["k_row"], j["n_keys"]): list(range(j["part"], j["part"] + j["n"])) for j in pl.key_join} == joins
    assert sorted(x for v in joins.values() for x in v) == list(range(pl.h["key_parts"]))
    # long tiles come first
    cost = [x["k_end"] - x["k_begin"] for x in pl.rows]
    assert cost == sorted(cost, reverse=True)


@needs_lib
def test_plan_is_a_function_of_the_problem_and_sizes_its_workspaces():
    a, b = (ip.AttentionPlan(8, 2, 128, [1, 1], [9000, 12], device="cpu") for _ in "ab")
    assert np.array_equal(a._host, b._host)
    pl = Plan(a)
    assert pl.h["parts"] > 1 and a.workspace_bytes > 0
    assert a.backward_workspace_bytes >= 2 * 8 * 4
    long = ip.AttentionPlan(32, 8, 128, [8192], [8192], device="cpu")
    assert long.workspace_bytes == 0 and Plan(long).h["n_join"] == 0


# --------------------------------------------------------------- refusals

def _problem(**kw):
    base = dict(n_seqs=2, heads=4, kv_heads=2, head_dim=64, q_rows=10, k_rows=20, dtype=ip.IPTTT_BF16,
                q_start=[0, 4], q_len=[4, 6], k_start=[0, 8], k_len=[8, 12])
    base.update(kw)
    arrays = {n: None if base[n] is None else (ctypes.c_int64 * max(1, len(base[n])))(*base[n])
              for n in ("q_start", "q_len", "k_start", "k_len")}
    c = at._CAttnProblem(base["n_seqs"], base["heads"], base["kv_heads"], base["head_dim"], base["q_rows"],
                         base["k_rows"], base["dtype"])
    for n, a in arrays.items():
        if a is not None:
            setattr(c, n, ctypes.cast(a, ctypes.POINTER(ctypes.c_int64)))
    c._keep = arrays
    return c


@needs_lib
@pytest.mark.parametrize("kw,code", [
    (dict(dtype=5), 3), (dict(heads=3), 2), (dict(heads=0), 2), (dict(kv_heads=0), 2), (dict(heads=5000, kv_heads=1), 2),
    (dict(head_dim=0), 2), (dict(head_dim=12), 2), (dict(head_dim=136), 2), (dict(n_seqs=0), 2), (dict(q_rows=-1), 2),
    (dict(q_rows=1 << 31), 2), (dict(k_rows=1 << 31), 2), (dict(q_len=None), 1), (dict(k_start=None), 1),
    (dict(q_len=[4, 7]), 5), (dict(q_len=[5, 5]), 5), (dict(q_start=[4, 0]), 5), (dict(q_start=[-1, 4]), 5),
    (dict(k_len=[8, 13]), 5), (dict(k_start=[-1, 8]), 5), (dict(k_len=[-1, 2]), 5), (dict(q_len=[1 << 62, 1]), 5),
])
def test_plan_refuses(kw, code):
    c, lib = _problem(**kw), at._lib()
    assert lib.ipttt_attn_validate(ctypes.byref(c)) == code
    assert lib.ipttt_attn_plan_bytes(ctypes.byref(c)) == 0
    buf = (ctypes.c_int64 * 4096)()
    assert lib.ipttt_attn_plan(ctypes.byref(c), buf, 8 * 4096) == code
    assert not any(buf)


@needs_lib
def test_plan_buffer_is_checked():
    c, lib = _problem(), at._lib()
    n = lib.ipttt_attn_plan_bytes(ctypes.byref(c))
    buf = (ctypes.c_int64 * (n // 8 + 2))()
    assert lib.ipttt_attn_plan(ctypes.byref(c), None, n) == 6
    assert lib.ipttt_attn_plan(ctypes.byref(c), buf, n - 1) == 6
    assert lib.ipttt_attn_plan(ctypes.byref(c), ctypes.addressof(buf) + 4, n) == 4
    assert not any(buf)
    assert lib.ipttt_attn_workspace_bytes(buf) == 0 and lib.ipttt_attn_workspace_bytes(None) == 0
    assert lib.ipttt_attn_plan(ctypes.byref(c), buf, n) == 0


def _heads(data=256, row=256, head=64):
    return struct.pack("Pqq", data or 0, row, head)


@needs_lib
def test_attention_refuses_before_any_launch():
    """Bad arguments come back as status codes with no device present."""
    lib, v, nan = at._lib(), ctypes.c_void_p, float("nan")
    p = ip.AttentionPlan(4, 2, 64, [4, 6], [8, 12], device="cpu")
    shared = ip.AttentionPlan(4, 2, 64, [4, 6], [8, 12], k_starts=[0, 4], device="cpu")
    junk = (ctypes.c_int64 * 64)()

    def fwd(plan=p.ref, dev=v(256), scale=0.1, q=_heads(), k=_heads(), vv=_heads(), o=_heads(), lse=v(256),
            ws=v(256), n=1 << 30):
        return lib.ipttt_attention(plan, dev, scale, q, k, vv, o, lse, ws, n, None)

    assert fwd(plan=None) == 1 and fwd(dev=None) == 1 and fwd(q=None) == 1 and fwd(lse=None) == 1
    assert fwd(k=_heads(data=None)) == 1
    assert fwd(plan=junk) == 8 and fwd(scale=nan) == 8 and fwd(scale=0.0) == 8 and fwd(scale=-1.0) == 8
    assert fwd(dev=v(264)) == 4 and fwd(q=_heads(data=264)) == 4 and fwd(lse=v(260)) == 4
    for bad in (dict(row=56), dict(head=56), dict(row=260), dict(head=68), dict(row=0), dict(row=(1 << 22) + 8),
                dict(head=1 << 41)):
        assert fwd(o=_heads(**bad)) == 2, bad
    # the heads of a group are addressed with 32-bit offsets; of key heads, one at a time
    assert fwd(q=_heads(head=1 << 30)) == 2 and fwd(k=_heads(head=1 << 39), o=None) == 1

    def bwd(plan=p.ref, dO=_heads(), dk=_heads(), ws=v(256), n=p.backward_workspace_bytes):
        return lib.ipttt_attention_backward(plan, v(256), 0.1, _heads(), _heads(), _heads(), _heads(), v(256), dO,
                                            _heads(), dk, _heads(), ws, n, None)

    assert bwd(dO=None) == 1 and bwd(dk=_heads(data=8)) == 4
    assert bwd(ws=None) == 6 and bwd(n=p.backward_workspace_bytes - 1) == 6 and bwd(ws=v(272)) == 4
    assert bwd(plan=shared.ref) == 5          # two sequences' gradients would meet in the shared keys
    one = ip.AttentionPlan(4, 2, 64, [1], [4000], device="cpu")
    assert one.workspace_bytes > 0
    assert fwd(plan=one.ref, ws=None) == 6 and fwd(plan=one.ref, n=one.workspace_bytes - 1) == 6
    assert fwd(plan=one.ref, ws=v(272)) == 4


@needs_lib
def test_qk_refuses_before_any_launch():
    lib, v = at._lib(), ctypes.c_void_p

    def call(q=_heads(), k=_heads(512), w=v(256), pos=v(256), table=v(256), qo=_heads(1024), ko=_heads(2048),
             vi=None, vo=None, rows=None, **kw):
        c = dict(tokens=10, heads=4, kv_heads=2, head_dim=64, table_rows=9, out_rows=10, dtype=ip.IPTTT_BF16, eps=1e-6)
        c.update(kw)
        return lib.ipttt_qk_norm_rope(ctypes.byref(at._CQKProblem(**c)), q, k, w, v(256), pos, table, qo, ko, vi, vo,
                                      rows, None)

    assert lib.ipttt_qk_norm_rope(None, *([None] * 12)) == 1
    for kw, code in ((dict(dtype=2), 3), (dict(tokens=0), 2), (dict(tokens=1 << 26), 2), (dict(heads=0), 2),
                     (dict(head_dim=4), 2), (dict(head_dim=256), 2), (dict(table_rows=0), 2), (dict(out_rows=9), 2),
                     (dict(out_rows=-1), 2), (dict(eps=float("inf")), 8), (dict(eps=-1.0), 8), (dict(q=None), 1),
                     (dict(w=None), 1), (dict(pos=None), 1), (dict(table=None), 1), (dict(vi=_heads()), 1),
                     (dict(vo=_heads()), 1), (dict(pos=v(258)), 4), (dict(rows=v(258)), 4), (dict(table=v(260)), 4),
                     (dict(k=_heads(row=60)), 2), (dict(qo=_heads(256, row=512)), 8),
                     (dict(ko=_heads(512), rows=v(256)), 8)):
        assert call(**kw) == code, kw

    def back(dq=_heads(1024), dz=_heads(4096), dw=v(256), ws=v(256), n=None):
        c = at._CQKProblem(10, 4, 2, 64, 9, 10, ip.IPTTT_F32, 1e-6)
        n = lib.ipttt_qk_backward_workspace_bytes(ctypes.byref(c)) if n is None else n
        return lib.ipttt_qk_norm_rope_backward(ctypes.byref(c), _heads(), _heads(), v(256), v(256), v(256), v(256),
                                               dz, _heads(8192), dq, _heads(2048), dw, v(256), ws, n, None)

    assert back(dq=None) == 1 and back(dw=None) == 1 and back(dw=v(260)) == 4
    assert back(ws=None) == 6 and back(n=16) == 6 and back(ws=v(272)) == 4
    assert back(dq=_heads(4096, row=512)) == 8


@needs_lib
def test_binding_checks_tensors():
    import torch
    T, H, KV, D, N = 3, 4, 2, 64, 5
    p = ip.QKProblem(T, H, KV, D, table_rows=N)

    def qk(**bad):
        a = dict(q=torch.zeros(T, H, D), k=torch.zeros(T, KV, D), w_q=torch.zeros(D), w_k=torch.zeros(D),
                 positions=torch.zeros(T, dtype=torch.int32), table=torch.zeros(N, D), q_out=torch.zeros(T, H, D),
                 k_out=torch.zeros(T, KV, D))
        a = {n: x.bfloat16() if n not in ("positions", "table") else x for n, x in a.items()}
        a.update(bad)
        ip.ipttt_qk_norm_rope(p, **a)

    with pytest.raises(ValueError, match=r"^q must be a \[3, 4, 64\] BFloat16 device tensor"):   # not on a device
        qk()
    with pytest.raises(ValueError, match="go together"):
        qk(v=torch.zeros(T, KV, D))
    with pytest.raises(ValueError):
        ip.AttentionPlan(4, 2, 64, [1, 2], [1], device="cpu")
