"""Host checks of the rest of the block (no GPU): the definitions' gradients
against differences, and what the C entries and the binding refuse before any
launch."""
import ctypes
import os

import numpy as np
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import test_weight_mlp_amd as ip
from oracle import block as ob
from test_weight_mlp_amd import block as bk

needs_lib = pytest.mark.skipif(not os.path.exists(ip.library_path), reason="libipttt.so not built")
OK, NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, ARG = 0, 1, 2, 3, 4, 6, 8


# ------------------------------------------------------------- definitions

def differences(f, x, dy, h=1e-6):
    """The gradient of <f(x), dy> by central differences."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + h
        up = (f() * dy).sum()
        x[i] = keep - h
        g[i] = (up - (f() * dy).sum()) / (2 * h)
        x[i] = keep
    return g


def near(a, b):
    return np.abs(a - b).max() <= 1e-7 * max(1.0, np.abs(b).max())


@pytest.mark.parametrize("center", [False, True])
def test_norm_gradients_of_the_definition(center):
    r = np.random.default_rng(0)
    x, w, b, dy, dres = r.normal(size=(3, 8)) + 0.5, r.normal(size=8), r.normal(size=8), r.normal(size=(3, 8)), None
    dx, dw, db = ob.norm_backward(x, w, dy, dres, center, 1e-3)
    for a, g in ((x, dx), (w, dw), (b, db)):
        assert near(differences(lambda: ob.norm(x, w, b, center, 1e-3), a, dy), g)
    more = r.normal(size=(3, 8))
    assert np.array_equal(ob.norm_backward(x, w, dy, more, center, 1e-3)[0], dx + more)


@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
def test_linear_gradients_of_the_definition(kind):
    r = np.random.default_rng(1)
    x, W, b, dy = r.normal(size=(3, 8)), r.normal(size=(16, 8)), r.normal(size=16), r.normal(size=(3, 16))
    _, pre = ob.linear(x, W, b, None, kind)
    for a, g in zip((x, W, b), ob.linear_backward(x, W, pre, dy, kind)):
        assert near(differences(lambda: ob.linear(x, W, b, None, kind)[0], a, dy), g)


def test_activations_far_out():
    v = np.array([-800.0, -40.0, 0.0, 40.0, 800.0])
    for kind in ("silu", "gelu"):
        assert np.allclose(ob.act(kind, v), [0, 0, 0, 40, 800]) and np.allclose(ob.slope(kind, v), [0, 0, 0.5, 1, 1])


def test_kept_values():
    g = np.array([[127.0, -63.5, 1.4, 1.6, 0.0] + [0.0] * 60 + [2.54, 1.0]])
    k = ob.kept8(g)
    assert k[0, :5].tolist() == [127.0, -64.0, 1.0, 2.0, 0.0]     # a tie goes away from zero
    assert np.allclose(k[0, 64:], [0.0, 2.54, 1.0])               # the second block: multiples of 0.02
    assert not ob.kept8(np.zeros((2, 70))).any()


def test_kept_values_of_ties():
    """Halves go to the even integer, as torch.round takes them."""
    g = np.array([[127.0, 0.5, -0.5, 1.5, -2.5, 62.5, 63.5, -126.5] + [0.0] * 56])
    assert ob.kept8(g)[0, :8].tolist() == [127.0, 0.0, 0.0, 2.0, -2.0, 62.0, 64.0, -126.0]


# ------------------------------------------------------------ the C entries

class Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64)]


def at(i):
    """A 256-byte aligned address that nothing may read."""
    return 0x7000000000 + (i << 32)


def rows(i, stride):
    return Rows(at(i), stride)


def pack(r):
    return None if r is None else ctypes.cast(ctypes.byref(r), ctypes.c_char_p)


def norm_call(p=None, x=rows(1, 64), w=at(2), b=at(3), y=rows(4, 64)):
    p = ip.NormProblem(4, 64) if p is None else p
    return bk._lib().ipttt_norm(p.ref, pack(x), w, b, pack(y), None)


def norm_backward_call(p=None, x=rows(1, 64), w=at(2), dy=rows(3, 64), dres=rows(4, 64), dx=rows(5, 64), dw=at(6),
                       db=at(7), ws=at(8), ws_bytes=1 << 30):
    p = ip.NormProblem(4, 64) if p is None else p
    return bk._lib().ipttt_norm_backward(p.ref, pack(x), w, pack(dy), pack(dres), pack(dx), dw, db, ws, ws_bytes, None)


def linear_call(p=None, x=rows(1, 64), W=at(2), b=at(3), res=rows(4, 128), y=rows(5, 128), pre=rows(6, 128), ws=at(7),
                ws_bytes=1 << 40):
    p = ip.LinearProblem(4, 64, 128) if p is None else p
    return bk._lib().ipttt_linear(p.ref, pack(x), W, b, pack(res), pack(y), pack(pre), ws, ws_bytes, None)


def linear_backward_call(p=None, x=rows(1, 64), W=at(2), pre=rows(3, 128), dy=rows(4, 128), dx=rows(5, 64), dW=at(6),
                         db=at(7), ws=at(8), ws_bytes=1 << 40):
    p = ip.LinearProblem(4, 64, 128, act=ip.IPTTT_ACT_GELU) if p is None else p
    return bk._lib().ipttt_linear_backward(p.ref, pack(x), W, pack(pre), pack(dy), pack(dx), dW, db, ws, ws_bytes, None)


NORM_PROBLEMS = [(dict(rows=0), SHAPE), (dict(rows=-1), SHAPE), (dict(rows=(1 << 26) - 3), SHAPE), (dict(dim=0), SHAPE),
                 (dict(dim=12), SHAPE), (dict(dim=16392), SHAPE), (dict(dtype=2), DTYPE), (dict(dtype=-1), DTYPE),
                 (dict(kind=2), ARG), (dict(kind=-1), ARG), (dict(eps=-1e-6), ARG), (dict(eps=float("nan")), ARG),
                 (dict(eps=float("inf")), ARG)]
LINEAR_PROBLEMS = [(dict(rows=0), SHAPE), (dict(rows=(1 << 26) - 3), SHAPE), (dict(in_dim=4), SHAPE),
                   (dict(in_dim=68), SHAPE), (dict(in_dim=(1 << 20) + 8), SHAPE), (dict(out_dim=0), SHAPE),
                   (dict(out_dim=129), SHAPE), (dict(out_dim=1 << 21), SHAPE), (dict(rows=1 << 25, out_dim=1 << 20), SHAPE),
                   (dict(in_dim=1 << 20, out_dim=1 << 20), SHAPE), (dict(dtype=2), DTYPE), (dict(act=3), ARG),
                   (dict(act=-1), ARG), (dict(grad_dtype=2), DTYPE), (dict(dtype=ip.IPTTT_F32, grad_dtype=ip.IPTTT_BF16), DTYPE)]


@needs_lib
@pytest.mark.parametrize("change, status", NORM_PROBLEMS)
def test_norm_problems_refused(change, status):
    p = ip.NormProblem(**dict(dict(rows=4, dim=64), **change))
    assert norm_call(p) == status and norm_backward_call(p) == status
    assert ip.ipttt_norm_backward_workspace_bytes(p) == 0


@needs_lib
@pytest.mark.parametrize("change, status", LINEAR_PROBLEMS)
def test_linear_problems_refused(change, status):
    p = ip.LinearProblem(**dict(dict(rows=4, in_dim=64, out_dim=128), **change))
    assert linear_call(p) == status and linear_backward_call(p) == status
    assert ip.ipttt_linear_workspace_bytes(p) == 0 and ip.ipttt_linear_backward_workspace_bytes(p) == 0


def bad_rows(name, i, width):
    """A row tensor's refusals: no data, an odd address, strides too short, odd and too long."""
    return [({name: Rows(None, width)}, NULL), ({name: Rows(at(i) + 8, width)}, ALIGN), ({name: rows(i, width - 8)}, SHAPE),
            ({name: rows(i, width + 4)}, SHAPE), ({name: rows(i, (1 << 22) + 8)}, SHAPE), ({name: rows(i, -width)}, SHAPE)]


NORM_ARGS = bad_rows("x", 1, 64) + bad_rows("y", 4, 64) + [
    (dict(x=None), NULL), (dict(y=None), NULL), (dict(w=at(2) + 8), ALIGN), (dict(b=at(3) + 4), ALIGN),
    (dict(y=rows(1, 72)), ARG)]
NORM_BACKWARD_ARGS = sum((bad_rows(n, i, 64) for n, i in (("x", 1), ("dy", 3), ("dres", 4), ("dx", 5))), []) + [
    (dict(x=None), NULL), (dict(dy=None), NULL), (dict(dx=None), NULL), (dict(w=at(2) + 8), ALIGN),
    (dict(dw=at(6) + 4), ALIGN), (dict(db=at(7) + 4), ALIGN), (dict(dx=rows(3, 72)), ARG), (dict(dx=rows(4, 72)), ARG),
    (dict(dx=rows(1, 72)), ARG), (dict(ws=None), WORKSPACE), (dict(ws_bytes=64), WORKSPACE), (dict(ws=at(8) + 16), ALIGN)] + [
    (dict([(n, at(i))]), ARG) for n, other in (("dw", 7), ("db", 6)) for i in (1, 2, 3, 4, 5, other)]
LINEAR_ARGS = bad_rows("x", 1, 64) + sum((bad_rows(n, i, 128) for n, i in (("res", 4), ("y", 5), ("pre", 6))), []) + [
    (dict(x=None), NULL), (dict(W=None), NULL), (dict(y=None), NULL), (dict(W=at(2) + 8), ALIGN), (dict(b=at(3) + 2), ALIGN),
    (dict(y=rows(1, 128)), ARG), (dict(y=rows(2, 128)), ARG), (dict(y=rows(3, 128)), ARG), (dict(y=rows(4, 136)), ARG),
    (dict(pre=rows(1, 128)), ARG), (dict(pre=rows(4, 128)), ARG), (dict(pre=rows(5, 128)), ARG)]
LINEAR_BACKWARD_ARGS = bad_rows("x", 1, 64) + bad_rows("pre", 3, 128) + bad_rows("dy", 4, 128) + bad_rows("dx", 5, 64) + [
    (dict(x=None), NULL), (dict(W=None), NULL), (dict(pre=None), NULL), (dict(dy=None), NULL), (dict(W=at(2) + 8), ALIGN),
    (dict(dW=at(6) + 8), ALIGN), (dict(db=at(7) + 8), ALIGN), (dict(dx=rows(1, 64)), ARG), (dict(dx=rows(4, 64)), ARG),
    (dict(dW=at(2)), ARG), (dict(dW=at(5)), ARG), (dict(db=at(6)), ARG), (dict(db=at(4)), ARG), (dict(ws=None), WORKSPACE),
    (dict(ws_bytes=1024), WORKSPACE), (dict(ws=at(8) + 16), ALIGN)]


@needs_lib
@pytest.mark.parametrize("call, args", [(norm_call, NORM_ARGS), (norm_backward_call, NORM_BACKWARD_ARGS),
                                        (linear_call, LINEAR_ARGS), (linear_backward_call, LINEAR_BACKWARD_ARGS)],
                         ids=["norm", "norm_backward", "linear", "linear_backward"])
def test_arguments_refused(call, args):
    for change, status in args:
        assert call(**change) == status, change


@needs_lib
@pytest.mark.parametrize("call, change", [(norm_call, dict(y=rows(2, 64))), (norm_call, dict(y=rows(3, 64))),
                                          (norm_backward_call, dict(dx=rows(2, 64)))], ids=["y over w", "y over b", "dx over w"])
def test_norm_outputs_over_a_weight_refused(call, change):
    assert call(**change) == ARG


@needs_lib
def test_problem_pointer_may_not_be_null():
    L, r = bk._lib(), rows(1, 64)
    assert L.ipttt_norm(None, pack(r), None, None, pack(r), None) == NULL
    assert L.ipttt_norm_backward(None, pack(r), None, pack(r), None, pack(r), None, None, None, 0, None) == NULL
    assert L.ipttt_linear(None, pack(r), at(1), None, None, pack(r), None, None, 0, None) == NULL
    assert L.ipttt_linear_backward(None, pack(r), at(1), None, pack(r), None, None, None, None, 0, None) == NULL
    assert L.ipttt_linear_workspace_bytes(None) == 0 and L.ipttt_norm_backward_workspace_bytes(None) == 0


@needs_lib
def test_8_bits_are_for_bf16_and_need_their_buffer():
    lib = ip.library()
    p = ip.Problem(1, 100, 64, 200, 16)
    need = ip.ipttt_saved8_bytes(p)
    # integers of G and U, four scales a token for each, the regions 256-byte aligned
    assert need == 2 * (20224 + 1792)

    def save(p=p, kept=at(5), n=need):
        return lib.ipttt_z_save8(p.ref, at(1), at(2), at(3), at(4), kept, n, None)

    def back(p=p, kept=at(5), n=need, ws=at(9)):
        return lib.ipttt_z_backward_saved8(p.ref, at(1), at(2), at(3), kept, n, at(4), at(6), at(7), at(8), ws, 1 << 40, None)

    for f in (save, back):
        assert f(kept=None) == NULL and f(n=need - 1) == WORKSPACE and f(kept=at(5) + 16) == ALIGN
        assert f(p=ip.Problem(1, 100, 64, 200, 16, ip.IPTTT_F32)) == DTYPE
        assert f(p=ip.Problem(1, 0, 64, 200, 16)) == SHAPE
    assert back(ws=None) == WORKSPACE
    assert ip.ipttt_saved8_bytes(ip.Problem(1, 100, 64, 200, 16, ip.IPTTT_F32)) == 0
    with pytest.raises(ValueError, match="keep8"):
        ip.allocate(ip.Problem(1, 100, 64, 200, 16, ip.IPTTT_F32), "cpu", save=True, keep8=True)
    with pytest.raises(ValueError, match="keep8"):
        ip.allocate(p, "cpu", keep8=True)
    b = ip.allocate(p, "cpu", save=True, keep8=True)
    assert b.GU is None and b.GU8.numel() == need


@needs_lib
def test_8_bits_add_nothing_to_the_backward_workspace_of_the_others():
    """A shape of the general path whose largest backward call is Z's: its transposes
    take more than the 8-bit products' parts, which lie in the same place."""
    t, d, f, c = 16384, 72, 4104, 512

    def r(n):
        return -(-n // 256) * 256

    own = 2 * r(t * f * 2) + 2 * r(d * f * 2) + 2 * r(t * f * 2) + r(t * d * 2)
    assert ip.ipttt_backward_workspace_bytes(ip.Problem(1, t, d, f, c)) == r(t) + r(t // c * 12) + own


@needs_lib
@pytest.mark.skipif(torch.cuda.is_available(), reason="host-only check: the addresses are none of a device's")
def test_8_bits_backward_asks_for_its_own_workspace_only():
    lib, t, d, f = ip.library(), 16384, 72, 4104
    p = ip.Problem(1, t, d, f, 512)
    need = ip.ipttt_saved8_bytes(p)

    def back(n):
        return lib.ipttt_z_backward_saved8(p.ref, at(1), at(2), at(3), at(5), need, at(4), at(6), at(7), at(8), at(9), n, None)

    # dG, dU and at most two tiles of 128 x 128 floats a compute unit for either product
    assert back(2 * t * f * 2 - 1) == WORKSPACE
    assert back(2 * t * f * 2 + 2 * 512 * 65536) not in (OK, WORKSPACE)


# --------------------------------------------------------------- the binding

class _Stream:
    cuda_stream = 0


def _calls(device, dt=torch.bfloat16):
    """Every launching call with tensors on a device that need not be there: tensors
    without memory, whose null pointers the C entries refuse."""
    M, K, N = 4, 64, 128
    norm, lin = ip.NormProblem(M, K), ip.LinearProblem(M, K, N, act=ip.IPTTT_ACT_SILU)
    with FakeTensorMode():
        def z(*s, t=dt):
            return torch.zeros(s, dtype=t, device=device)

        f32, u8 = torch.float32, torch.uint8
        fwd = dict(x=z(M, K), w=z(K), b=z(K), y=z(M, K))
        back = dict(x=z(M, K), w=z(K), dy=z(M, K), dx=z(M, K), dw=z(K, t=f32), db=z(K, t=f32), ws=z(1 << 16, t=u8), dres=z(M, K))
        lfwd = dict(x=z(M, K), W=z(N, K), y=z(M, N), b=z(N), res=z(M, N), pre=z(M, N), ws=z(1 << 16, t=u8))
        lback = dict(x=z(M, K), W=z(N, K), dy=z(M, N), dx=z(M, K), dW=z(N, K), db=z(N, t=f32), ws=z(1 << 16, t=u8), pre=z(M, N))
    return [(lambda a: ip.ipttt_norm(norm, **a, stream=_Stream), fwd),
            (lambda a: ip.ipttt_norm_backward(norm, **a, stream=_Stream), back),
            (lambda a: ip.ipttt_linear(lin, **a, stream=_Stream), lfwd),
            (lambda a: ip.ipttt_linear_backward(lin, **a, stream=_Stream), lback)]


@needs_lib
@pytest.mark.filterwarnings("ignore")
def test_binding_refuses_tensors_of_two_devices_or_of_another(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    for (call, args), (_, others) in zip(_calls("cuda:0"), _calls("cuda:1")):
        for name in args:
            what = "x is on device 1, the current device is 0" if name == "x" else f"{name} must be on device 0"
            with pytest.raises(ValueError, match="^" + what):
                call(dict(args, **{name: others[name]}))


@needs_lib
@pytest.mark.filterwarnings("ignore")
def test_binding_refuses_shapes_types_and_strides(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    for (call, args), (_, doubles) in zip(_calls("cuda:0"), _calls("cuda:0", torch.float64)):
        for name, t in args.items():
            if name == "ws":
                continue
            with FakeTensorMode():
                wrong = [torch.zeros([s + 8 for s in t.shape], dtype=t.dtype, device="cuda:0"),
                         torch.zeros(t.shape, dtype=torch.float16, device="cuda:0"),
                         torch.zeros(tuple(t.shape) + (1,), dtype=t.dtype, device="cuda:0"),
                         torch.zeros(tuple(t.shape)[::-1], dtype=t.dtype, device="cuda:0").t() if t.dim() == 2 else
                         torch.zeros(2 * t.numel(), dtype=t.dtype, device="cuda:0")[::2]]
            for w in wrong:
                with pytest.raises(ValueError, match=f"^{name} must be"):
                    call(dict(args, **{name: w}))
            with pytest.raises(TypeError, match=f"^{name} must be a tensor"):
                call(dict(args, **{name: 3}))
        with pytest.raises(ip.IptttError):   # tensors without memory
            call(args)


@needs_lib
def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64).bfloat16()
    with pytest.raises(ValueError, match="^x must be"):
        ip.ipttt_norm(ip.NormProblem(4, 64), x, None, None, x)
    with pytest.raises(ValueError, match="^x must be"):
        ip.ipttt_linear(ip.LinearProblem(4, 64, 64), x, torch.zeros(64, 64).bfloat16(), x)
