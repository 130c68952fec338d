"""Host checks of the attention half's calls and plans (no GPU): what the binding
and the C entries refuse, and what a plan may not depend on."""
import ctypes
import os
import struct
import subprocess
import sys

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import test_weight_mlp_amd as ip
from test_attention_host import Plan
from test_weight_mlp_amd import attention as at

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
needs_lib = pytest.mark.skipif(not os.path.exists(ip.library_path), reason="libipttt.so not built")


@needs_lib
def test_binding_refuses_a_plan_that_is_not_on_the_device():
    """The kernels would read its items through a host pointer: the calls look at
    the plan's table before anything else and launch nothing."""
    T, H, KV, D = 4, 4, 2, 64
    plan = ip.AttentionPlan(H, KV, D, [T], [T], device="cpu")
    b = ip.AttentionBuffers(plan, grads=True, device="cpu")
    q, k = torch.zeros(T, H, D).bfloat16(), torch.zeros(T, KV, D).bfloat16()
    with pytest.raises(ValueError, match="^the plan's table must be a contiguous device tensor"):
        ip.ipttt_attention(plan, q, k, k, b.o, b.lse, b.ws)
    with pytest.raises(ValueError, match="^the plan's table must be a contiguous device tensor"):
        ip.ipttt_attention_backward(plan, q, k, k, b.o, b.lse, q, b.dq, b.dk, b.dv, b.ws)


class _Stream:
    cuda_stream = 0


def _calls(device):
    """Every launching call with its tensors on a device that need not be there:
    tensors without memory, whose null pointers the C entries refuse."""
    T, H, KV, D = 4, 4, 2, 64
    p = ip.QKProblem(T, H, KV, D, table_rows=6)
    plan = ip.AttentionPlan(H, KV, D, [T], [T], device="cpu")
    with FakeTensorMode():
        def z(*s, t=torch.bfloat16):
            return torch.zeros(s, dtype=t, device=device)

        f32, i32, u8 = torch.float32, torch.int32, torch.uint8
        table = torch.zeros(plan.table.shape, dtype=plan.table.dtype, device=device)
        base = dict(q=z(T, H, D), k=z(T, KV, D), w_q=z(D), w_k=z(D), positions=z(T, t=i32), table=z(6, D, t=f32))
        qk = dict(base, q_out=z(T, H, D), k_out=z(T, KV, D), v=z(T, KV, D), v_out=z(T, KV, D), rows=z(T, t=i32))
        back = dict(base, dq_out=z(T, H, D), dk_out=z(T, KV, D), dq=z(T, H, D), dk=z(T, KV, D), dw_q=z(D, t=f32),
                    dw_k=z(D, t=f32), ws=z(1 << 20, t=u8))
        fwd = dict(q=z(T, H, D), k=z(T, KV, D), v=z(T, KV, D), o=z(T, H, D), lse=z(T, H, t=f32), ws=z(1 << 20, t=u8))
        bwd = dict(fwd, dO=z(T, H, D), dq=z(T, H, D), dk=z(T, KV, D), dv=z(T, KV, D))
    plan.table = table
    return [(lambda a: ip.ipttt_qk_norm_rope(p, **a, stream=_Stream), qk),
            (lambda a: ip.ipttt_qk_norm_rope_backward(p, **a, stream=_Stream), back),
            (lambda a: ip.ipttt_attention(plan, **a, stream=_Stream), fwd),
            (lambda a: ip.ipttt_attention_backward(plan, **a, stream=_Stream), bwd)]


@needs_lib
@pytest.mark.filterwarnings("ignore")
def test_binding_refuses_tensors_of_two_devices(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    for (call, args), (_, others) in zip(_calls("cuda:0"), _calls("cuda:1")):
        for name in args:
            # q decides which device is the call's; in the norm it is the first tensor
            what = "q is on device 1, the current device is 0" if name == "q" else f"{name} must be on device 0"
            with pytest.raises(ValueError, match="^" + what):
                call(dict(args, **{name: others[name]}))


@needs_lib
def test_binding_refuses_tensors_that_are_not_on_the_current_device(monkeypatch):
    """Kernels go to the current device, where another one's memory need not be mapped."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    for call, args in _calls("cuda:1"):
        with pytest.raises(ValueError, match="on device 1, the current device is 0"):
            call(args)


def _heads(data, row=128, head=64):
    return struct.pack("Pqq", data, row, head)


@needs_lib
@pytest.mark.parametrize("v_out,rows", [(_heads(4096), 256), (_heads(4096, row=256), None),
                                        (_heads(4096, head=192), None)], ids=["rows", "row stride", "head stride"])
def test_values_over_themselves_are_refused_unless_row_for_row(v_out, rows):
    """Other waves' rows are still to be read while this one's are written."""
    c = at._CQKProblem(10, 4, 2, 64, 9, 10, ip.IPTTT_BF16, 1e-6)
    ptr = ctypes.c_void_p
    assert at._lib().ipttt_qk_norm_rope(ctypes.byref(c), _heads(256, row=256), _heads(512), ptr(256), ptr(256), ptr(256),
                                        ptr(256), _heads(1024, row=256), _heads(2048), _heads(4096), v_out, ptr(rows),
                                        None) == 8


def _beside_idle(ql, kl, dt):
    """The plan of these sequences, and with a pool's idle slots after them."""
    idle = 31
    return (Plan(ip.AttentionPlan(32, 8, 128, q, k, dt, device="cpu"))
            for q, k in ((ql, kl), (ql + [0] * idle, kl + [16000] * idle)))


@needs_lib
@pytest.mark.parametrize("dt", [ip.IPTTT_BF16, ip.IPTTT_F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("ql,kl", [([1], [4097]), ([1, 2, 1], [700, 5000, 64]), ([1, 900], [4000, 900])])
def test_sequences_without_queries_do_not_change_the_forward_of_others(ql, kl, dt):
    alone, beside = _beside_idle(ql, kl, dt)
    assert beside.few == alone.few and beside.rows == alone.rows and beside.join == alone.join


@needs_lib
@pytest.mark.parametrize("dt", [ip.IPTTT_BF16, ip.IPTTT_F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("ql,kl", [([1000], [1000]), ([300, 41], [300, 90])])
def test_sequences_without_queries_do_not_change_the_backward_of_others(ql, kl, dt):
    """Their keys' tiles only write zeros, and fill no CU."""
    alone, beside = _beside_idle(ql, kl, dt)
    assert beside.dq == alone.dq and beside.dq_join == alone.dq_join and beside.key_join == alone.key_join
    assert [x for x in beside.key if x["q_len"] > 0] == alone.key
    assert len(beside.key) == len(alone.key) + 31 * 125


def test_package_imports_where_torch_has_no_raw_stream():
    """Builds of torch without devices lack the name; it is looked up by the first
    call on a device tensor."""
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'): del torch._C._cuda_getCurrentRawStream\n"
            "import test_weight_mlp_amd as ip\n"
            "print(ip.Problem(1, 8, 64, 128, 8).rows, ip.AttentionPlan.__name__)\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT, timeout=100)
    assert r.returncode == 0 and r.stdout.split() == ["1", "AttentionPlan"], r.stderr


def test_library_is_linked_where_the_marshalling_module_cannot_be_built(monkeypatch, tmp_path):
    """The layer needs only the library, which needs only hipcc; the missing half is
    reported once that is there."""
    from test_weight_mlp_amd import build as b
    lib = tmp_path / "libipttt.so"
    monkeypatch.setattr(b, "LIB", str(lib))
    monkeypatch.setattr(b, "OBJDIR", str(tmp_path))
    monkeypatch.setattr(b, "hipcc", lambda: "hipcc")
    monkeypatch.setattr(b, "_compile", lambda src, sanitize=False: src)

    def no_compiler(verbose=False):
        raise FileNotFoundError("c++")

    def link(cmd, **kw):
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(b, "build_marshal", no_compiler)
    monkeypatch.setattr(b.subprocess, "run", link)
    with pytest.raises(RuntimeError, match="libipttt.so is built.*attention"):
        b.build(jobs=2)
    assert lib.exists()


@needs_lib
@pytest.mark.parametrize("heads,kv,dim,ql,kl,dt", [(32, 8, 64, [1800], [1800], ip.IPTTT_BF16),
                                                   (16, 8, 64, [3900], [3900], ip.IPTTT_F32),
                                                   (16, 8, 64, [300, 700], [4000, 700], ip.IPTTT_BF16)])
def test_calls_of_two_workgroups_a_cu_fold_their_order(heads, kv, dim, ql, kl, dt):
    """257 to 512 workgroups start together, the later ones second on a CU: the
    longest tiles come first, then the others from the shortest."""
    pl = Plan(ip.AttentionPlan(heads, kv, dim, ql, kl, dt, device="cpu"))
    assert 256 < len(pl.rows) * kv <= 512
    keys = [x["k_end"] - x["k_begin"] for x in pl.rows]
    first, second = keys[:256 // kv], keys[256 // kv:]
    assert first == sorted(first, reverse=True) and second == sorted(second) and min(first) >= max(second)
