"""Host checks of the attention half's calls and plans (no GPU): what the binding
and the C entries refuse, and what a plan may not depend on."""
import os

import pytest
import torch

import test_weight_mlp_amd as ip

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
