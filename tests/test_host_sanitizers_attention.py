"""The attention half's host code -- argument checks, the plan's counting,
filling and sorting, workspace sizes -- under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only)."""
import textwrap

import pytest
import torch

from test_host_sanitizers import _run, sanitized  # noqa: F401  (the fixture)

pytestmark = [pytest.mark.slow,
              pytest.mark.skipif(torch.cuda.is_available(), reason="host-only check: no device present")]


def test_attention_host_tests_clean_under_asan_and_ubsan(sanitized):  # noqa: F811
    lib, env = sanitized
    out = _run(env, ["-m", "pytest", "-q", "-p", "no:cacheprovider", "tests/test_attention_host.py"])
    assert " passed" in out and "failed" not in out


def test_plans_of_random_sequences_stay_in_their_buffers(sanitized):  # noqa: F811
    """Plans written to buffers of exactly their size, over random heads and
    lengths, zero lengths among them."""
    lib, env = sanitized
    code = textwrap.dedent("""
        import random
        import numpy as np
        import test_weight_mlp_amd as ip
        r = random.Random(0)
        for i in range(200):
            kv = r.choice([1, 2, 3, 8])
            n = r.randint(1, 12)
            ql = [r.choice([0, 1, 2, 5, r.randint(0, 3000)]) for _ in range(n)]
            kl = [r.choice([0, 1, q, r.randint(0, 9000)]) for q in ql]
            p = ip.AttentionPlan(kv * r.choice([1, 2, 4, 7, 32]), kv, r.choice([8, 64, 128]), ql, kl,
                                 r.choice([0, 1]), device="cpu")
            assert p.workspace_bytes % 256 == 0 and p.backward_workspace_bytes % 256 == 0
        print("done", i)
    """)
    assert "done 199" in _run(env, ["-c", code])
