"""The host code of the rest of the block -- argument checks, workspace layouts --
under AddressSanitizer and UndefinedBehaviorSanitizer (CPU only)."""
import pytest
import torch

from test_host_sanitizers import _run, sanitized  # noqa: F401  (the fixture)

pytestmark = [pytest.mark.slow,
              pytest.mark.skipif(torch.cuda.is_available(), reason="host-only check: no device present")]


def test_block_host_tests_clean_under_asan_and_ubsan(sanitized):  # noqa: F811
    lib, env = sanitized
    out = _run(env, ["-m", "pytest", "-q", "-p", "no:cacheprovider", "tests/test_block_host.py"])
    assert " passed" in out and "failed" not in out
