"""The refusals and workspace arithmetic of the dense feed-forward operators
(tests/test_dense_host.py) against the host sources built with AddressSanitizer
and UndefinedBehaviorSanitizer, as tests/test_host_sanitized.py does for the rest."""
import os
import subprocess
import sys

import pytest

from test_host_sanitized import ROOT, _runtime


def test_dense_host_tests_pass_under_asan_and_ubsan():
    from quantized_routed_expert_fp32_amd.csrc import build as B
    asan, ubsan = _runtime("libasan.so"), _runtime("libubsan.so")
    if not asan or not ubsan:
        pytest.skip("the sanitizer runtimes are not installed with g++")
    env = dict(os.environ)
    env.update(MOE_LIBRARY=B.build_host_sanitized(), LD_PRELOAD=f"{asan}:{ubsan}",
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_dense_host.py")],
                       capture_output=True, text=True, env=env, cwd=ROOT, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "runtime error" not in out and "AddressSanitizer" not in out, out[-4000:]
    assert " passed" in out
