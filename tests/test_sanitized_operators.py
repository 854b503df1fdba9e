"""The host side of the dense linear's and the gradient list's C ABI under
AddressSanitizer and UndefinedBehaviorSanitizer: tests/test_operators_abi.py
again in a child process against the host-sanitized build (CPU only; see
test_sanitized_abi.py, which does the same for the POET-X layer's calls)."""
import os
import subprocess
import sys

import pytest

from tests.test_sanitized_abi import ROOT, _stale


def test_operators_abi_under_host_sanitizers():
    import torch
    if torch.cuda.is_available():
        pytest.skip("host-validation tests use fake device addresses; run them without a GPU")
    from orthogonal_equivalence_amd import build as B
    try:
        B.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available to build the sanitized library")
    if _stale(B.SAN_LIB):
        B.build(sanitize=True)
    env = dict(os.environ)
    env.update(POETX_LIBRARY=B.SAN_LIB, LD_PRELOAD=B.sanitizer_runtime(),
               ASAN_OPTIONS="detect_leaks=0:detect_odr_violation=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_operators_abi.py")],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout[-4000:] + r.stderr[-4000:]
    assert r.returncode == 0, out
    assert "passed" in r.stdout and "AddressSanitizer" not in out and "runtime error" not in out, out
