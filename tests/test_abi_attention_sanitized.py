"""The attention calls' argument checks under AddressSanitizer and
UndefinedBehaviorSanitizer (the build and the reasons are those of
test_abi_sanitized.py)."""
import os
import subprocess
import sys

import pytest

from fp4_block_scaled_x16_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(not os.path.exists(build.CLANG), reason="clang++ of ROCm not installed")
def test_attention_abi_checks_under_asan_and_ubsan():
    env = dict(os.environ, FP4_LIB=build.build_sanitized(), LD_PRELOAD=build.sanitizer_runtime(),
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    p = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_abi_attention.py")],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    report = p.stdout[-3000:] + p.stderr[-3000:]
    assert p.returncode == 0, report
    assert "runtime error" not in report and "AddressSanitizer" not in report, report
    assert " passed" in p.stdout
