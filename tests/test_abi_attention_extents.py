"""Outputs whose strides are so large that their extent passes 63 bits: whether rows
overlap is told without overflow.  Also under UndefinedBehaviorSanitizer."""
import os
import subprocess
import sys

import pytest

from fp4_block_scaled_x16_amd import build
from test_abi import lib  # noqa: F401 (fixture)
from test_abi_attention import ARG, SHAPE, back, heads, norm, rope, write

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAR = 1 << 61


def test_rows_overlap_at_strides_whose_product_wraps(lib):  # noqa: F811
    """Head h + 1 of a token and head h of the next lie on one another; 8 times the
    stride is 2^64."""
    for tokens, n in ((4, 9), (9, 4), (17, 17)):
        h, bad = heads(heads=n), heads(heads=n, token_stride=FAR, head_stride=FAR)
        assert rope(lib, tokens=tokens, q=h, qo=bad) == ARG and b"overlap" in lib.fp4_last_error()
        assert back(lib, tokens=tokens, q=h, dq=h, qi=bad) == ARG and b"overlap" in lib.fp4_last_error()
        assert write(lib, tokens=tokens, n=norm(), pos=0x10000, q=h, qo=bad) == ARG


def test_rows_apart_at_such_strides(lib):  # noqa: F811
    """Rows that do not overlap are not what such a call fails for (here: other heads)."""
    for ts, hs in ((FAR, 128), (128, FAR), (1 << 62, FAR)):
        out = heads(heads=2, token_stride=ts, head_stride=hs)
        assert rope(lib, tokens=2, q=heads(heads=4), qo=out) == SHAPE, (ts, hs, lib.fp4_last_error())


@pytest.mark.skipif(not os.path.exists(build.CLANG), reason="clang++ of ROCm not installed")
@pytest.mark.skipif("FP4_LIB" in os.environ, reason="this is the sanitized run")
def test_extents_under_asan_and_ubsan():
    env = dict(os.environ, FP4_LIB=build.build_sanitized(), LD_PRELOAD=build.sanitizer_runtime(),
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    p = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", os.path.abspath(__file__)],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    report = p.stdout[-3000:] + p.stderr[-3000:]
    assert p.returncode == 0 and "runtime error" not in report and " passed" in p.stdout, report
