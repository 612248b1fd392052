"""How attention shares the tokens of requests: attention_plan.hpp, which the host and the
kernels have in common, compiled for the CPU and run over sizes and lengths of the whole
range (attention_plan_check.cpp), under UndefinedBehaviorSanitizer."""
import os
import subprocess

import pytest

from conftest import ROOT
from fp4_block_scaled_x16_amd import build

DRAWS = 20000


@pytest.mark.skipif(not os.path.exists(build.CLANG), reason="clang++ of ROCm not installed")
def test_parts_are_those_that_there_is_room_for(tmp_path):
    """No lengths give more parts than the plan, by which the launch and the workspace are
    sized, and the parts of a request are together the whole of it."""
    exe = str(tmp_path / "plan")
    subprocess.run([build.CLANG, "-O2", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=undefined",
                    "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"),
                    "-I" + build.CSRC, os.path.join(ROOT, "tests", "attention_plan_check.cpp"), "-o", exe],
                   check=True, capture_output=True)
    p = subprocess.run([exe, str(DRAWS)], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, (p.stdout + p.stderr)[-3000:]
    quotients, planned, longer, even, part = (int(v) for v in p.stdout.split())
    # each way of sharing came up often, and parts of more than 2^12 steps of 128 tokens
    assert quotients == 3 * 200 * DRAWS and min(planned, longer, even) >= DRAWS // 20 and part > 1 << 19
