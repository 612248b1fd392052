"""Calls of attention that take several launches: the arguments of each, from
attention_plan.hpp compiled for the CPU (attention_launches_check.cpp), under
UndefinedBehaviorSanitizer."""
import os
import subprocess

import pytest

from conftest import ROOT
from fp4_block_scaled_x16_amd import build


@pytest.mark.skipif(not os.path.exists(build.CLANG), reason="clang++ of ROCm not installed")
def test_launches_cover_every_request_once(tmp_path):
    exe = str(tmp_path / "launches")
    subprocess.run([build.CLANG, "-O2", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=undefined",
                    "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"),
                    "-I" + build.CSRC, os.path.join(ROOT, "tests", "attention_launches_check.cpp"), "-o", exe],
                   check=True, capture_output=True)
    p = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert p.returncode == 0, (p.stdout + p.stderr)[-3000:]
    assert int(p.stdout) > 512          # 2^31 - 1 requests alone take that many
