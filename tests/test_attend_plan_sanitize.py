"""The attention's own plan under AddressSanitizer and UndefinedBehaviorSanitizer: attend_plan.cpp with two million sizes that
the entry point lets through (tests/c/attend_plan_validate.cpp). No GPU and no kernel is involved."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-fno-omit-frame-pointer", "-g", "-O1"]
INC = ["-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", f"-I{os.path.join(ROOT, 'include')}"]


def test_attention_plan_under_sanitizers(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("no host compiler or HIP headers")
    exe = str(tmp_path / "attend_plan_validate")
    sources = [os.path.join(ROOT, "rank_recurrent_state_amd", "csrc", "attend_plan.cpp"), os.path.join(ROOT, "tests", "c", "attend_plan_validate.cpp")]
    res = subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", *SAN, *INC, *sources, "-o", exe], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1")
    res = subprocess.run([exe], capture_output=True, text=True, timeout=120, env=env)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "attend_plan_validate ok" in res.stdout
