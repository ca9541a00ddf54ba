"""The argument checks of the scan, norm and beam calls under AddressSanitizer
and UndefinedBehaviorSanitizer (host code, CPU only)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_checks_under_sanitizers(tmp_path):
    inc = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include")
    exe = str(tmp_path / "ops")
    subprocess.run(["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", inc, "-o", exe,
                    os.path.join(ROOT, "tests", "ops_sanitize.cpp"),
                    "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-g", "-O1"],
                   check=True)
    res = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0 and "sanitized checks ok" in res.stdout, res.stdout + res.stderr
