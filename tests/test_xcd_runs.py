"""The scan kernels' mapping of workgroups to chains, walked on the host (CPU only)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_every_chain_is_taken_once(tmp_path):
    exe = str(tmp_path / "check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-o", exe,
                    os.path.join(HERE, "xcd_runs_check.cpp")], check=True)
    res = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0 and "xcd runs ok" in res.stdout, res.stdout


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_slots_and_waits_stay_in_bounds(tmp_path):
    """Malformed offsets, counts from an overwritten counter, words that never come."""
    exe = str(tmp_path / "bounds")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", "-Wno-unknown-pragmas", "-o", exe,
                    os.path.join(HERE, "split_check.cpp")], check=True)
    res = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0 and "bounds ok" in res.stdout, res.stdout + res.stderr
