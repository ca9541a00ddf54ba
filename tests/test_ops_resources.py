"""Register budget of the scan, norm and beam kernels: none spills or uses
scratch memory (see test_build_resources.py for the mixer's). CPU only."""
import os
import re
import subprocess

import pytest

from gated_deltanet_token_amd import build as gbuild


@pytest.mark.skipif(not os.path.exists(gbuild.hipcc()), reason="hipcc not available")
@pytest.mark.parametrize("src", ["gdn_scan.hip", "gdn_norm.hip", "gdn_beam.hip"])
def test_no_kernel_spills_registers(tmp_path, src):
    cmd = [gbuild.hipcc()] + gbuild.compile_flags() + [
        "-c", os.path.join(gbuild.CSRC, src), "-o", str(tmp_path / "k.o"),
        "-Rpass-analysis=kernel-resource-usage"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    name, seen, spills = None, 0, []
    for line in res.stderr.splitlines():
        m = re.search(r"Function Name: (\S+)", line)
        if m:
            name = m.group(1)
            seen += 1
        m = re.search(r"(VGPRs Spill|ScratchSize \[bytes/lane\]): (\d+)", line)
        if m and int(m.group(2)) > 0:
            spills.append((name, m.group(1), int(m.group(2))))
    assert seen > 0 and not spills, spills
