"""What the compiler reports of the plain many-row attention kernels' registers (no GPU needed).

Their loop takes all 256 vector registers at D = 128 and nearly all scalar ones, so what is added to the shared body can push whole
groups of scalar registers out in every tile: seen as 96 and 112 spilled scalars, where 30 to 57 wait outside of the loop.
"""
import os
import re
import subprocess

import pytest

from bit_gemm_w4_amd import build


def test_no_scalar_groups_are_spilled(tmp_path):
    name = "k_kvattn_many.hip"
    if not os.path.exists(build.HIPCC):
        pytest.skip("no compiler")
    r = subprocess.run([build.HIPCC, *build.FLAGS, *build.FILE_FLAGS[name], "--cuda-device-only", "-S", "-Rpass-analysis=kernel-resource-usage",
                        os.path.join(build.CSRC, name), "-o", str(tmp_path / "k.s")], capture_output=True, text=True, check=True)
    kernels = re.findall(r"Function Name: (\S+).*?SGPRs Spill: (\d+).*?VGPRs Spill: (\d+)", r.stderr, re.S)
    assert len(kernels) == 12
    for kernel, scalars, vectors in kernels:
        assert int(scalars) <= 60 and int(vectors) <= 20, (kernel, scalars, vectors)
