"""The mixer operators' kernels keep their registers: they hold the whole state in
registers, and none may spill vector registers to scratch memory."""
import os
import re
import subprocess

import pytest

from selective_state_space_56_amd import build as B


@pytest.mark.parametrize("src", ["linattn_bf16.hip", "linattn_f32.hip", "linattn.hip", "linattn_update.hip", "qknorm.hip"])
def test_no_vector_register_spills(src, tmp_path):
    cmd = [B.hipcc()] + B.COMMON + B.DEVICE + ["-Rpass-analysis=kernel-resource-usage", "-c", os.path.join(B.CSRC, src),
                                               "-o", str(tmp_path / "k.o")]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    names = re.findall(r"Function Name: (\S+)", r.stderr)
    spills = [int(n) for n in re.findall(r"VGPRs Spill: (\d+)", r.stderr)]
    scratch = [int(n) for n in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", r.stderr)]
    assert names and len(names) == len(spills) == len(scratch)
    bad = [(n, s, m) for n, s, m in zip(names, spills, scratch) if s or m]
    assert not bad, bad
