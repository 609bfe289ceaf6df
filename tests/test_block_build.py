"""The block operators' kernels keep their registers: none may spill vector
registers to scratch memory. The kernels hold whole tiles in registers, and a
build of the recurrence's backward whose tile did not fit gave wrong gradients
where the compiler had spilled (a register cap too low for the kernel); with
room the same source was right."""
import os
import re
import subprocess

import pytest

from selective_state_space_56_amd import build as B


@pytest.mark.parametrize("src", ["gated.hip", "norm.hip", "conv_bwd.hip"])
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
