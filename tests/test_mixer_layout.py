"""What the mixer kernels read 16 bytes at a time in LDS lies on 16 bytes, the
second element of an array too."""
import subprocess

import pytest

from selective_state_space_56_amd import build as B

CHECK = """
#include "linattn.h"
using mscan::Decays;
template <int C> struct Check {
  static_assert(alignof(Decays<C>) % 16 == 0, "alignment");
  static_assert(sizeof(Decays<C>[2]) == 2 * sizeof(Decays<C>) && sizeof(Decays<C>) % 16 == 0, "second element");
  static_assert(offsetof(Decays<C>, down) % 16 == 0 && offsetof(Decays<C>, end) % 16 == 0, "members");
};
template struct Check<STEPS>;
"""


@pytest.mark.parametrize("steps", [32, 64])
def test_decays_lie_on_16_bytes(steps, tmp_path):
    src = tmp_path / "check.hip"
    src.write_text(CHECK.replace("STEPS", str(steps)))
    r = subprocess.run([B.hipcc()] + B.COMMON + B.DEVICE + ["-fsyntax-only", str(src)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
