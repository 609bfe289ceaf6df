"""The build refuses a block operator's source whose kernels spill registers,
whichever compiler reports it (compiled here, never run)."""
import os

import pytest

from selective_state_space_56_amd import build as B

SPILLS = """
#include <hip/hip_runtime.h>
__global__ __attribute__((amdgpu_num_vgpr(24))) __launch_bounds__(64) void tight_kernel(const float* in, float* out) {
  float v[64];
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = in[i * 64 + threadIdx.x];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 64; ++i) out[i * 64 + threadIdx.x] = v[(i * 7 + 3) % 64] * v[i];
}
"""
FITS = """
#include <hip/hip_runtime.h>
__global__ void roomy_kernel(float* out) { out[threadIdx.x] = 1.0f; }
"""


@pytest.fixture
def sources(tmp_path, monkeypatch):
    monkeypatch.setattr(B, "CSRC", str(tmp_path))
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "out"))

    def put(name, text):
        (tmp_path / name).write_text(text)
        return os.path.join(str(tmp_path / "out"), os.path.splitext(name)[0] + ".o")
    return put


def test_a_spilling_kernel_is_refused(sources):
    obj = sources("gated.hip", SPILLS)
    with pytest.raises(RuntimeError, match="spill registers.*tight_kernel"):
        B._compile("gated.hip")
    assert not os.path.exists(obj)  # an incremental build must not pick it up


def test_a_kernel_with_room_is_built(sources):
    obj = sources("norm.hip", FITS)
    assert B._compile("norm.hip") == obj and os.path.exists(obj)


def test_the_report_is_read_by_kernel():
    text = """x.hip:3:0: remark: Function Name: a_kernel [-Rpass-analysis=kernel-resource-usage]
x.hip:3:0: remark:     ScratchSize [bytes/lane]: 0 [-Rpass-analysis=kernel-resource-usage]
x.hip:3:0: remark:     VGPRs Spill: 0 [-Rpass-analysis=kernel-resource-usage]
x.hip:9:0: remark: Function Name: b_kernel [-Rpass-analysis=kernel-resource-usage]
x.hip:9:0: remark:     ScratchSize [bytes/lane]: 12 [-Rpass-analysis=kernel-resource-usage]
x.hip:9:0: remark:     VGPRs Spill: 3 [-Rpass-analysis=kernel-resource-usage]"""
    assert B.spilling(text) == ["b_kernel"]
    with pytest.raises(RuntimeError, match="no register usage"):
        B.spilling("remark: nothing known")
