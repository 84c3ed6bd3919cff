"""The build's own check: kernels of the row operators do not spill vector
registers."""
import importlib.util
import os
import shutil

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SPILLS = """
#include <hip/hip_runtime.h>
__global__ void __launch_bounds__(64) __attribute__((amdgpu_num_vgpr(24))) k_many(const float* x, float* y) {
  float v[64];
  for (int i = 0; i < 64; ++i) v[i] = x[i * 64 + threadIdx.x];
  __syncthreads();
  for (int i = 0; i < 64; ++i) y[i * 64 + threadIdx.x] = v[i] * v[63 - i];
}
"""
FITS = """
#include <hip/hip_runtime.h>
__global__ void k_one(const float* x, float* y) { y[threadIdx.x] = x[threadIdx.x]; }
"""


def load():
    spec = importlib.util.spec_from_file_location("_build_under_test",
                                                  os.path.join(ROOT, "soft_clustering_amd", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_spills_are_read_from_the_remarks():
    b = load()
    line = "a.hip:3:1: remark: {} [-Rpass-analysis=kernel-resource-usage]\n"
    text = "".join(line.format(v) for v in (
        "Function Name: k_a", "    VGPRs: 128", "    SGPRs Spill: 4", "    VGPRs Spill: 0",
        "Function Name: k_b", "    SGPRs Spill: 0", "    VGPRs Spill: 17"))
    assert b.spilled(text) == [("k_b", 17)]
    assert b.spilled("") == []


def test_kernels_of_the_row_operators_are_checked():
    b = load()
    assert {"gmm_mx.hip", "gmm_draw.hip"} <= set(b.NO_SPILL) <= set(b.SOURCES)


@pytest.mark.skipif(not (shutil.which("hipcc") or os.path.exists("/opt/rocm/bin/hipcc")), reason="no hipcc")
def test_a_spilling_kernel_ends_the_build(tmp_path):
    b = load()
    b.CSRC = b.BUILD = str(tmp_path)
    name = b.NO_SPILL[0]
    (tmp_path / name).write_text(FITS)
    assert os.path.exists(b._compile(name, False, False))
    (tmp_path / name).write_text(SPILLS)
    with pytest.raises(RuntimeError, match="k_many"):
        b._compile(name, False, False)
    assert not os.path.exists(tmp_path / name.replace(".hip", ".o"))  # an incremental build must not take it
