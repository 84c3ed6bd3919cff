"""No kernel of the row operators uses the result of a matrix instruction before
it is there (a race that some runs win)."""
import os
import shutil
import subprocess

import pytest

from tests import matrix_waits as W
from tests.test_build_cpu import load

PRODUCT = "v_mfma_scale_f32_16x16x128_f8f6f4 v[32:35], v[24:31], v[66:73], v[32:35], v58, v57 op_sel_hi:[0,0,0]"


def code(*lines):
    return ["_Z1kv:", *lines, "s_endpgm"]


def find(*lines):
    return W.early_uses(W.functions("\n".join(code(*lines)))["_Z1kv"])


def test_uses_are_found():
    use = "ds_write_b128 v56, v[32:35]"
    assert find(PRODUCT, use)[0][2:] == (0, 11)
    assert find(PRODUCT, "s_nop 9", use)[0][2:] == (10, 11)
    assert not find(PRODUCT, "s_nop 10", use)
    assert not find(PRODUCT, "ds_write_b128 v56, v[36:39]")
    assert find(PRODUCT, "v_mov_b32 v1, v35") and find(PRODUCT, "v_mov_b32 v32, v1")
    # over a branch, on either side, and round a loop
    assert find(PRODUCT, "s_cbranch_scc1 .L1", "s_nop 15", "s_endpgm", ".L1:", use)[0][2] == 1
    assert find(".L0:", "v_add_f32 v1, v1, v33", "s_nop 3", PRODUCT, "s_cbranch_scc1 .L0")[0][2] == 1
    assert not find(PRODUCT, "s_branch .L1", use, ".L1:", "s_nop 10")
    # a product on top is chained, one that takes the result as a factor is not
    assert not find(PRODUCT, PRODUCT, "s_nop 15", use)
    assert find(PRODUCT, PRODUCT.replace("v[24:31]", "v[30:37]").replace("v[32:35]", "v[80:83]"))
    with pytest.raises(ValueError, match="passes"):
        find("v_mfma_f32_4x4x1_16b_f32 v[0:3], v4, v5, v[0:3]")
    assert W.needed(PRODUCT + " cbsz:4 blgp:4") == 7


@pytest.mark.skipif(not (shutil.which("hipcc") or os.path.exists("/opt/rocm/bin/hipcc")), reason="no hipcc")
def test_kernels_wait_for_their_products():
    b = load()
    sources = [s for s in b.NO_SPILL if "__builtin_amdgcn_mfma" in open(os.path.join(b.CSRC, s)).read()]
    assert "gmm_mx.hip" in sources
    running = [subprocess.Popen([b.hipcc(), *[f for f in b.FLAGS if f != "-fPIC"], "--cuda-device-only", "-S",
                                 os.path.join(b.CSRC, s), "-o", "-"], stdout=subprocess.PIPE,
                                stderr=subprocess.DEVNULL, text=True) for s in sources]
    for source, child in zip(sources, running):
        asm = child.communicate()[0]
        assert child.returncode == 0, source
        kernels = W.functions(asm)
        assert sum(line.startswith("v_mfma") for c in kernels.values() for line in c) > 100, source
        bad = {name: W.early_uses(c) for name, c in kernels.items()}
        assert not any(bad.values()), {name: found[:2] for name, found in bad.items() if found}
