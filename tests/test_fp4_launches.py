"""CPU test of the 4-bit cache's and the sampling's kernels, which start while the launch ahead of them still runs: what that
launch may be writing is read with loads that stay behind the wait for it (see test_early_launches.py)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantized_skinny_gb300", "csrc")


@pytest.mark.parametrize("source", ["qmm_kv_fp4.cu", "qmm_attn_fp4.cu", "qmm_sample.cu", "qmm_norm_rope.cu", "q4k_attn_parts.cuh"])
def test_loads_stay_behind_the_wait(source):
    with open(os.path.join(CSRC, source), encoding="utf-8") as fh:
        code = re.sub(r"//[^\n]*", "", fh.read())
    assert "griddepcontrol.wait" in code
    found = [line.strip() for line in code.split("\n") if re.search(r"__ldg\(|__ldcg\(|\.nc\b|ldg_nc", line)]
    assert not found, found
