"""CPU test of the kernels that start while the launch ahead of them still runs (programmatic dependent
launch): what that launch may be writing is read with loads that stay behind the wait for it.  A load
marked read-only for the kernel's lifetime (__ldg, ld.global.nc) may be taken for invariant and moved
ahead, and the memory is not read-only for that long; of a load with a cache hint (__ldcg) no order
is promised."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantized_skinny_gb300", "csrc")


@pytest.mark.parametrize("source,forbidden", [
    ("q4k_fma.cu", r"__ldg\(|ldg_nc_v4\(xr|\.nc\b"),                  # X
    ("qmm_lora.cu", r"__ldcg\(|ldg_nc_v4\(e\.|__ldg\(.*e\.[XYt]"),   # X, Y0 and t
    ("qmm_norm_rope.cu", r"__ldg\(|\.nc\b|ldg_nc"),                # Q, K, V, positions, slots, weights and table
])
def test_loads_stay_behind_the_wait(source, forbidden):
    with open(os.path.join(CSRC, source), encoding="utf-8") as fh:
        code = re.sub(r"//[^\n]*", "", fh.read())
    assert "griddepcontrol.wait" in code
    found = [line.strip() for line in code.split("\n") if re.search(forbidden, line)]
    assert not found, found
