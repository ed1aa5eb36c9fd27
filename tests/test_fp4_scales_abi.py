"""CPU tests of the factor between a 4-bit cache's scores and the softmax's: scale * k_scale may not take them
out of fp32's range."""
import pytest

from test_fp4_sample_abi import fp4_attn, qmm  # noqa: F401
from test_layer_abi import ALIGN, SHAPE


@pytest.mark.parametrize("scale,k_scale", [(2.0 ** 100, 2.0 ** 60), (2.0 ** 127, 4.0), (2.0 ** 94, 1.0), (2.0 ** 34, 2.0 ** 60)])
def test_products_out_of_range_are_refused(qmm, scale, k_scale):  # noqa: F811
    lib, a = qmm.load(), fp4_attn(qmm, k_scale=k_scale, scale=scale)
    assert lib.qmm_attn_fp4_workspace_bytes(a) == 0
    assert lib.qmm_attn_shared_fp4(a, 16, 1 << 40, None) == SHAPE


@pytest.mark.parametrize("scale,k_scale", [(2.0 ** 93, 1.0), (2.0 ** 33, 2.0 ** 60), (2.0 ** -149, 2.0 ** -60), (2.0 ** -126, 1.0),
                                           (2.0 ** 120, 2.0 ** -60), (2.0 ** -120, 2.0 ** 60)])
def test_products_in_range_are_taken(qmm, scale, k_scale):  # noqa: F811
    lib, a = qmm.load(), fp4_attn(qmm, k_scale=k_scale, scale=scale, Q=24)
    assert lib.qmm_attn_fp4_workspace_bytes(a) > 0
    assert lib.qmm_attn_shared_fp4(a, 16, 1 << 40, None) == ALIGN      # the next check's answer
