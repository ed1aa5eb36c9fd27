"""GPU tests of qmm_attn_shared_fp4's form for few rows of many keys: every test of test_gpu_attn_fp4.py again, its page lists
with room for more keys than the call writes to its workspace in 16 bits."""
import pytest
import torch

import test_gpu_attn_fp4 as small
from bit_quantized_skinny_gb300 import build_lib

pytestmark = pytest.mark.gpu
BF16, F16 = small.BF16, small.F16
ROOM = 26 << 20                     # bytes in 16 bits that the lists have room for; the call's border is 24 MiB


@pytest.fixture(scope="module")
def qmm():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    build_lib.build()
    from bit_quantized_skinny_gb300 import qmm as q
    q.load()
    return q


class Roomy(small.Case):
    def __init__(self, *args, **more):
        super().__init__(*args, **more)
        B, per = self.pages.shape
        if B:
            room = -(-ROOM // (4 * self.Hk * self.Q.shape[2] * self.page * B))
            self.pages = torch.cat([self.pages, torch.zeros(B, max(0, room - per), dtype=torch.int32, device="cuda")], 1)


@pytest.fixture(autouse=True)
def roomy(monkeypatch):
    monkeypatch.setattr(small, "Case", Roomy)


@pytest.mark.parametrize("rows,lens,prefix,Hq,Hk,D,page,dtype", [
    ([1], [1], 0, 1, 1, 128, 16, BF16),
    ([1], [1], 0, 2, 1, 64, 16, F16),
    ([1], [700], 0, 40, 8, 128, 16, BF16),
    ([1], [129], 127, 5, 1, 128, 16, BF16),
    ([1] * 16, [37 + 61 * k for k in range(16)], 1000, 10, 2, 128, 64, BF16),
    ([8] * 4, [90, 8, 500, 129], 2050, 10, 2, 128, 64, BF16),
    ([0, 3, 6, 1, 0, 5], [9, 3, 777, 1, 0, 128], 301, 24, 3, 64, 32, F16),
    ([16] * 20, [16 + 13 * k for k in range(20)], 600, 10, 2, 128, 128, BF16),
    ([30, 50], [31, 300], 257, 2, 1, 64, 256, BF16),
    ([70], [300], 0, 4, 2, 128, 16, F16),
    ([2, 3], [5, 4096], 0, 7, 7, 64, 4096, BF16),
    ([1] * 3, [128, 256, 384], 128, 3, 3, 128, 128, BF16),
    ([5] * 60, [5 + k for k in range(60)], 17, 2, 2, 64, 16, BF16),
    ([26], [64], 64, 5, 1, 128, 64, BF16),
    ([31], [200], 400, 5, 1, 128, 64, BF16),
])
def test_against_the_formula(qmm, rows, lens, prefix, Hq, Hk, D, page, dtype):
    c = Roomy(rows, lens, prefix, Hq, Hk, D, page, dtype)
    n = c.T * Hq
    assert qmm.attn_fp4_workspace_bytes(c.args(qmm)) < 2 * n * D * 4 + 152 * 256 * D * 4 + 2 * n * 16 + 152 * 256 * 16 + (1 << 20)
    small.test_against_the_formula(qmm, rows, lens, prefix, Hq, Hk, D, page, dtype)


def test_rows_that_see_nothing_and_padding(qmm):
    small.test_rows_that_see_nothing_and_padding(qmm)


@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, F16)])
def test_later_rows_values_do_not_reach_earlier_rows(qmm, D, dtype):
    small.test_later_rows_values_do_not_reach_earlier_rows(qmm, D, dtype)


def test_large_and_equal_scores(qmm):
    small.test_large_and_equal_scores(qmm)


@pytest.mark.parametrize("factor", [2.0 ** -100, 2.0 ** 90])
def test_queries_of_any_size(qmm, factor):
    small.test_queries_of_any_size(qmm, factor)


@pytest.mark.parametrize("scales", [(1.0, 1.0), (2.0 ** -60, 2.0 ** -20), (0.3, 2.0 ** 20)])
def test_tensor_scales(qmm, scales):
    small.test_tensor_scales(qmm, scales)


def test_strided_rows(qmm):
    small.test_strided_rows(qmm)


def test_same_bits_again_and_on_another_stream(qmm):
    small.test_same_bits_again_and_on_another_stream(qmm)


def test_lengths_change_between_graph_replays(qmm):
    small.test_lengths_change_between_graph_replays(qmm)


def test_indices_out_of_range_are_reported(qmm):
    small.test_indices_out_of_range_are_reported(qmm)


def test_row_starts_out_of_range_are_reported(qmm):
    small.test_row_starts_out_of_range_are_reported(qmm)


def test_random_shapes(qmm):
    small.test_random_shapes(qmm)


def test_many_calls_of_ragged_streams(qmm):
    small.test_many_calls_of_ragged_streams(qmm)


def test_concurrent_streams(qmm):
    small.test_concurrent_streams(qmm)


def test_a_wait_that_runs_out_is_reported(qmm):
    """With a bound far below a memory access's latency the first waits give up: the call ends, sets bit 0, and
    the next call (default bound) is right."""
    c = Roomy([8] * 4, [90, 8, 500, 129], 2050, 10, 2, 128, 64)
    qmm.set_wait_limit(2, 50)
    try:
        c.run(qmm)
    finally:
        qmm.set_wait_limit(0, 0)
    assert qmm.device_status() & 1 and qmm.device_status() == 0
    c.run(qmm).check()
    assert qmm.device_status() == 0
