"""GPU tests of qmm_attn_shared_fp4 with many rows a key, where the call writes the keys and values to its workspace in 16
bits first: the same checks as with few rows, with the same tolerances (the products' operands are the same
values, and the weights keep at least as many bits)."""
import pytest
import torch

from bit_quantized_skinny_gb300 import build_lib
from test_gpu_attn_fp4 import BF16, F16, NAN_BYTE, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qmm():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    build_lib.build()
    from bit_quantized_skinny_gb300 import qmm as q
    q.load()
    return q


def expands(qmm, c):
    """Whether the workspace has room for the keys and values of c in 16 bits (that of few rows has some 20 MB)."""
    n, D, Hk = -(-c.prefix // c.page) + c.pages.numel(), c.Q.shape[2], c.Hk
    rows = c.T * c.Q.shape[1]
    base = 2 * rows * D * 4 + 152 * 256 * D * 4 + 2 * rows * 16 + 152 * 256 * 16
    return qmm.attn_fp4_workspace_bytes(c.args(qmm)) >= base + n * c.page * Hk * D * 4


@pytest.mark.parametrize("rows,lens,prefix,Hq,Hk,D,page,dtype", [
    ([160], [160], 0, 1, 1, 128, 16, BF16),
    ([32], [33], 0, 5, 1, 64, 16, F16),
    ([16] * 20, [16 + 13 * k for k in range(20)], 1600, 10, 2, 128, 128, BF16),
    ([3] * 30, [3 + 7 * k for k in range(30)], 5001, 10, 2, 64, 32, F16),
    ([0, 90, 0, 77, 1, 300], [9, 90, 0, 400, 1, 300], 301, 24, 3, 128, 32, BF16),
    ([40, 70], [41, 300], 257, 64, 1, 64, 256, BF16),
    ([200], [300], 4097, 8, 1, 128, 4096, F16),
    ([700], [700], 0, 7, 7, 128, 64, BF16),
    ([26] * 9, [64 + k for k in range(9)], 640, 40, 8, 128, 64, BF16),
])
def test_against_the_formula(qmm, rows, lens, prefix, Hq, Hk, D, page, dtype):
    c = Case(rows, lens, prefix, Hq, Hk, D, page, dtype)
    assert expands(qmm, c)
    c.run(qmm).check()
    assert qmm.device_status() == 0


def test_few_rows_of_many_keys_do_not_expand(qmm):
    c = Case([8] * 4, [90, 8, 500, 129], 2050, 10, 2, 128, 64)
    assert expands(qmm, c)                                       # few keys
    c.pages = torch.cat([c.pages, torch.zeros(4, 200, dtype=torch.int32, device="cuda")], 1)
    assert not expands(qmm, c)


def test_rows_that_see_nothing_and_padding(qmm):
    c = Case([4, 200, 0, 30], [2, 150, 0, 3], 0, 6, 2, 128, 16, pad_rows=3)
    assert expands(qmm, c)
    c.run(qmm).check()
    seen = torch.tensor([2, 3] + list(range(54, 204)) + [231, 232, 233], device="cuda")
    none = torch.ones(c.T, dtype=torch.bool, device="cuda")
    none[seen] = False
    assert bool((c.O[none] == 0).all()) and bool(c.lse[none].isneginf().all())
    c = Case([100, 2], [0, 1], 40, 6, 2, 128, 16, pad_rows=40).run(qmm)     # the prefix alone
    c.check()
    assert expands(qmm, c) and bool((c.O[102:] == 0).all()) and bool(c.lse[102:].isneginf().all())
    assert qmm.device_status() == 0


@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, F16)])
def test_later_rows_values_do_not_reach_earlier_rows(qmm, D, dtype):
    """A NaN block in the key and value of a drafted row stays with the rows that see it."""
    c = Case([60, 60], [194, 63], 70, 10, 2, D, 16, dtype=dtype)
    assert expands(qmm, c)
    c.poke(c.K, 0, 192, 0, 1, NAN_BYTE)                          # row 58 of stream 0 and on
    c.poke(c.V, 1, 61, 0, 1, NAN_BYTE)                           # row 58 of stream 1 and on
    c.poke(c.V, 1, 62, 1, D // 16 - 1, NAN_BYTE)
    c.run(qmm)
    c.check(rows=torch.tensor(list(range(58)) + list(range(60, 118)), device="cuda"))
    assert bool(c.O[58:60, :5].isnan().all())                    # a NaN key: every value of the head's rows
    assert bool(c.O[118:, :5, 16:32].isnan().all()) and bool(c.O[119, 5:, D - 16:].isnan().all())
    rest = torch.ones(2, 10, D, dtype=torch.bool, device="cuda")
    rest[:, :5, 16:32] = False
    rest[1, 5:, D - 16:] = False
    O, _, S = c.plain()
    ok = (c.O[118:].double() - O[118:]).abs() <= c.tolerance(O[118:], S[118:])
    assert bool(ok[rest].all())
    assert bool(c.O[58:60, 5:].isfinite().all())


@pytest.mark.parametrize("factor", [2.0 ** -100, 2.0 ** 90])
def test_queries_of_any_size(qmm, factor):
    """bf16 queries far outside fp16's range, with the scale that makes ordinary scores of them; a row of zeros, and one whose
    scores are all nothing."""
    c = Case([30, 31], [100, 260], 130, 10, 2, 128, 32)
    assert expands(qmm, c)
    c.Q[1] = 0
    c.Q[2, 3] *= 2.0 ** -20
    c.Q *= factor
    c.scale /= factor
    c.run(qmm).check()
    c.scale = 2.0 ** -140                                        # every key weighs the same
    c.run(qmm).check()


@pytest.mark.parametrize("scales", [(1.0, 1.0), (2.0 ** -60, 2.0 ** -20), (0.3, 2.0 ** 20)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_tensor_scales(qmm, scales, dtype):
    c = Case([70, 50], [70, 200], 90, 6, 2, 64, 16, dtype=dtype)
    assert expands(qmm, c)
    c.scale *= 0.04 / scales[0]
    c.scales = scales
    if dtype == F16:                                             # O itself has to fit into fp16
        c.scales = (scales[0], min(scales[1], 2.0 ** 8))
    c.run(qmm)
    O, lse, S = c.plain()
    tol = 2.0 ** -8 * O.abs() + 2.0 ** -10 * S + 290 * 2.0 ** -31 * 6.0 * c.scales[1] / 0.055 + 2.0 ** -24 * max(c.scales[1], 1.0)
    assert bool(((c.O.double() - O).abs() <= tol).all())


def test_strided_rows(qmm):
    """Q and O as column ranges of wider buffers, in both types (bf16 queries are written again, fp16 ones are not)."""
    for dtype in (BF16, F16):
        c = Case([30, 40], [50, 45], 100, 10, 2, 128, 16, dtype=dtype)
        assert expands(qmm, c)
        wide = torch.zeros(c.T, 24, 128, dtype=dtype, device="cuda")
        wide[:, 5:15] = c.Q
        out = torch.full((c.T, 24, 128), 9.0, dtype=dtype, device="cuda")
        c.Q, c.O = wide[:, 5:15], out[:, 7:17]
        c.run(qmm).check()
        assert bool((out[:, :7] == 9).all()) and bool((out[:, 17:] == 9).all())


def test_same_bits_again_on_another_stream_and_at_once(qmm):
    """Calls that use one workspace one after the other, and two at once with a workspace each."""
    cases = [Case([16] * 12, [20 + 31 * k for k in range(12)], 1500, 40, 8, 128, 64, seed=s) for s in (1, 2)]
    first = []
    for c in cases:
        assert expands(qmm, c)
        c.run(qmm).check()
        first.append((c.O.clone(), c.lse.clone()))
    args = [c.args(qmm) for c in cases]
    size = max(qmm.attn_fp4_workspace_bytes(a) for a in args)
    ws = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in cases]
    side = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for a in args:
            qmm.attn_shared_fp4(a, ws[0])
    torch.cuda.synchronize()
    for c, (O, lse) in zip(cases, first):
        assert torch.equal(c.O, O) and torch.equal(c.lse, lse)
        c.O.fill_(3.0)
    torch.cuda.synchronize()
    for _ in range(20):
        for a, w, s in zip(args, ws, side):
            qmm.attn_shared_fp4(a, w, stream=s)
    torch.cuda.synchronize()
    for c, (O, lse) in zip(cases, first):
        assert torch.equal(c.O, O) and torch.equal(c.lse, lse)
    assert qmm.device_status() == 0


def test_lengths_change_between_graph_replays(qmm):
    c = Case([40, 40, 20], [90, 200, 30], 130, 10, 2, 128, 16)
    assert expands(qmm, c)
    a = c.args(qmm)
    ws = torch.empty(qmm.attn_fp4_workspace_bytes(a), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmm.attn_shared_fp4(a, ws)
    for lens in ([90, 200, 30], [2, 77, 30], [64, 0, 17]):
        c.lens = lens
        c.lens_dev.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        c.check()


def test_indices_out_of_range_are_reported(qmm):
    """A page number or a length out of range: status bit 2, the other streams' rows are right."""
    c = Case([40, 40, 20], [90, 200, 30], 130, 10, 2, 128, 16)
    assert expands(qmm, c)
    rest = torch.tensor(list(range(40)) + list(range(80, 100)), device="cuda")
    held = int(c.pages[1, 3])
    for bad in (c.n_pages, -7):
        c.pages[1, 3] = bad
        c.run(qmm)
        assert qmm.device_status() == 4 and qmm.device_status() == 0
        c.pages[1, 3] = held
        c.check(rows=rest)
    for bad in (1 << 30, -3):
        c.lens_dev[1] = bad
        c.run(qmm)
        assert qmm.device_status() == 4
        c.check(rows=rest)


def test_a_workspace_of_few_rows_is_refused(qmm):
    c = Case([40, 40, 20], [90, 200, 30], 130, 10, 2, 128, 16)
    a = c.args(qmm)
    ws = torch.empty(qmm.attn_fp4_workspace_bytes(a) - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(qmm.QmmError):
        qmm.attn_shared_fp4(a, ws)


def test_a_wait_that_runs_out_is_reported(qmm):
    c = Case([40, 40, 20], [90, 200, 30], 2050, 10, 2, 128, 16)
    assert expands(qmm, c)
    qmm.set_wait_limit(2, 50)
    try:
        c.run(qmm)
    finally:
        qmm.set_wait_limit(0, 0)
    assert qmm.device_status() & 1 and qmm.device_status() == 0
    c.run(qmm).check()
    assert qmm.device_status() == 0
