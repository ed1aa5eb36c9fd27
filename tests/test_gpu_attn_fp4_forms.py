"""GPU tests of qmm_attn_shared_fp4's two forms: which one a call takes, and what both have to hold alike."""
import math

import pytest
import torch

import fp4_plain
from bit_quantized_skinny_gb300 import build_lib
from test_gpu_attn_fp4 import BF16, F16, Case

pytestmark = pytest.mark.gpu
ROOM = 26 << 20                     # bytes in 16 bits; with room for at most 24 MiB, or with many rows a key, keys are expanded


@pytest.fixture(scope="module")
def qmm():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    build_lib.build()
    from bit_quantized_skinny_gb300 import qmm as q
    q.load()
    return q


def roomy(c):
    """The same call with page lists that have room for more keys than are expanded where few rows see them."""
    B, per = c.pages.shape
    room = -(-ROOM // (4 * c.Hk * c.Q.shape[2] * c.page * B))
    c.pages = torch.cat([c.pages, torch.zeros(B, max(0, room - per), dtype=torch.int32, device="cuda")], 1)
    return c


def expands(qmm, c):
    """Whether the call has its keys and values in 16 bits in the workspace, besides the sums that either form has there."""
    T, Hq, D = c.Q.shape
    sums = 2 * T * Hq * (4 * D + 16) + 152 * 256 * (4 * D + 16) + 5 * 256
    values = (c.prefix_pages.numel() + c.pages.numel()) * c.page * c.Hk * D * 4
    need = qmm.attn_fp4_workspace_bytes(c.args(qmm))
    assert 0 < need <= sums or need >= sums - 5 * 256 + values
    return need > sums


def set_keys(c, values):
    """Own keys of stream 0 (values[n, Hk, D]); every other slot's key is 0."""
    n = values.shape[0]
    j = torch.arange(n, device="cuda")
    y = torch.zeros(c.n_pages * c.page, *values.shape[1:], dtype=torch.float64, device="cuda")
    y[c.pages[0].long()[j // c.page] * c.page + j % c.page] = values
    c.K = fp4_plain.pack(*fp4_plain.quantise(y.float().double(), c.scales[0]), c.page)


@pytest.mark.parametrize("m,Hq,D,dtype", [(1, 40, 128, BF16), (1, 64, 64, F16), (4, 40, 128, BF16), (9, 48, 128, F16)])
def test_lse_where_few_keys_have_the_weight(qmm, m, Hq, D, dtype):
    """One key of each 128 has more weight than the one before it by some 2^0.4, so that a few of them have most of the sum and a
    weight's rounding to 16 bits (2^-12) would show.  A row's score is the product of two of its values with the key's, exact in
    fp32; lse is below 16, its score's factor is off by three roundings and the exponential's argument by one (2^-22 of 23 at most),
    a weight by 2^-22, and a sum of a few hundred parts by 2^-20 at the very most: 2^-16.5 altogether."""
    Hk, n, page = 8, 40000, 64
    c = Case([m], [n], 0, Hq, Hk, D, page, dtype)
    g = torch.Generator(device="cuda").manual_seed(5)
    c.Q = torch.zeros(m, Hq, D, dtype=dtype, device="cuda")
    c.Q[..., 0] = c.Q[..., 16] = (0.9 + 0.2 * torch.rand(m, Hq, generator=g, device="cuda")).to(dtype)
    tile = torch.arange(n, device="cuda") // 128
    want = torch.where(torch.arange(n, device="cuda") % 128 == 37, 15.0 - 0.4 * (tile.max() - tile), -120.0)   # log2 of the weight
    y = torch.zeros(n, Hk, D, dtype=torch.float64, device="cuda")
    y[..., 0] = (want * math.log(2.0))[:, None]
    c.scale = 1.0
    coarse = fp4_plain.unpack(fp4_plain.pack(*fp4_plain.quantise(y.float().double(), c.scales[0]), page), Hk, D, page, c.scales[0])
    y[..., 16] = y[..., 0] - coarse[..., 0]
    set_keys(c, y)
    assert not expands(qmm, c)
    for _ in range(2):
        c.run(qmm)
        _, lse, _ = c.plain()
        assert bool(((c.lse.double() - lse).abs() <= 2.0 ** -16.5).all()), (c.lse.double() - lse).abs().max().item()
    assert qmm.device_status() == 0


@pytest.mark.parametrize("rows,lens,prefix,Hq,Hk,D,page,dtype", [
    ([1] * 5, [700, 3, 129, 1, 400], 0, 40, 8, 128, 16, BF16),
    ([8] * 4, [90, 8, 500, 129], 2050, 10, 2, 128, 64, BF16),
    ([0, 3, 6, 1, 0, 5], [9, 3, 777, 1, 0, 128], 301, 24, 3, 64, 32, F16),
])
def test_both_forms_of_a_call(qmm, rows, lens, prefix, Hq, Hk, D, page, dtype):
    """The same call with narrow and with wide page lists.  Both forms take scores, sums and lse in fp32: lse within 2^-15 (scores of
    at most 10, summed over D values in fp32 either way), O within a rounding to its type and the weights' roundings to 16 bits."""
    c = Case(rows, lens, prefix, Hq, Hk, D, page, dtype)
    assert expands(qmm, c)
    c.run(qmm).check()
    O, lse = c.O.clone(), c.lse.clone()
    assert not expands(qmm, roomy(c))
    c.run(qmm).check()
    fine = lse.isfinite()
    assert torch.equal(fine, c.lse.isfinite()) and bool(((c.lse - lse).abs()[fine] <= 2.0 ** -15).all())
    _, _, S = c.plain()
    u = torch.finfo(dtype).eps / 2
    assert bool(((c.O.double() - O.double()).abs() <= 2 * u * O.double().abs() + 2.0 ** -10 * S + 2.0 ** -24).all())
    assert qmm.device_status() == 0


@pytest.mark.parametrize("wide", [False, True])
def test_pages_that_no_row_needs_may_hold_anything(qmm, wide):
    """A stream without rows may have any page numbers, and so may the prefix of a call whose rows are all padding."""
    c = Case([2, 0, 3], [90, 200, 30], 130, 10, 2, 128, 16)
    c.pages[1] = torch.tensor([-3, 1 << 30], dtype=torch.int32, device="cuda").repeat(c.pages.shape[1])[:c.pages.shape[1]]
    c = roomy(c) if wide else c
    assert expands(qmm, c) is not wide
    c.run(qmm)
    assert qmm.device_status() == 0
    c.pages[1] = 0
    c.check()
    c = Case([0, 0], [40, 0], 70, 10, 2, 128, 16, pad_rows=4)
    c.prefix_pages[:], c.pages[:] = -7, 1 << 30
    c = roomy(c) if wide else c
    assert expands(qmm, c) is not wide
    c.run(qmm)
    assert qmm.device_status() == 0 and bool((c.O == 0).all()) and bool(c.lse.isneginf().all())


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("product,keys", [(2.0 ** 93, 0.0), (2.0 ** -126, 1.0)])
def test_scales_at_the_ends_of_their_range(qmm, wide, dtype, product, keys):
    """The smallest factor between a key's score and the softmax's, and the largest one over keys of zeros: all weights are equal."""
    c = Case([3, 2], [100, 260], 130, 10, 2, 128, 32, dtype, scales=(2.0 ** -5, 0.055))   # (the product is exactly the range's end)
    c = roomy(c) if wide else c
    c.scale = product / c.scales[0]
    c.Q[1] = 0
    if keys == 0.0:
        c.K[:] = 0
    assert expands(qmm, c) is not wide
    c.run(qmm).check()
    assert qmm.device_status() == 0
