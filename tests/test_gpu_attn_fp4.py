"""GPU tests of qmm_attn_shared_fp4 against its formula in 64 bits, over the values that the caches hold.

Bound per value of O, with u the unit roundoff of its type and S the sum of softmax weights times |v|: one rounding
of O (u |O|), one rounding of each weight to fp16 for the tensor cores (2^-11 S, and for weights below its normal range
2^-24 of the largest weight's unit, which lies at 2^7: 2^-31 for each key on the largest |v|), and the fp32 errors as in the
16-bit form's test: 2^-11 S.  Keys, values and queries enter exactly (a bf16 query beside a value 2^24 times
as large does not; there are none here).  lse: the score's error, 2^-12 absolutely."""
import math

import pytest
import torch

import fp4_plain
import layer_plain as plain
from bit_quantized_skinny_gb300 import build_lib

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16
NAN_BYTE = 0x7F


@pytest.fixture(scope="module")
def qmm():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    build_lib.build()
    from bit_quantized_skinny_gb300 import qmm as q
    q.load()
    return q


class Case:
    """Inputs of one call: streams of rows[b] rows and lens[b] own keys behind `prefix` keys."""

    def __init__(self, rows, lens, prefix, Hq, Hk, D, page, dtype=BF16, pad_rows=0, seed=0, spare=4, scales=(0.04, 0.055)):
        g = torch.Generator(device="cuda").manual_seed(seed + sum(lens) + prefix)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.rows, self.lens, self.prefix, self.page, self.dtype, self.Hk, self.scales = rows, lens, prefix, page, dtype, Hk, scales
        self.starts = [0]
        for m in rows:
            self.starts.append(self.starts[-1] + m)
        self.T = self.starts[-1] + pad_rows
        own = [-(-n // page) for n in lens]
        n_pre = -(-prefix // page)
        self.n_pages = n_pre + sum(own) + spare
        order = torch.randperm(self.n_pages, generator=g, device="cuda").int()
        self.prefix_pages = order[:n_pre].contiguous()
        self.pages = torch.zeros(len(rows), max(own, default=0) + 1, dtype=torch.int32, device="cuda")
        at = n_pre
        for b, k in enumerate(own):
            self.pages[b, :k] = order[at:at + k]
            at += k
        self.Q = (1.5 * rnd(self.T, Hq, D)).to(dtype)
        n = self.n_pages * page
        # slots that no row sees hold what a cache may hold: large values, and NaN in every other one
        codes = torch.full((2, n, Hk, D), 15, dtype=torch.long, device="cuda")
        scale = torch.full((2, n, Hk, D // 16), 126, dtype=torch.long, device="cuda")
        scale[:, 1::2] = NAN_BYTE
        for table, m in [(self.prefix_pages, prefix)] + [(self.pages[b], m) for b, m in enumerate(lens)]:
            j = torch.arange(m, device="cuda")
            at = table.long()[j // page] * page + j % page
            for k in range(2):
                codes[k, at], scale[k, at] = fp4_plain.quantise(rnd(m, Hk, D).double(), scales[k])
        self.K, self.V = (fp4_plain.pack(codes[k], scale[k], page) for k in range(2))
        self.scale = D ** -0.5
        self.O = torch.full((self.T, Hq, D), 3.0, dtype=dtype, device="cuda")
        self.lse = torch.full((self.T, Hq), 3.0, device="cuda")
        self.lens_dev = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.starts_dev = torch.tensor(self.starts, dtype=torch.int32, device="cuda")

    def poke(self, cache, b, j, h, block, byte):
        """The scale byte of one block of own key j of stream b."""
        D, page = self.Q.shape[2], self.page
        slot_page = int(self.pages[b, j // page])
        at = (slot_page * self.Hk + h) * page * D * 9 // 16 + page * D // 2 + j % page * (D // 16) + block
        cache[at] = byte

    def args(self, qmm, lse=True):
        return qmm.make_attn_fp4(self.Q, self.K, self.V, self.Hk, self.page, self.prefix_pages, self.prefix, self.pages,
                                 self.lens_dev, self.starts_dev, self.O, scale=self.scale, k_scale=self.scales[0],
                                 v_scale=self.scales[1], lse=self.lse if lse else None)

    def run(self, qmm, stream=None):
        a = self.args(qmm)
        ws = torch.full((qmm.attn_fp4_workspace_bytes(a),), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        qmm.attn_shared_fp4(a, ws, stream=stream)
        torch.cuda.synchronize()
        return self

    def plain(self):
        D = self.Q.shape[2]
        K, V = (fp4_plain.unpack(c, self.Hk, D, self.page, s) for c, s in ((self.K, self.scales[0]), (self.V, self.scales[1])))
        return plain.attention(self.Q, K, V, self.page, self.prefix_pages, self.prefix, self.pages, self.lens, self.starts, self.scale)

    def tolerance(self, O, S):
        keys = self.prefix + max(self.lens, default=0)
        return plain.UNIT[self.dtype] * O.abs() + 2.0 ** -10 * S + keys * 2.0 ** -31 * 6.0 + 2.0 ** -24

    def check(self, rows=None):
        O, lse, S = self.plain()
        pick = slice(None) if rows is None else rows
        err = (self.O.double() - O).abs()
        bad = ~(err <= self.tolerance(O, S))[pick]
        assert not bool(bad.any()), f"max error {err[pick].max().item()}, {int(bad.sum())} values over the bound"
        a, b = self.lse.double()[pick], lse[pick]
        assert torch.equal(a.isinf(), b.isinf())
        fine = b.isfinite()
        assert bool(((a - b).abs()[fine] <= 2.0 ** -12).all())


@pytest.mark.parametrize("rows,lens,prefix,Hq,Hk,D,page,dtype", [
    ([1], [1], 0, 1, 1, 128, 16, BF16),
    ([1], [1], 0, 2, 1, 64, 16, F16),
    ([1], [700], 0, 40, 8, 128, 16, BF16),
    ([1], [129], 127, 5, 1, 128, 16, BF16),
    ([1] * 16, [37 + 61 * k for k in range(16)], 1000, 10, 2, 128, 64, BF16),
    ([8] * 4, [90, 8, 500, 129], 2050, 10, 2, 128, 64, BF16),
    ([0, 3, 6, 1, 0, 5], [9, 3, 777, 1, 0, 128], 301, 24, 3, 64, 32, F16),
    ([16] * 20, [16 + 13 * k for k in range(20)], 600, 10, 2, 128, 128, BF16),
    ([40, 70], [41, 300], 257, 8, 1, 64, 256, BF16),
    ([300], [300], 0, 4, 2, 128, 16, F16),
    ([200, 1], [333, 40], 128, 64, 1, 128, 32, BF16),
    ([2, 3], [5, 4096], 0, 7, 7, 64, 4096, BF16),
    ([1] * 3, [128, 256, 384], 128, 3, 3, 128, 128, BF16),
    ([5] * 60, [5 + k for k in range(60)], 17, 2, 2, 64, 16, BF16),
    ([26], [64], 64, 5, 1, 128, 64, BF16),
    ([52], [200], 400, 5, 1, 128, 64, BF16),
])
def test_against_the_formula(qmm, rows, lens, prefix, Hq, Hk, D, page, dtype):
    Case(rows, lens, prefix, Hq, Hk, D, page, dtype).run(qmm).check()
    assert qmm.device_status() == 0


def test_rows_that_see_nothing_and_padding(qmm):
    """Rows before a stream's first key, streams without keys, rows of no stream: O = 0, lse = -inf."""
    c = Case([4, 2, 0, 3], [2, 0, 0, 3], 0, 6, 2, 128, 16, pad_rows=3).run(qmm)
    c.check()
    assert bool((c.O[:2] == 0).all()) and bool((c.O[4:6] == 0).all()) and bool((c.O[9:] == 0).all())
    assert bool(c.lse[9:].isneginf().all())
    c = Case([2, 2], [0, 1], 40, 6, 2, 128, 16, pad_rows=40).run(qmm)     # the prefix alone
    c.check()
    assert bool((c.O[4:] == 0).all()) and bool(c.lse[4:].isneginf().all())
    c = Case([], [], 40, 4, 2, 64, 16, pad_rows=5).run(qmm)
    assert bool((c.O == 0).all()) and bool(c.lse.isneginf().all())
    c = Case([], [], 16, 4, 2, 64, 16)
    qmm.attn_shared_fp4(c.args(qmm), torch.empty(max(16, qmm.attn_fp4_workspace_bytes(c.args(qmm))), dtype=torch.uint8,
                                                 device="cuda"))
    assert qmm.device_status() == 0


@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, F16)])
def test_later_rows_values_do_not_reach_earlier_rows(qmm, D, dtype):
    """A NaN block in the key and value of a drafted row stays with the rows that see it."""
    c = Case([6, 6], [140, 9], 70, 10, 2, D, 16, dtype=dtype)
    c.poke(c.K, 0, 138, 0, 1, NAN_BYTE)
    c.poke(c.V, 1, 7, 0, 1, NAN_BYTE)
    c.poke(c.V, 1, 8, 1, D // 16 - 1, NAN_BYTE)
    c.run(qmm)
    c.check(rows=torch.tensor([0, 1, 2, 3, 6, 7, 8, 9], device="cuda"))
    assert bool(c.O[4:6, :5].isnan().all())                      # a NaN key: every value of the head's rows
    assert bool(c.O[10:12, :5, 16:32].isnan().all()) and bool(c.O[11, 5:, D - 16:].isnan().all())
    rest = torch.ones(2, 10, D, dtype=torch.bool, device="cuda")
    rest[:, :5, 16:32] = False
    rest[1, 5:, D - 16:] = False
    O, _, S = c.plain()
    ok = (c.O[10:12].double() - O[10:12]).abs() <= c.tolerance(O[10:12], S[10:12])
    assert bool(ok[rest].all())
    assert bool(c.O[4:6, 5:].isfinite().all())


@pytest.mark.parametrize("D,dtype", [(128, F16), (128, BF16), (64, F16)])
def test_an_early_draft_value_in_a_block_of_two_row_tiles(qmm, D, dtype):
    """A NaN in the value of the fifth of 40 drafted rows, whose key is far below the others in score (its weight is 0
    in 16 bits): the rows of both row tiles that see it get it, and every call gives the same bits."""
    c = Case([40], [150], 70, 5, 1, D, 16, dtype=dtype)          # 25 rows a tile
    c.Q = c.Q.abs()
    slot = int(c.pages[0, 114 // 16]) * 16 + 114 % 16
    run = slot // 16 * 16 * D * 9 // 16
    c.K[run + slot % 16 * (D // 2):run + (slot % 16 + 1) * (D // 2)] = 0xFF      # -6 of the block's scale
    for block in range(D // 16):
        c.poke(c.K, 0, 114, 0, block, 0x60)                                      # 32: values of -7.7
    c.poke(c.V, 0, 114, 0, 0, NAN_BYTE)
    c.run(qmm)
    assert bool(c.O[4:, :, :16].isnan().all())
    O, lse, S = c.plain()
    ok = (c.O.double() - O).abs() <= c.tolerance(O, S)
    assert bool(ok[:, :, 16:].all()) and bool(ok[:4].all())
    first = c.O.clone()
    args, ws = c.args(qmm), torch.empty(qmm.attn_fp4_workspace_bytes(c.args(qmm)), dtype=torch.uint8, device="cuda")
    for _ in range(200):
        c.O.fill_(3.0)
        qmm.attn_shared_fp4(args, ws)
        assert torch.equal(c.O.view(torch.int16), first.view(torch.int16))
    assert qmm.device_status() == 0


def test_large_and_equal_scores(qmm):
    """Scores near the exponential's range: large queries, and all keys equal."""
    c = Case([2, 2], [300, 300], 500, 4, 2, 128, 32)
    c.Q *= 16
    c.run(qmm)
    O, lse, S = c.plain()
    # |scores| reach some hundreds: fp32 errors of up to 128 * 2^-24 * 700 on each
    assert bool(((c.O.double() - O).abs() <= 2.0 ** -8 * O.abs() + 2.0 ** -6 * S).all())
    assert bool(((c.lse.double() - lse).abs() <= 2.0 ** -7).all())
    c = Case([2], [300], 500, 4, 2, 128, 32)
    c.K[:] = 0
    c.run(qmm).check()


@pytest.mark.parametrize("factor", [2.0 ** -100, 2.0 ** 90])
def test_queries_of_any_size(qmm, factor):
    """bf16 queries far outside fp16's range, with the scale that makes ordinary scores of them; a row of zeros."""
    c = Case([3, 1], [100, 260], 130, 10, 2, 128, 32)
    c.Q[1] = 0
    c.Q[2, 3] *= 2.0 ** -20
    c.Q *= factor
    c.scale /= factor
    c.run(qmm).check()


@pytest.mark.parametrize("scales", [(1.0, 1.0), (2.0 ** -60, 2.0 ** -20), (0.3, 2.0 ** 20)])
def test_tensor_scales(qmm, scales):
    c = Case([2, 5], [70, 200], 90, 6, 2, 64, 16, dtype=BF16, scales=(0.04, 0.055))
    c.scale *= 0.04 / scales[0]
    c.scales = scales
    c.run(qmm)
    O, lse, S = c.plain()
    keys = 290
    tol = 2.0 ** -8 * O.abs() + 2.0 ** -10 * S + keys * 2.0 ** -31 * 6.0 * scales[1] / 0.055 + 2.0 ** -24 * scales[1]
    assert bool(((c.O.double() - O).abs() <= tol).all())


def test_strided_rows(qmm):
    """Q and O as column ranges of wider buffers."""
    c = Case([3, 4], [50, 20], 100, 10, 2, 128, 16)
    wide = torch.zeros(c.T, 24, 128, dtype=BF16, device="cuda")
    wide[:, 5:15] = c.Q
    out = torch.full((c.T, 24, 128), 9.0, dtype=BF16, device="cuda")
    c.Q, c.O = wide[:, 5:15], out[:, 7:17]
    c.run(qmm).check()
    assert bool((out[:, :7] == 9).all()) and bool((out[:, 17:] == 9).all())


def test_same_bits_again_and_on_another_stream(qmm):
    c = Case([8, 3, 1, 9], [800, 40, 333, 1200], 1500, 40, 8, 128, 64).run(qmm)
    first, lse = c.O.clone(), c.lse.clone()
    c.check()
    side = torch.cuda.Stream()
    c.O.fill_(3.0)
    side.wait_stream(torch.cuda.current_stream())
    c.run(qmm, stream=side)
    assert torch.equal(c.O, first) and torch.equal(c.lse, lse)


def test_lengths_change_between_graph_replays(qmm):
    c = Case([2, 2, 2], [90, 200, 30], 130, 10, 2, 128, 16)
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
    c = Case([2, 2, 2], [90, 200, 30], 130, 10, 2, 128, 16)
    rest = torch.tensor([0, 1, 4, 5], device="cuda")
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


def test_row_starts_out_of_range_are_reported(qmm):
    c = Case([2, 2, 2], [90, 200, 30], 130, 10, 2, 128, 16)
    for bad in ([0, 2, 1, 6], [0, 2, 100, 6], [0, -4, 4, 6], [0, 2, 4, 1 << 30]):
        c.starts_dev.copy_(torch.tensor(bad, dtype=torch.int32))
        c.run(qmm)
        assert qmm.device_status() == 4, bad


def test_cache_beyond_32_bit_offsets(qmm):
    """Pages behind the first 4 GiB of each cache."""
    Hk, D, page = 8, 128, 64
    bytes_of_page = page * Hk * D * 9 // 16
    c = Case([2, 3], [150, 70], 200, 16, Hk, D, page)
    n_pages = (5 << 30) // bytes_of_page
    shift = n_pages - c.n_pages
    K, V = (torch.empty(n_pages * bytes_of_page, dtype=torch.uint8, device="cuda") for _ in range(2))
    K[shift * bytes_of_page:], V[shift * bytes_of_page:] = c.K, c.V
    want = c.plain()
    c.K, c.V = K, V
    c.prefix_pages += shift
    c.pages += shift
    c.run(qmm)
    c.plain = lambda: want
    c.check()


def test_random_shapes(qmm):
    import random
    r = random.Random(11)
    for trial in range(12):
        Hk, D = r.choice([1, 2, 3]), r.choice([64, 128])
        B = r.randint(1, 24)
        rows = [r.randint(0, r.choice([1, 4, 33])) for _ in range(B)]
        lens = [r.randint(0, r.choice([20, 150, 900])) for _ in range(B)]
        c = Case(rows, lens, r.choice([0, r.randint(1, 900)]), Hk * r.randint(1, 9), Hk, D,
                 r.choice([16, 32, 64, 128, 256]), r.choice([BF16, F16]), pad_rows=r.randint(0, 3), seed=trial)
        if c.T:
            c.run(qmm).check()
    assert qmm.device_status() == 0


def test_many_calls_of_ragged_streams(qmm):
    """Short and long segments of one and two row tiles in turn, call after call behind each other: every wait
    ends (bit 0 of the status word) and every call gives the same bits."""
    import random
    r = random.Random(3)
    for D, dtype, G in ((64, F16, 8), (128, BF16, 5), (128, BF16, 64)):
        cases = [Case([r.randint(0, 2 * (128 // G) + 3) for _ in range(29)], [r.choice([0, 1, 40, 64, 65, 300, 900]) for _ in range(29)],
                      p, 2 * G, 2, D, 32, dtype, seed=k) for k, p in enumerate((0, 60, 1700))]
        first = []
        for c in cases:
            c.run(qmm).check()
            first.append(c.O.clone())
        args = [c.args(qmm) for c in cases]
        ws = torch.empty(max(qmm.attn_fp4_workspace_bytes(a) for a in args), dtype=torch.uint8, device="cuda")
        for _ in range(60):
            for a in args:
                qmm.attn_shared_fp4(a, ws)
        torch.cuda.synchronize()
        assert qmm.device_status() == 0
        for c, f in zip(cases, first):
            assert torch.equal(c.O, f)


def test_concurrent_streams(qmm):
    """Calls on two streams with a workspace each do not disturb each other."""
    a = Case([2] * 8, [300 + k for k in range(8)], 900, 10, 2, 128, 32)
    b = Case([5] * 6, [70 * k + 9 for k in range(6)], 400, 24, 3, 64, 16, F16)
    a.run(qmm)
    b.run(qmm)
    want = a.O.clone(), b.O.clone()
    args = [a.args(qmm), b.args(qmm)]
    ws = [torch.empty(qmm.attn_fp4_workspace_bytes(x), dtype=torch.uint8, device="cuda") for x in args]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for x, w, st in zip(args, ws, streams):
            qmm.attn_shared_fp4(x, w, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(a.O, want[0]) and torch.equal(b.O, want[1]) and qmm.device_status() == 0


@pytest.mark.parametrize("rows,lens,prefix,Hq,Hk,D,page,dtype", [
    # prompts: many blocks of rows, whose last keys differ, behind a prefix and without one
    ([1500], [2100], 513, 10, 2, 128, 64, BF16),
    ([700, 900], [700, 1300], 0, 3, 3, 64, 128, F16),
    ([333], [5000], 0, 64, 1, 128, 256, BF16),
    # many pieces to join for a row, few rows and more
    ([5] * 8, [40 + 9 * k for k in range(8)], 9000, 40, 8, 128, 64, BF16),
    ([4] * 20, [1500 + 70 * k for k in range(20)], 6000, 20, 2, 64, 16, F16),
    ([1, 1], [40000, 33001], 0, 10, 2, 128, 64, BF16),
])
def test_long_streams_against_the_formula(qmm, rows, lens, prefix, Hq, Hk, D, page, dtype):
    c = Case(rows, lens, prefix, Hq, Hk, D, page, dtype).run(qmm)
    c.check()
    first = c.O.clone()
    assert torch.equal(c.run(qmm).O, first)
    assert qmm.device_status() == 0
