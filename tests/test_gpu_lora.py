"""GPU tests of qmm_run_lora against its formula in 64 bits.

Bound per value: the final sum rounds once (2^-24 |Y|, doubled for the second addition of Y0), and
the two products sum at most K + rank + 64 fp32 terms in any order, each sum a tree of short chains
of at most K/32 + 64 terms: (K/32 + rank + 128) 2^-24 of S, the sum of |scale b a x|."""
import pytest
import torch

import layer_plain as plain
from bit_quantized_skinny_gb300 import build_lib

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def qmm():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    build_lib.build()
    from bit_quantized_skinny_gb300 import qmm as q
    q.load()
    return q


def make(M, widths, K, ranks, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    X = rnd(M, K).to(BF16)
    adapters = [[((rnd(r, K) * K ** -0.5).to(BF16), rnd(r, N).to(BF16), 0.25 + 0.5 * k) for k, r in enumerate(ranks)]
                for N in widths]
    return X, adapters, [rnd(M, N) for N in widths]


def call(qmm, X, adapters, Y0, Y, ids, rank_max, n_adapters=None):
    M, K = X.shape
    entries = qmm.make_lora_entries([(qmm.make_lora_adapters(a), X, y0, y, y.shape[1], K)
                                     for a, y0, y in zip(adapters, Y0, Y)])
    ws = torch.full((qmm.lora_workspace_bytes(entries, M, rank_max),), 255, dtype=torch.uint8, device="cuda")
    qmm.run_lora(entries, torch.tensor(ids, dtype=torch.int32, device="cuda"), M, rank_max, ws)
    torch.cuda.synchronize()


def check(Y, Y0, X, ids, adapters):
    K = X.shape[1]
    want, S = plain.lora(X, Y0, ids, adapters)
    rank = max([adapters[a][0].shape[0] for a in ids if a >= 0], default=0)
    tol = 2.0 ** -23 * (want.abs() + Y0.double().abs()) + (K / 32 + rank + 128) * 2.0 ** -24 * S
    err = (Y.double() - want).abs()
    assert bool((err <= tol).all()), f"max error {err.max().item()}, over by {(err - tol).max().item()}"


@pytest.mark.parametrize("M,widths,K,ranks,ids", [
    (1, [256], 256, [1], [0]),
    (1, [5120, 1024, 1024], 5120, [16, 8], [1]),
    (3, [1], 256, [4, 4], [1, -1, 0]),
    (13, [1001, 64], 2304, [3, 17, 48, 64], [0, 1, 2, 3, -1, 0, 0, 2, 1, 3, 3, 3, -1]),
    (32, [777], 512, [5, 31], [0, 1] * 16),
    (32, [520], 512, [256], [0] * 32),
    (32, [264], 1280, [7 + 3 * k for k in range(32)], list(range(31, -1, -1))),
    (9, [300], 17408, [64, 128], [1, 1, 1, 1, 1, 0, 1, 1, 1]),
    (5, [333], 768, [8], [-1] * 5),
    (8, [4099], 4352, [255, 33], [0, 0, 1, 0, 1, 1, -1, 0]),
])
def test_against_the_formula(qmm, M, widths, K, ranks, ids):
    X, adapters, Y0 = make(M, widths, K, ranks, seed=M + K)
    Y = [torch.full_like(y, 7.0) for y in Y0]
    call(qmm, X, adapters, Y0, Y, ids, max(ranks))
    assert qmm.device_status() == 0
    for y, y0, a in zip(Y, Y0, adapters):
        check(y, y0, X, ids, a)


def test_in_place_beside_the_projection_bitwise(qmm):
    """In place over a product's result: the same bits as out of place; rows without adapter untouched."""
    X, adapters, Y0 = make(6, [640], 1024, [12, 20], seed=3)
    ids = [0, -1, 1, 0, -1, 1]
    Y = [torch.empty_like(Y0[0])]
    call(qmm, X, adapters, Y0, Y, ids, 20)
    again = [Y0[0].clone()]
    call(qmm, X, adapters, again, again, ids, 32)
    assert torch.equal(again[0], Y[0])
    assert torch.equal(Y[0][[1, 4]], Y0[0][[1, 4]])


def test_rows_do_not_depend_on_their_batch(qmm):
    """A row's bits are those of a call with that row alone."""
    X, adapters, Y0 = make(7, [512], 2304, [16, 40], seed=4)
    ids = [1, 0, 1, 1, 0, 1, 1]
    Y = [torch.empty_like(Y0[0])]
    call(qmm, X, adapters, Y0, Y, ids, 40)
    for i in range(7):
        one = [torch.empty_like(Y0[0][:1])]
        call(qmm, X[i:i + 1].contiguous(), adapters, [Y0[0][i:i + 1].contiguous()], one, [ids[i]], 40)
        assert torch.equal(one[0][0], Y[0][i])


def test_unaligned_b_rows_and_zero_rank(qmm):
    """Bt on a 2-byte boundary, and an adapter of rank 0."""
    X, adapters, Y0 = make(2, [512], 512, [8, 8], seed=5)
    raw = torch.empty(8 * 512 + 1, dtype=BF16, device="cuda")
    A, Bt, scale = adapters[0][0]
    raw[1:] = Bt.reshape(-1)
    items = [(A, raw[1:].view(8, 512), scale), (A[:0], Bt[:0], 1.0)]
    Y = [torch.empty_like(Y0[0])]
    call(qmm, X, [items], Y0, Y, [0, 1], 8)
    assert qmm.device_status() == 0
    check(Y[0], Y0[0], X, [0, 1], items)
    assert torch.equal(Y[0][1], Y0[0][1])


def test_nan_in_an_adapter_stays_with_its_rows(qmm):
    X, adapters, Y0 = make(4, [256], 512, [8, 8], seed=6)
    adapters[0][1][0][3, 7] = float("nan")
    Y = [torch.empty_like(Y0[0])]
    call(qmm, X, adapters, Y0, Y, [0, 1, -1, 0], 8)
    assert bool(Y[0][1].isnan().all()) and bool(Y[0][[0, 2, 3]].isfinite().all())


def test_bad_ids_and_ranks_are_reported(qmm):
    X, adapters, Y0 = make(4, [256], 512, [8, 16], seed=7)
    Y = [torch.empty_like(Y0[0])]
    call(qmm, X, adapters, Y0, Y, [0, 2, -5, 1000000], 16)
    assert qmm.device_status() == 4 and qmm.device_status() == 0
    check(Y[0][:1], Y0[0][:1], X[:1], [0], adapters[0])
    call(qmm, X, adapters, Y0, Y, [0, 1, 0, 0], 8)          # adapter 1 has more ranks than promised
    assert qmm.device_status() == 4
    check(Y[0][[0, 2, 3]], Y0[0][[0, 2, 3]], X[[0, 2, 3]], [0, 0, 0], adapters[0])


def test_ids_change_between_graph_replays(qmm):
    X, adapters, Y0 = make(4, [384, 256], 512, [8, 16], seed=8)
    Y = [torch.empty_like(y) for y in Y0]
    entries = qmm.make_lora_entries([(qmm.make_lora_adapters(a), X, y0, y, y.shape[1], 512)
                                     for a, y0, y in zip(adapters, Y0, Y)])
    ws = torch.empty(qmm.lora_workspace_bytes(entries, 4, 16), dtype=torch.uint8, device="cuda")
    ids = torch.tensor([0, 0, 0, 0], dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmm.run_lora(entries, ids, 4, 16, ws)
    for now in ([0, 1, -1, 0], [1, 1, 1, 1]):
        ids.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for y, y0, a in zip(Y, Y0, adapters):
            check(y, y0, X, now, a)


@pytest.mark.parametrize("M,widths,K,ranks,ids", [
    # wide projections and many adapters in the table: a block of columns to each warp
    (32, [20480], 256, [5] * 32, [7] * 32),
    (32, [20481], 256, [1 + k % 7 for k in range(32)], [k // 3 for k in range(32)]),
    (32, [20483, 264], 512, [9] * 40, [39, 0] * 16),
    (17, [65544], 256, [4] * 20, [-1] * 3 + [19] * 5 + list(range(9))),
    # adapters with more rows than a warp takes at a time, in runs that alternate
    (31, [1032, 8], 17408, [64] * 4, [0, 1, 2, 3, 0, 0, 1] * 4 + [-1, 3, 3]),
    # warps that take several pieces of K, the last run and the last chunk shorter; chunks in pieces
    (16, [96, 40, 33], 8960 + 256, [40] * 16, list(range(16))),
    (24, [72], 33024, [61, 64] * 12, list(range(24))),
    (32, [24], 66560, [130] * 32, list(range(32))),
])
def test_many_rows_and_many_adapters(qmm, M, widths, K, ranks, ids):
    X, adapters, Y0 = make(M, widths, K, ranks, seed=M + K + 1)
    Y = [torch.full_like(y, 7.0) for y in Y0]
    call(qmm, X, adapters, Y0, Y, ids, max(ranks))
    assert qmm.device_status() == 0
    for y, y0, a in zip(Y, Y0, adapters):
        check(y, y0, X, ids, a)


def test_rows_do_not_depend_on_the_adapters_in_use(qmm):
    """A row of a call with many adapters has the bits of the same row alone with its own."""
    X, adapters, Y0 = make(32, [1000], 8704, [48] * 32, seed=11)
    Y, one = [torch.empty_like(Y0[0])], [torch.empty_like(Y0[0][:1])]
    call(qmm, X, adapters, Y0, Y, list(range(32)), 48)
    for i in (0, 13, 31):
        call(qmm, X[i:i + 1].clone(), [adapters[0][i:i + 1]], [Y0[0][i:i + 1].clone()], one, [0], 48)
        assert torch.equal(one[0][0], Y[0][i])


def test_a_table_with_a_misaligned_adapter(qmm):
    """A on an 8-byte boundary in a table built by hand: reported, its rows get Y0."""
    X, adapters, Y0 = make(3, [256], 512, [8, 8], seed=12)
    Y = [torch.full_like(Y0[0], 7.0)]
    table = qmm.make_lora_adapters(adapters[0])
    raw = torch.zeros(8 * 512 + 4, dtype=BF16, device="cuda")
    host = table.cpu()
    host.view(torch.int64)[host.numel() // 16] = raw.data_ptr() + 8   # the second adapter's first word
    table.copy_(host)
    entries = qmm.make_lora_entries([(table, X, Y0[0], Y[0], 256, 512)])
    ws = torch.empty(qmm.lora_workspace_bytes(entries, 3, 8), dtype=torch.uint8, device="cuda")
    qmm.run_lora(entries, torch.tensor([0, 1, 0], dtype=torch.int32, device="cuda"), 3, 8, ws)
    torch.cuda.synchronize()
    assert qmm.device_status() == 4
    check(Y[0][[0, 2]], Y0[0][[0, 2]], X[[0, 2]], [0, 0], adapters[0])
    assert torch.equal(Y[0][1], Y0[0][1])


@pytest.mark.parametrize("N,K,rank", [(512, 512, 16), (520, 1280, 72), (1000, 768, 32), (264, 512, 200)])
def test_bits_do_not_depend_on_where_bt_lies(qmm, N, K, rank):
    """The same adapter with Bt on 16-byte and on 2-byte boundaries."""
    X, adapters, Y0 = make(3, [N], K, [rank], seed=13)
    A, Bt, scale = adapters[0][0]
    Y = [torch.empty_like(Y0[0])]
    call(qmm, X, [[(A, Bt, scale)]], Y0, Y, [0, -1, 0], rank)
    for shift in (1, 4, 7):
        raw = torch.empty(rank * N + shift, dtype=BF16, device="cuda")
        raw[shift:] = Bt.reshape(-1)
        other = [torch.empty_like(Y0[0])]
        call(qmm, X, [[(A, raw[shift:].view(rank, N), scale)]], Y0, other, [0, -1, 0], rank)
        assert torch.equal(other[0], Y[0])


def test_bits_do_not_depend_on_table_batch_or_form(qmm):
    """A row beside a wide projection: alone (the ranks shared by warps), and among 32 rows with a table of 40
    adapters (a block of columns to each warp)."""
    N, K = 20480, 512
    X, adapters, Y0 = make(32, [N], K, [72] * 4 + [9] * 36, seed=14)
    ids = [0, 1, 2, 3, 0, 0] + list(range(4, 30))
    Y, one = [torch.empty_like(Y0[0])], [torch.empty_like(Y0[0][:1])]
    call(qmm, X, adapters, Y0, Y, ids, 72)
    check(Y[0], Y0[0], X, ids, adapters[0])
    for i in (0, 3, 5, 17):
        call(qmm, X[i:i + 1].clone(), [adapters[0][ids[i]:ids[i] + 1]], [Y0[0][i:i + 1].clone()], one, [0], 72)
        assert torch.equal(one[0][0], Y[0][i])
