"""GPU tests of qmm_sample against its definition in 64 bits.

Tokens are equal wherever the 64-bit form is further than 2^-36 of the sum of weights from another token: the kernel's
weights are off by a few 2^-43 each, of sums of at least one weight of 1, and a sum of n weights of size w adds their
roundings' spread, sqrt(n) 2^-43, below 2^-36 w n for all n and w here.  A logprob is off by that, and by one rounding to
fp32: 2^-24 |logprob| + 2^-24."""
import math

import pytest
import torch

import fp4_plain
from bit_quantized_skinny_gb300 import build_lib

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def qmm():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    build_lib.build()
    from bit_quantized_skinny_gb300 import qmm as q
    q.load()
    return q


ROWS = [(1.0, 0, 1.0, 0.0), (0.7, 0, 0.9, 0.0), (1.0, 50, 1.0, 0.0), (1.0, 50, 0.9, 0.0), (0.0, 0, 1.0, 0.0), (1.0, 0, 1.0, 0.05),
        (0.8, 40, 0.95, 0.02), (1.5, 1000, 0.99, 0.001), (1.0, 1, 1.0, 0.0), (1.0, 0, 0.0, 0.0), (1.0, 0, 1.0, 1.0),
        (3.0, 0, 0.5, 0.0), (0.01, 0, 0.9, 0.0), (1e-30, 5, 0.9, 0.1), (1e30, 0, 1.0, 0.0), (1.0, 7, 0.3, 0.0), (-1.0, 3, 0.5, 0.1),
        (1.0, -4, 2.0, -1.0), (1.0, 3, 1.0, 2.0), (math.inf, 0, 0.25, 0.0)]


def run(qmm, x, rows, u, **more):
    T = x.shape[0]
    col = lambda k, d: torch.tensor([rows[t % len(rows)][k] for t in range(T)], dtype=d, device="cuda")
    tokens, logprobs = torch.full((T,), -7, dtype=torch.int32, device="cuda"), torch.full((T,), 7.0, device="cuda")
    args = qmm.make_sample(x, u, tokens, temperature=col(0, F32), top_k=col(1, torch.int32), top_p=col(2, F32),
                           min_p=col(3, F32), logprobs=logprobs, **more)
    qmm.sample(args)
    torch.cuda.synchronize()
    return tokens, logprobs


def check(x, rows, u, tokens, logprobs, least=0.9):
    f32 = lambda v: torch.tensor(v, dtype=F32).item()
    clear = 0
    for t in range(x.shape[0]):
        temperature, k, p, m = rows[t % len(rows)]
        token, logprob, margin = fp4_plain.sample(x[t].double(), f32(temperature), k, f32(p), f32(m), u[t].item())
        if margin <= 2.0 ** -36:
            continue
        clear += 1
        assert tokens[t].item() == token, (t, rows[t % len(rows)], tokens[t].item(), token, margin)
        got = logprobs[t].item()
        assert got == logprob if math.isinf(logprob) else abs(got - logprob) <= 2.0 ** -24 * (abs(logprob) + 1), (t, got, logprob)
    assert clear >= least * x.shape[0]


def logits(T, V, dtype=F32, seed=0, spread=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed + V)
    x = torch.randn(T, V, generator=g, device="cuda") * spread
    few = torch.randint(0, V, (T, 20), generator=g, device="cuda")
    x.scatter_add_(1, few, 9.0 * torch.rand(T, 20, generator=g, device="cuda"))
    return x.to(dtype), torch.rand(T, generator=g, device="cuda")


@pytest.mark.parametrize("V,dtype", [(1, F32), (2, F32), (3, BF16), (31, F32), (33, F16), (1000, F32), (1023, BF16), (4097, F32),
                                     (32003, BF16), (32003, F16), (50257, F32), (131071, F32), (248320, F32), (393216, F32),
                                     (393215, BF16)])
def test_against_the_definition(qmm, V, dtype):
    x, u = logits(2 * len(ROWS), V, dtype)
    tokens, logprobs = run(qmm, x, ROWS, u)
    check(x, ROWS, u, tokens, logprobs)
    assert qmm.device_status() == 0


@pytest.mark.parametrize("spread", [0.0, 0.02, 0.5, 8.0])
def test_flat_and_sharp_rows(qmm, spread):
    x, u = logits(len(ROWS), 60000, seed=3, spread=spread)
    if spread == 0.0:
        x = torch.full_like(x, -1.25)      # every logit the same: whole tokens of weight 1
    tokens, logprobs = run(qmm, x, ROWS, u)
    check(x, ROWS, u, tokens, logprobs, least=0.8)


def test_many_random_numbers_on_one_row(qmm):
    """Neighbouring tokens of a flat row, and what a filter leaves: the tokens' counts are those of their weights."""
    V, T = 200, 4000
    x = torch.randn(1, V, device="cuda").expand(T, V)     # rows that are one row (stride 0 is refused: ld < V)
    x = x.contiguous()
    u = (torch.arange(T, device="cuda") + 0.5) / T
    rows = [(1.0, 60, 0.9, 0.0)]
    tokens, _ = run(qmm, x, rows, u)
    w = fp4_plain.sample(x[0].double(), 1.0, 60, torch.tensor(0.9).item(), 0.0, 0.0)
    assert bool((tokens.diff() >= 0).all()) and tokens[0].item() == w[0]
    order = torch.argsort(x[0].double(), descending=True)
    p = torch.softmax(x[0].double()[order][:60], 0)
    kept = order[:60][(p.cumsum(0) - p) < torch.tensor(0.9).item()]
    share = torch.zeros(V, dtype=torch.float64, device="cuda")
    share[kept] = torch.softmax(x[0].double()[kept], 0)
    counts = torch.bincount(tokens, minlength=V).double() / T
    assert bool(((counts - share).abs() <= 1.0 / T + 1e-9).all())     # even random numbers: at most one more or less


def test_ties_go_to_the_lowest_index(qmm):
    V = 5000
    x = torch.zeros(6, V, device="cuda")
    x[:, 100::7] = 2.0
    x[3:, 9] = 2.0
    x[:, 50] = -0.0
    top = [9 if t >= 3 else 100 for t in range(6)]
    u = torch.tensor([0.0, 0.5, 0.999, 0.0, 0.5, 0.999], device="cuda")
    tokens, _ = run(qmm, x, [(0.0, 0, 1.0, 0.0)], u)
    assert tokens.tolist() == top
    tokens, _ = run(qmm, x, [(1.0, 1, 1.0, 0.0)], u)
    assert tokens.tolist() == top
    tokens, logprobs = run(qmm, x, [(1.0, 3, 1.0, 0.0)], u)     # the three lowest of the tied ones
    assert tokens.tolist() == [100, 107, 114, 9, 100, 107]
    assert bool(((logprobs - math.log(1 / 3)).abs() < 1e-6).all())
    n = len(range(100, V, 7))
    k = n + 10                                                  # all of those, and the first ten of the zeros
    tokens, _ = run(qmm, x[:3], [(1e9, k, 1.0, 0.0)], torch.tensor([0.0, 9.5 / k, 10.5 / k], device="cuda"))
    assert tokens.tolist() == [0, 9, 100]
    check(x, [(1.0, 900, 0.7, 0.0)], u, *run(qmm, x, [(1.0, 900, 0.7, 0.0)], u), least=0.5)


def test_masked_and_special_logits(qmm):
    V = 3000
    x, u = logits(8, V, seed=5)
    x[0] = -math.inf
    x[1] = math.nan
    x[2, ::2] = -math.inf
    x[3, 1::2] = math.nan
    x[4, [70, 900]] = math.inf
    x[5] = -math.inf
    x[5, 2999] = -3e38
    x[6] = torch.finfo(F32).min
    x[6, 17] = 1.0
    x[7, 0], x[7, 1] = 3e38, -3e38
    for rows in ([(1.0, 0, 1.0, 0.0)], [(0.0, 0, 1.0, 0.0)], [(0.8, 20, 0.9, 0.0)], [(1.0, 2500, 1.0, 0.0)], [(1.0, 0, 0.5, 0.01)]):
        tokens, logprobs = run(qmm, x, rows, u)
        assert tokens[0].item() == tokens[1].item() == -1 and bool(logprobs[:2].isneginf().all())
        assert tokens[4].item() in (70, 900) and tokens[5].item() == 2999 and tokens[6].item() == 17 and tokens[7].item() == 0
        check(x, rows, u, tokens, logprobs, least=0.5)


def test_parameters_that_are_off_or_odd(qmm):
    x, u = logits(6, 2000, seed=9)
    plain_tokens, plain_logprobs = run(qmm, x, [(1.0, 0, 1.0, 0.0)], u)
    tokens = torch.zeros(6, dtype=torch.int32, device="cuda")
    qmm.sample(qmm.make_sample(x, u, tokens))
    assert torch.equal(tokens, plain_tokens)
    nan = math.nan
    got, _ = run(qmm, x, [(1.0, 0, nan, nan)], u)
    assert torch.equal(got, plain_tokens)
    got, _ = run(qmm, x, [(nan, 0, 1.0, 0.0)], u)
    assert torch.equal(got.long(), x.argmax(-1))
    got, _ = run(qmm, x, [(1.0, 2000, 1.0, 0.0)], u)
    assert torch.equal(got, plain_tokens)
    got, _ = run(qmm, x, [(1.0, 1 << 30, 1.0, 0.0)], u)
    assert torch.equal(got, plain_tokens)
    for odd, as_if in ((1.0, 1 - 2.0 ** -24), (7.0, 1 - 2.0 ** -24), (-1.0, 0.0), (nan, 0.0), (1e-40, 1e-40)):
        got, _ = run(qmm, x, [(1.0, 0, 1.0, 0.0)], torch.full((6,), odd, device="cuda"))
        want, _ = run(qmm, x, [(1.0, 0, 1.0, 0.0)], torch.full((6,), as_if, device="cuda"))
        assert torch.equal(got, want)


def test_strided_and_unaligned_rows(qmm):
    for dtype, V, ld, first in ((F32, 1001, 1003, 1), (BF16, 777, 801, 3), (F16, 4000, 4001, 1), (F32, 4096, 4100, 4)):
        wide = torch.full((9, ld), 50.0, device="cuda").to(dtype).flatten()
        x, u = logits(8, V, dtype, seed=1)
        view = wide[first:first + 8 * ld].view(8, ld)[:, :V]
        view.copy_(x)
        got = run(qmm, view, ROWS, u)
        want = run(qmm, x, ROWS, u)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        check(x, ROWS, u, *got)


def test_rows_do_not_depend_on_each_other(qmm):
    x, u = logits(60, 30011, seed=4)
    tokens, logprobs = run(qmm, x, ROWS, u)
    for t in (0, 7, 33, 59):
        row = [ROWS[t % len(ROWS)]]
        got = run(qmm, x[t:t + 1], row, u[t:t + 1])
        assert torch.equal(got[0], tokens[t:t + 1]) and torch.equal(got[1], logprobs[t:t + 1])


def accept(tokens, fed, starts):
    accepted, after = [], []
    for r0, r1 in zip(starts, starts[1:]):
        n = 0
        while r0 + n + 1 < r1 and tokens[r0 + n] == fed[r0 + n + 1]:
            n += 1
        accepted.append(n)
        after.append(tokens[r0 + n] if r1 > r0 else -1)
    return accepted, after


@pytest.mark.parametrize("rows", [[8, 8, 8, 8], [1], [0, 3, 0, 0, 17, 1], [40], [1] * 300, [0, 0]])
def test_drafts(qmm, rows):
    starts = [0]
    for m in rows:
        starts.append(starts[-1] + m)
    T, V, B = starts[-1] + 2, 501, len(rows)       # two rows behind the last stream
    x, u = logits(T, V, seed=T)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    tokens, _ = run(qmm, x, ROWS, u)
    fed = tokens.roll(1).clone()
    fed[torch.rand(T, generator=torch.Generator().manual_seed(T)).cuda() < 0.25] = 3
    accepted, after = i32([9] * B), i32([9] * B)
    got, _ = run(qmm, x, ROWS, u, fed=fed, row_starts=i32(starts), accepted=accepted, next=after)
    assert torch.equal(got, tokens)
    want = accept(tokens.tolist(), fed.tolist(), starts)
    assert (accepted.tolist(), after.tolist()) == want
    assert qmm.device_status() == 0


def test_row_starts_out_of_range_are_reported(qmm):
    x, u = logits(6, 100)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    for bad in ([0, 2, 1, 6], [0, -4, 4, 6], [0, 2, 4, 1 << 30], [-1, 2, 4, 6]):
        accepted, after = i32([9] * 3), i32([9] * 3)
        run(qmm, x, [(1.0, 0, 1.0, 0.0)], u, fed=i32([0] * 6), row_starts=i32(bad), accepted=accepted, next=after)
        assert qmm.device_status() == 4, bad
        assert bool((accepted < 6).all()) and bool((accepted >= 0).all())


def test_no_rows(qmm):
    x = torch.empty(0, 50, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    empty, accepted, after = i32([]), i32([9, 9]), i32([9, 9])
    qmm.sample(qmm.make_sample(x, x[:, 0], empty))
    qmm.sample(qmm.make_sample(x, x[:, 0].contiguous(), empty, fed=empty, row_starts=i32([0, 0, 0]), accepted=accepted, next=after))
    assert accepted.tolist() == [0, 0] and after.tolist() == [-1, -1]


def test_streams_and_graph(qmm):
    x, u = logits(8, 40001, seed=8)
    want = run(qmm, x, ROWS, u)
    col = lambda k, d: torch.tensor([ROWS[t][k] for t in range(8)], dtype=d, device="cuda")
    tokens = torch.zeros(8, dtype=torch.int32, device="cuda")
    args = qmm.make_sample(x, u, tokens, temperature=col(0, F32), top_k=col(1, torch.int32), top_p=col(2, F32), min_p=col(3, F32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qmm.sample(args, stream=side)
    side.synchronize()
    assert torch.equal(tokens, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmm.sample(args)
    x2, u2 = logits(8, 40001, seed=80)
    want = run(qmm, x2, ROWS, u2)
    x.copy_(x2)
    u.copy_(u2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(tokens, want[0])


def test_calls_behind_each_other_and_at_once(qmm):
    """Calls on two streams, many behind each other: every one gives the same tokens."""
    a, ua = logits(32, 100003, seed=1)
    b, ub = logits(5, 7000, BF16, seed=2)
    want = run(qmm, a, ROWS, ua), run(qmm, b, ROWS, ub)
    col = lambda T, k, d: torch.tensor([ROWS[t % len(ROWS)][k] for t in range(T)], dtype=d, device="cuda")
    make = lambda x, u, tokens: qmm.make_sample(x, u, tokens, temperature=col(len(x), 0, F32), top_k=col(len(x), 1, torch.int32),
                                                top_p=col(len(x), 2, F32), min_p=col(len(x), 3, F32))
    ta, tb = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (32, 5))
    args = make(a, ua, ta), make(b, ub, tb)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, st in zip(args, streams):
            qmm.sample(x, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(ta, want[0][0]) and torch.equal(tb, want[1][0])
