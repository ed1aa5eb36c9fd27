"""GPU tests of qmm_sample where its parameters are at the ends of their ranges: temperatures and logits whose quotients leave
fp32's range, and min_p next to 1.  Tokens are those of the definition, a logprob is off by 2^-24 (|logprob| + 1) as in
test_gpu_sample.py."""
import math

import pytest
import torch

from bit_quantized_skinny_gb300 import build_lib
from test_gpu_sample import logits, run

pytestmark = pytest.mark.gpu
INF = math.inf


@pytest.fixture(scope="module")
def qmm():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    build_lib.build()
    from bit_quantized_skinny_gb300 import qmm as q
    q.load()
    return q


def near(got, want):
    return abs(got - want) <= 2.0 ** -24 * (abs(want) + 1)


def of_equal_weights(stays, u):
    """Token and logprob where the tokens of the sorted list `stays` weigh the same."""
    return stays[int(u * len(stays))], -math.log(len(stays))


@pytest.mark.parametrize("V", [1, 2, 500, 5000, 100003])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_infinite_temperature(qmm, V, dtype):
    """Every weight is 1: min_p of at most 1 lets all tokens stay, above 1 the first alone."""
    x, u = logits(12, V, dtype, seed=1)
    for row in ((INF, 0, 1.0, 1.0), (INF, 0, 1.0, 0.5), (INF, 0, 1.0, 2.0 ** -149), (INF, 0, 1.0, 0.0), (INF, 0, 1.0, 2.0),
                (INF, 0, 1.0, INF), (INF, 1000, 1.0, 1.0), (INF, 60000, 1.0, 1.0), (INF, 60000, 1.0, 3.0), (INF, 3, 1.0, 1.0)):
        tokens, logprobs = run(qmm, x, [row], u)
        for t in range(len(x)):
            order = torch.argsort(x[t].double(), descending=True, stable=True).tolist()
            stays = order[:row[1] or V] if row[3] <= 1 else order[:1]
            token, logprob = of_equal_weights(sorted(stays), u[t].double().item())
            assert tokens[t].item() == token and near(logprobs[t].item(), logprob), (row, t)


@pytest.mark.parametrize("top,temperature", [(0.0, 1.0), (0.0, 0.3), (0.0, 7.0), (1e-4, 1.0), (-0.75, 40.0), (20.0, 1.0)])
def test_min_p_next_to_1(qmm, top, temperature):
    """Two tokens, the second one on the border that min_p draws, or just below it, by many units of its weight: one stays
    with the first, the other does not.  (What is picked of the two goes by u = 0.75 of their sum.)"""
    T, V = 400, 3001
    g = torch.Generator().manual_seed(11)
    f32 = lambda v: torch.tensor(v, dtype=torch.float32).item()
    top, temperature = f32(top), f32(temperature)
    x, u = torch.full((T, V), top - 9.0 * temperature - 1.0), torch.full((T,), 0.75)
    x[:, 40] = top
    rows, want = [], []
    for t in range(T):
        low, high = (0.995, 0.999999) if t % 4 else (0.05, 0.995)
        mp = f32(low + (high - low) * torch.rand((), generator=g).item())
        border = top + temperature * math.log(mp)
        at = torch.tensor(border, dtype=torch.float32)
        steps = torch.tensor(-INF if t % 2 else INF, dtype=torch.float32)
        while True:   # the next logit on the wanted side whose weight is 2^-38 from min_p
            w = math.exp((at.item() - top) / temperature)
            if (w - mp < -2.0 ** -38) if t % 2 else (w - mp > 2.0 ** -38):
                break
            at = torch.nextafter(at, steps)
        x[t, 2000] = at
        rows.append((temperature, 0, 1.0, mp))
        if t % 2:
            want.append((40, 0.0))
        else:
            want.append((40, -math.log(1 + w)) if 0.75 * (1 + w) < 1 else (2000, math.log(w / (1 + w))))
    tokens, logprobs = run(qmm, x.cuda(), rows, u.cuda())
    for t in range(T):
        assert tokens[t].item() == want[t][0] and near(logprobs[t].item(), want[t][1]), (t, rows[t], x[t, 2000].item())


@pytest.mark.parametrize("V,n", [(20000, 2000), (20000, 1024), (20000, 1025), (100003, 9000), (248320, 3)])
def test_many_infinite_logits(qmm, V, n):
    """+inf logits share the weight; top_k counts them and then the others, which weigh nothing."""
    x, u = logits(9, V, seed=3)
    g = torch.Generator(device="cuda").manual_seed(V)
    at = torch.stack([torch.randperm(V, generator=g, device="cuda")[:n].sort().values for _ in range(9)])
    x.scatter_(1, at, INF)
    for k in (0, 1, n - 1, n, n + 1, 5000, V - 1):
        for p, mp in ((1.0, 0.0), (0.5, 0.0), (1.0, 0.3), (0.25, 1.0)):
            if k > V:
                continue
            tokens, logprobs = run(qmm, x, [(1.0, k, p, mp)], u)
            for t in range(9):
                stays = at[t, :k or n].tolist()
                stays = stays[:math.ceil(p * len(stays))]      # the weights before a token's are less than p of all
                token, logprob = of_equal_weights(stays, u[t].double().item())
                assert tokens[t].item() == token and near(logprobs[t].item(), logprob), (k, p, mp, t)


def test_logits_whose_difference_leaves_fp32(qmm):
    """Logits of both signs near the largest fp32: their difference over a large temperature is an ordinary number."""
    V = 2000
    x = torch.full((8, V), -INF)
    at = [(5, 3e38), (900, -3e38), (901, -2.5e38), (1700, 1e38)]
    for i, v in at:
        x[:, i] = v
    u = (torch.arange(8) + 0.5) / 8
    for temperature in (INF, 3.4e38, 1e38, 2.0 ** 125):
        for k, mp in ((0, 0.0), (3, 0.0), (0, 0.05), (4, 0.01)):
            tokens, logprobs = run(qmm, x.cuda(), [(temperature, k, 1.0, mp)], u.cuda())
            exact = {i: torch.tensor(v).double().item() for i, v in at}
            scale = torch.tensor(temperature).double().item()
            w = {i: math.exp((v - exact[5]) / scale) for i, v in exact.items()}
            if k:
                w = {i: w[i] for i in sorted(w, key=lambda i: -exact[i])[:k]}
            w = {i: w[i] for i in sorted(w) if w[i] >= mp}
            total = sum(w.values())
            for t in range(8):
                upto = 0.0
                for i in w:
                    upto += w[i]
                    if upto > u[t].item() * total:
                        break
                assert tokens[t].item() == i and near(logprobs[t].item(), math.log(w[i] / total)), (temperature, k, mp, t)


@pytest.mark.parametrize("temperature", [2.0 ** -149, 2.0 ** -140, 1e-42, 1e-39, 3e-38, 2.0 ** -70])
def test_temperatures_and_logits_next_to_zero(qmm, temperature):
    """Logits that differ by a few of the smallest temperatures, and others that are all far below."""
    V = 3000
    T = torch.tensor(temperature).double().item()
    x = torch.full((8, V), -1.0)
    x[:, 1::2] = -3e38
    at = {700: 0.0, 701: -T, 1500: -3 * T, 2500: -T, 2999: -6 * T}
    for i, v in at.items():
        x[:, i] = v                                              # (exact: a few bits times a power of two, or rounded as `exact` is)
    exact = {i: x[0, i].double().item() for i in at}
    u = (torch.arange(8) + 0.5) / 8
    for k, p, mp in ((0, 1.0, 0.0), (3, 1.0, 0.0), (0, 1.0, 0.2), (0, 0.8, 0.0), (4, 0.9, 0.01)):
        tokens, logprobs = run(qmm, x.cuda(), [(temperature, k, p, mp)], u.cuda())
        w = {i: math.exp(v / T) for i, v in exact.items()}
        order = sorted(w, key=lambda i: (-exact[i], i))[:k or None]
        limit, before, stays = torch.tensor(p).item() * sum(w[i] for i in order), 0.0, []
        for i in order:
            if (p == 1.0 or before < limit) and w[i] >= mp:
                stays.append(i)
            before += w[i]
        total = sum(w[i] for i in stays)
        for t in range(8):
            upto = 0.0
            for i in sorted(stays):
                upto += w[i]
                if upto > u[t].item() * total:
                    break
            assert tokens[t].item() == i and near(logprobs[t].item(), math.log(w[i] / total)), (k, p, mp, t)
