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
