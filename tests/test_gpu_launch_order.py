"""GPU tests of calls behind each other with nothing between them, where the later launch starts while the
earlier one runs and reads what it writes: the bits are those of the same calls one at a time."""
import pytest
import torch

from bit_quantized_skinny_gb300 import build_lib, inputs

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def qmm():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    build_lib.build()
    from bit_quantized_skinny_gb300 import qmm as q
    q.load()
    return q


def same_bits_without_waiting(steps, outputs, rounds=20):
    """steps: callables that enqueue work, in stream order; outputs: the tensors that they write."""
    torch.cuda.synchronize()
    want = []
    for step, out in zip(steps, outputs):
        step()
        torch.cuda.synchronize()
        want.append(out.clone())
    for _ in range(rounds):
        for out in outputs:
            out.zero_()
        for step in steps:
            step()
        torch.cuda.synchronize()
        for a, b in zip(want, outputs):
            assert torch.equal(a, b)


def test_product_of_one_row_behind_the_step_that_writes_its_activations(qmm, oracle_lib):
    """norm_rope writes X, the CUDA-core product of one row reads it; several X in turn."""
    N, K = 512, 1024
    W = torch.from_numpy(oracle_lib.pack(inputs.weights_f32(N, K, 3))).cuda()
    steps, outputs = [], []
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.empty(1, K // 128, 128, dtype=BF16, device="cuda")     # one buffer, written again and again
    for k in range(12):
        q = torch.randn(1, K // 128, 128, generator=g, device="cuda")
        args = qmm.make_norm_rope(q, None, None, None, None, None, None, None, X, None, None)
        Y = torch.zeros(1, N, device="cuda")

        def step(args=args, Y=Y):
            qmm.norm_rope(args)
            qmm.run(W, N, K, X.view(1, K), Y, variant=qmm.VARIANT_FMA)
        steps.append(step)
        outputs.append(Y)
    same_bits_without_waiting(steps, outputs)
    assert qmm.device_status() == 0
