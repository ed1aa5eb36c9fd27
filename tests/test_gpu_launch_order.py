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


def adapters(qmm, widths, K, n, rank, g):
    items = [[((torch.randn(rank, K, generator=g, device="cuda") * K ** -0.5).to(BF16),
               torch.randn(rank, N, generator=g, device="cuda").to(BF16), 1.0) for _ in range(n)] for N in widths]
    return items, [qmm.make_lora_adapters(a) for a in items]


def test_adapters_on_one_workspace(qmm):
    """Calls of different shapes in turn, both forms of the second launch, on one workspace; the second call of
    each pair is in place over the first one's result."""
    g = torch.Generator(device="cuda").manual_seed(2)
    keep, steps, outputs, need = [], [], [], 0
    for M, widths, K, n, rank in ((32, [20480], 512, 32, 16), (3, [1001, 64], 2304, 2, 40), (32, [264], 8704, 8, 64)):
        items, tables = adapters(qmm, widths, K, n, rank, g)
        X = torch.randn(M, K, generator=g, device="cuda").to(BF16)
        Y0, Y = [torch.randn(M, N, generator=g, device="cuda") for N in widths], [torch.zeros(M, N, device="cuda") for N in widths]
        ids = torch.arange(M, dtype=torch.int32, device="cuda") % n
        first = qmm.make_lora_entries([(t, X, a, b, N, K) for t, a, b, N in zip(tables, Y0, Y, widths)])
        again = qmm.make_lora_entries([(t, X, b, b, N, K) for t, b, N in zip(tables, Y, widths)])
        need = max(need, qmm.lora_workspace_bytes(first, M, rank))
        keep.append((items, tables))

        def step(first=first, again=again, ids=ids, M=M, rank=rank):
            qmm.run_lora(first, ids, M, rank, ws)
            qmm.run_lora(again, ids, M, rank, ws)
        steps.append(step)
        outputs.append(Y[0])
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    same_bits_without_waiting(steps, outputs)
    assert qmm.device_status() == 0


def test_adapters_on_two_streams(qmm):
    """Calls on two streams with a workspace each do not disturb each other."""
    g = torch.Generator(device="cuda").manual_seed(3)
    calls = []
    for M, N, K, n, rank in ((32, 20480, 512, 32, 16), (17, 2560, 5120, 5, 48)):
        items, (table,) = adapters(qmm, [N], K, n, rank, g)
        X, Y0 = torch.randn(M, K, generator=g, device="cuda").to(BF16), torch.randn(M, N, generator=g, device="cuda")
        Y, ids = torch.zeros(M, N, device="cuda"), torch.arange(M, dtype=torch.int32, device="cuda") % n
        e = qmm.make_lora_entries([(table, X, Y0, Y, N, K)])
        ws = torch.empty(qmm.lora_workspace_bytes(e, M, rank), dtype=torch.uint8, device="cuda")
        calls.append((e, ids, M, rank, ws, Y, items))
    want = []
    for e, ids, M, rank, ws, Y, _ in calls:
        qmm.run_lora(e, ids, M, rank, ws)
        torch.cuda.synchronize()
        want.append(Y.clone())
        Y.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(40):
        for (e, ids, M, rank, ws, Y, _), st in zip(calls, streams):
            qmm.run_lora(e, ids, M, rank, ws, stream=st)
    torch.cuda.synchronize()
    for w, c in zip(want, calls):
        assert torch.equal(w, c[5])
    assert qmm.device_status() == 0


def test_attention_behind_the_write_of_its_cache(qmm):
    """norm_rope writes the last key and value of a stream, the attention reads them; pass after pass."""
    Hq, Hk, D, page, n = 10, 2, 128, 16, 60
    g = torch.Generator(device="cuda").manual_seed(4)
    Kc, Vc = (torch.randn(8 * page, Hk, D, generator=g, device="cuda").to(BF16) for _ in range(2))
    pages = torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8)
    lens, starts = torch.tensor([n], dtype=torch.int32, device="cuda"), torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    queries = torch.empty(2, Hq, D, dtype=BF16, device="cuda")
    slots = torch.tensor([n - 2, n - 1], device="cuda")
    steps, outputs = [], []
    ws = None
    for k in range(10):
        q, kk, v = (torch.randn(2, h, D, generator=g, device="cuda") for h in (Hq, Hk, Hk))
        norm = qmm.make_norm_rope(q, kk, v, None, None, None, None, slots, queries, Kc, Vc)
        O = torch.zeros(2, Hq, D, dtype=BF16, device="cuda")
        attn = qmm.make_attn(queries, Kc, Vc, page, None, 0, pages, lens, starts, O, scale=D ** -0.5)
        if ws is None:
            ws = torch.empty(qmm.attn_workspace_bytes(attn), dtype=torch.uint8, device="cuda")

        def step(norm=norm, attn=attn):
            qmm.norm_rope(norm)
            qmm.attn_shared(attn, ws)
        steps.append(step)
        outputs.append(O)
    same_bits_without_waiting(steps, outputs)
    assert qmm.device_status() == 0
