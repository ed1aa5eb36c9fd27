"""GPU tests of qmm_norm_rope against its formula in 64 bits.

Bound per value, from the arithmetic: one rounding to the output type (unit roundoff u, plus half the
smallest fp16 subnormal), and fp32 steps before it: the sum of D squares (at most D + 8 roundings
of the mean square, so half of that on its root), the root, two products and the rotation's two,
each 2^-24, on values of at most |a| + |b|: 2^-24 (D/2 + 16) (|a| + |b|)."""
import pytest
import torch

import layer_plain as plain
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


def table(max_pos, rot):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()


def check(got, want, size, D):
    tol = plain.UNIT[got.dtype] * want.abs() + 2.0 ** -24 * (D / 2 + 16) * size + 2.0 ** -25
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), f"max error {err.max().item()}, over the bound by {(err - tol).max().item()}"


@pytest.mark.parametrize("T,Hq,Hk,D,rot,interleaved,src,dst", [
    (1, 40, 8, 128, 128, False, F32, BF16),
    (32, 40, 8, 128, 128, False, F32, BF16),
    (7, 5, 1, 64, 64, True, F32, F16),
    (33, 24, 3, 64, 32, True, BF16, F16),
    (19, 3, 3, 64, 16, False, F16, BF16),
    (130, 6, 2, 256, 64, False, F32, BF16),
    (11, 6, 2, 256, 256, True, BF16, BF16),
    (9, 4, 2, 128, 48, False, F16, F16),
    (9, 4, 2, 128, 0, False, F32, BF16),
    (1500, 10, 2, 128, 128, False, F32, BF16),
])
def test_against_the_formula(qmm, T, Hq, Hk, D, rot, interleaved, src, dst):
    g = torch.Generator(device="cuda").manual_seed(T + D)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    pad = 8   # rows of a wider buffer: the q, k and v of one fused projection
    fused = (rnd(T, (Hq + 2 * Hk) * D + pad) * torch.exp(2 * rnd(T, 1))).to(src)
    Q = fused[:, :Hq * D].unflatten(1, (Hq, D))
    K = fused[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    V = fused[:, (Hq + Hk) * D:(Hq + 2 * Hk) * D].unflatten(1, (Hk, D))
    qw, kw = 1 + 0.3 * rnd(D), 1 + 0.3 * rnd(D)
    cs = table(5000, rot) if rot else None
    pos = torch.randint(0, 5000, (T,), generator=g, device="cuda").int()
    n_slots = T + 37
    slots = torch.randperm(n_slots, generator=g, device="cuda")[:T].clone()
    slots[T // 2] = -1 if T > 1 else slots[0]      # a padding row
    Kc, Vc = (torch.full((n_slots, Hk, D), 5.0, dtype=dst, device="cuda") for _ in range(2))
    out = torch.full((T, Hq, D), 5.0, dtype=dst, device="cuda")
    args = qmm.make_norm_rope(Q, K, V, qw, kw, cs, pos, slots, out, Kc, Vc, eps=1e-6, interleaved=interleaved)
    qmm.norm_rope(args)
    torch.cuda.synchronize()
    assert qmm.device_status() == 0
    check(out, *plain.norm_rope(Q, qw, 1e-6, cs, pos, interleaved), D)
    live = slots >= 0
    check(Kc[slots[live]], *(v[live] for v in plain.norm_rope(K, kw, 1e-6, cs, pos, interleaved)), D)
    assert torch.equal(Vc[slots[live]], V[live].to(dst))
    rest = torch.ones(n_slots, dtype=torch.bool, device="cuda")
    rest[slots[live]] = False
    assert bool((Kc[rest] == 5.0).all()) and bool((Vc[rest] == 5.0).all())


def test_without_weights_keys_or_values(qmm):
    T, H, D = 5, 3, 128
    Q, K = torch.randn(T, H, D, device="cuda"), torch.randn(T, 1, D, device="cuda")
    cs, pos = table(64, D), torch.arange(T, dtype=torch.int32, device="cuda")
    out = torch.empty(T, H, D, dtype=BF16, device="cuda")
    qmm.norm_rope(qmm.make_norm_rope(Q, None, None, None, None, cs, pos, None, out, None, None))
    check(out, *plain.norm_rope(Q, None, 1e-6, cs, pos, False), D)
    Kc, slots = torch.zeros(8, 1, D, dtype=BF16, device="cuda"), torch.arange(T, device="cuda") + 2
    qmm.norm_rope(qmm.make_norm_rope(Q, K, None, None, None, cs, pos, slots, out, Kc, None))
    check(Kc[2:2 + T], *plain.norm_rope(K, None, 1e-6, cs, pos, False), D)


def test_zero_rows_zero_heads_and_special_values(qmm):
    D = 64
    cs, pos = table(16, D), torch.zeros(3, dtype=torch.int32, device="cuda")
    Q = torch.zeros(3, 2, D, device="cuda")
    Q[1, 0, 5] = float("nan")
    Q[2, 1] = 1e-30
    out = torch.empty(3, 2, D, dtype=BF16, device="cuda")
    qmm.norm_rope(qmm.make_norm_rope(Q, None, None, None, None, cs, pos, None, out, None, None))
    torch.cuda.synchronize()
    assert bool((out[0] == 0).all()) and bool(out[1, 0].isnan().all()) and bool((out[1, 1] == 0).all())
    assert bool(out[2].isfinite().all())
    empty = torch.empty(0, 2, D, device="cuda")
    qmm.norm_rope(qmm.make_norm_rope(empty, None, None, None, None, cs, pos[:0], None, out[:0], None, None))


def test_indices_out_of_range_are_reported_and_write_nothing(qmm):
    T, H, D = 4, 2, 128
    Q, K, V = (torch.randn(T, H, D, device="cuda") for _ in range(3))
    cs = table(10, D)
    pos = torch.tensor([0, 10, -1, 3], dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, 1, 1 << 40, 2], device="cuda")
    out = torch.empty(T, H, D, dtype=BF16, device="cuda")
    Kc, Vc = (torch.zeros(4, H, D, dtype=BF16, device="cuda") for _ in range(2))
    qmm.norm_rope(qmm.make_norm_rope(Q, K, V, None, None, cs, pos, slots, out, Kc, Vc))
    assert qmm.device_status() == 4 and qmm.device_status() == 0
    good = torch.tensor([0, 3], device="cuda")
    check(out[good], *(v[good] for v in plain.norm_rope(Q, None, 1e-6, cs, pos.clamp(0, 9), False)), D)
    assert torch.equal(Vc[slots[good]], V[good].to(BF16)) and bool((Vc[3] == 0).all())


def test_other_stream_and_graph(qmm):
    T, H, D = 8, 4, 128
    Q = torch.randn(T, H, D, device="cuda")
    cs, pos = table(100, D), torch.arange(T, dtype=torch.int32, device="cuda")
    out = torch.empty(T, H, D, dtype=BF16, device="cuda")
    args = qmm.make_norm_rope(Q, None, None, None, None, cs, pos, None, out, None, None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qmm.norm_rope(args, stream=side)
    side.synchronize()
    first = out.clone()
    check(first, *plain.norm_rope(Q, None, 1e-6, cs, pos, False), D)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmm.norm_rope(args)
    pos += 50
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    check(out, *plain.norm_rope(Q, None, 1e-6, cs, pos, False), D)


def test_behind_the_launch_that_writes_its_inputs(qmm):
    """Call after call behind adapters that write q, k and v in place, with nothing between them: the bits
    of the same calls one at a time."""
    T, Hq, Hk, D, width = 32, 40, 8, 128, 512
    g = torch.Generator(device="cuda").manual_seed(9)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    widths = [Hq * D, Hk * D, Hk * D]
    X = [rnd(T, width).to(BF16) for _ in range(8)]
    adapters = [[((rnd(16, width) * width ** -0.5).to(BF16), rnd(16, N).to(BF16), 1.0) for _ in range(4)] for N in widths]
    tables = [qmm.make_lora_adapters(a) for a in adapters]
    y0, y = [rnd(T, N) for N in widths], [torch.empty(T, N, device="cuda") for N in widths]
    ids = torch.arange(T, dtype=torch.int32, device="cuda") % 4
    cs, pos = table(256, D), torch.arange(T, dtype=torch.int32, device="cuda")
    slots = torch.arange(T, device="cuda")
    calls = []
    for x in X:
        entries = qmm.make_lora_entries([(t, x, a, b, N, width) for t, a, b, N in zip(tables, y0, y, widths)])
        out = torch.zeros(T, Hq, D, dtype=BF16, device="cuda")
        Kc, Vc = (torch.zeros(T, Hk, D, dtype=BF16, device="cuda") for _ in range(2))
        args = qmm.make_norm_rope(y[0].view(T, Hq, D), y[1].view(T, Hk, D), y[2].view(T, Hk, D), None, None, cs, pos, slots,
                                  out, Kc, Vc)
        calls.append((entries, args, (out, Kc, Vc)))
    ws = torch.empty(qmm.lora_workspace_bytes(calls[0][0], T, 16), dtype=torch.uint8, device="cuda")
    want = []
    for entries, args, outs in calls:
        qmm.run_lora(entries, ids, T, 16, ws)
        torch.cuda.synchronize()
        qmm.norm_rope(args)
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
    for _ in range(20):
        for _, _, outs in calls:
            for t in outs:
                t.zero_()
        for entries, args, _ in calls:
            qmm.run_lora(entries, ids, T, 16, ws)
            qmm.norm_rope(args)
        for w, (_, _, outs) in zip(want, calls):
            assert all(torch.equal(a, b) for a, b in zip(w, outs))
    assert qmm.device_status() == 0


@pytest.mark.parametrize("T,Hq,Hk,D,rot,interleaved,src,dst", [
    # more than 2048 fp32 rows: two heads at a time; heads that leave the last step half or all but empty
    (2049, 13, 3, 64, 32, False, F32, BF16),
    (2050, 5, 1, 64, 64, True, F32, F16),
    (4099, 7, 1, 128, 128, False, F32, BF16),
    (2301, 9, 2, 128, 48, True, F32, F16),
    (2111, 3, 2, 256, 256, False, F32, F16),
    (2051, 2, 1, 256, 64, True, F32, BF16),
    # as many rows of 16 bits: one head at a time
    (4099, 7, 1, 128, 128, True, BF16, BF16),
])
def test_many_rows_against_the_formula(qmm, T, Hq, Hk, D, rot, interleaved, src, dst):
    test_against_the_formula(qmm, T, Hq, Hk, D, rot, interleaved, src, dst)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_rows_without_values_or_rotation(qmm, D):
    T, Hq, Hk = 2500, 5, 2
    Q, K = torch.randn(T, Hq, D, device="cuda"), torch.randn(T, Hk, D, device="cuda")
    out, Kc = torch.empty(T, Hq, D, dtype=BF16, device="cuda"), torch.full((T + 1, Hk, D), 5.0, dtype=BF16, device="cuda")
    slots = torch.randperm(T + 1, device="cuda")[:T].clone()
    slots[::7] = -1
    qmm.norm_rope(qmm.make_norm_rope(Q, K, None, None, None, None, None, slots, out, Kc, None))
    check(out, *plain.norm_rope(Q, None, 1e-6, None, None, False), D)
    live = slots >= 0
    check(Kc[slots[live]], *(v[live] for v in plain.norm_rope(K, None, 1e-6, None, None, False)), D)
    rest = torch.ones(T + 1, dtype=torch.bool, device="cuda")
    rest[slots[live]] = False
    assert bool((Kc[rest] == 5.0).all())


@pytest.mark.parametrize("T,Hq,Hk,D,rot,interleaved,dst", [
    # heads that fill an even number of steps, the last one partly; seven steps, the last pair half empty
    (2049, 9, 3, 64, 64, False, BF16),
    (2050, 45, 2, 64, 16, True, F16),
    (2111, 21, 2, 128, 128, True, BF16),
    (2053, 5, 1, 128, 64, False, F16),
    (2049, 9, 2, 256, 128, False, BF16),
])
def test_many_rows_in_pairs_of_heads(qmm, T, Hq, Hk, D, rot, interleaved, dst):
    test_against_the_formula(qmm, T, Hq, Hk, D, rot, interleaved, F32, dst)
