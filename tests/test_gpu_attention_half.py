"""GPU test of the attention half as one chain (products, adapters, norm and rotation into the cache,
attention, o projection) against the same chain in 64 bits on the oracle's dequantized weights.

The bound: the chain rounds to 16 bits three times (queries, cached keys and values, O, each 2^-8 of its
value) and once in the softmax weights; every value of Y sums a few hundred such errors of random
sign.  2^-5 of the root mean square of the row covers them; a wrong head, slot, page or adapter is of
the size of the row itself."""
import numpy as np
import pytest
import torch

import layer_plain as plain
from bit_quantized_skinny_gb300 import build_lib, inputs

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


def test_chain_of_verify_passes(qmm, oracle_lib):
    from bit_quantized_skinny_gb300.attention_half import AttentionHalf

    width, Hq, Hk, D, page, prefix = 512, 8, 2, 64, 16, 75
    shape = {"q": (Hq * D, width), "k": (Hk * D, width), "v": (Hk * D, width), "o": (width, Hq * D)}
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    packed = {n: oracle_lib.pack(inputs.weights_f32(N, K, 40 + k)) for k, (n, (N, K)) in enumerate(shape.items())}
    dense = {n: torch.from_numpy(oracle_lib.dequant(packed[n], *shape[n])).cuda().double() for n in shape}
    weights = {n: torch.from_numpy(p).cuda() for n, p in packed.items()}
    items = {n: [((rnd(r, K) * K ** -0.5).to(BF16), (0.2 * rnd(r, N)).to(BF16), 0.5 + r / 8) for r in (8, 5)]
             for n, (N, K) in shape.items()}
    tables = {n: qmm.make_lora_adapters(v) for n, v in items.items()}
    rows, lens = [3, 1, 4], [20, 33, 4]           # own keys after the pass
    T = sum(rows)
    starts = [0, 3, 4, 8]
    n_pages = 40
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    prefix_pages, own = order[:5].contiguous(), order[5:29].view(3, 8).contiguous()
    Kc, Vc = (rnd(n_pages * page, Hk, D).to(BF16) for _ in range(2))
    q_norm, k_norm = 1 + 0.1 * rnd(D), 1 + 0.1 * rnd(D)
    inv = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
    angle = torch.arange(256, dtype=torch.float64, device="cuda")[:, None] * inv
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
    half = AttentionHalf(weights, width, Hq, Hk, D, T, 3, Kc, Vc, page, 8, q_norm, k_norm, cos_sin, prefix_pages, prefix,
                         adapters=tables, rank_max=8)
    ids = [0, 1, -1, 1, 0, 0, -1, 1]
    half.ids.copy_(torch.tensor(ids))
    half.pages.copy_(own)
    half.row_starts.copy_(torch.tensor(starts))

    def set_pass(lens):
        pos, slots = [], []
        for b, (m, n) in enumerate(zip(rows, lens)):
            for i in range(m):
                j = n - m + i
                pos.append(prefix + j)
                slots.append(int(own[b, j // page]) * page + j % page)
        half.positions.copy_(torch.tensor(pos))
        half.slots.copy_(torch.tensor(slots))
        half.kv_lens.copy_(torch.tensor(lens))
        half.X.copy_(rnd(T, width))

    def check(lens, before_k, before_v):
        X = half.X.double()
        y = {}
        for n in "qkv":
            y[n], _ = plain.lora(half.X, X @ dense[n].T, ids, items[n])
        q, _ = plain.norm_rope(y["q"].view(T, Hq, D), q_norm, 1e-6, cos_sin, half.positions, False)
        k, _ = plain.norm_rope(y["k"].view(T, Hk, D), k_norm, 1e-6, cos_sin, half.positions, False)
        Kp, Vp = before_k.double(), before_v.double()
        Kp[half.slots], Vp[half.slots] = k, y["v"].view(T, Hk, D)
        O, _, _ = plain.attention(q, Kp, Vp, page, prefix_pages, prefix, own, lens, starts, D ** -0.5)
        want, _ = plain.lora(O.view(T, Hq * D), O.view(T, Hq * D) @ dense["o"].T, ids, items["o"])
        rms = want.square().mean(-1, keepdim=True).sqrt()
        err = (half.Y.double() - want).abs() / rms
        assert err.max().item() < 2.0 ** -5 * 4 and err.square().mean().sqrt().item() < 2.0 ** -5, err.max().item()
        unwritten = torch.ones(n_pages * page, dtype=torch.bool, device="cuda")
        unwritten[half.slots] = False
        assert torch.equal(Kc[unwritten], before_k[unwritten]) and torch.equal(Vc[unwritten], before_v[unwritten])

    set_pass(lens)
    before = Kc.clone(), Vc.clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()                  # the products' workspace is the stream's: one call before the capture
    half.run(stream=side)
    side.synchronize()
    check(lens, *before)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        half.run()
    for step in range(3):                       # later passes: each stream accepted some of its rows
        lens = [n + k for n, k in zip(lens, (3, 1, 2))]
        set_pass(lens)
        before = Kc.clone(), Vc.clone()
        graph.replay()
        torch.cuda.synchronize()
        check(lens, *before)
    assert qmm.device_status() == 0


def test_a_full_verify_pass(qmm, oracle_lib):
    """4 requests of 8 drafted rows with an adapter each, 8 query heads to a key/value head: 32 rows are two row
    tiles for the prefix.  Per row, the root mean square of the error is at most 2^-5 of the row's (the bound
    above), and no value is off by more than four of those (a bell curve's 16384 values)."""
    from bit_quantized_skinny_gb300.attention_half import AttentionHalf

    width, Hq, Hk, D, page, prefix, B, m = 512, 16, 2, 128, 32, 700, 4, 8
    T = B * m
    shape = {"q": (Hq * D, width), "k": (Hk * D, width), "v": (Hk * D, width), "o": (width, Hq * D)}
    g = torch.Generator(device="cuda").manual_seed(6)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    packed = {n: oracle_lib.pack(inputs.weights_f32(N, K, 60 + k)) for k, (n, (N, K)) in enumerate(shape.items())}
    dense = {n: torch.from_numpy(oracle_lib.dequant(packed[n], *shape[n])).cuda().double() for n in shape}
    items = {n: [((rnd(r, K) * K ** -0.5).to(BF16), (0.2 * rnd(r, N)).to(BF16), 1.0) for r in (16, 64, 8, 33)]
             for n, (N, K) in shape.items()}
    lens, starts = [8, 40, 130, 95], [0, 8, 16, 24, 32]
    n_pages = 80
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    prefix_pages, own = order[:22].contiguous(), order[22:62].view(B, 10).contiguous()
    Kc, Vc = (rnd(n_pages * page, Hk, D).to(BF16) for _ in range(2))
    q_norm, k_norm = 1 + 0.1 * rnd(D), 1 + 0.1 * rnd(D)
    inv = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
    angle = torch.arange(1024, dtype=torch.float64, device="cuda")[:, None] * inv
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
    half = AttentionHalf({n: torch.from_numpy(p).cuda() for n, p in packed.items()}, width, Hq, Hk, D, T, B, Kc, Vc, page, 10,
                         q_norm, k_norm, cos_sin, prefix_pages, prefix,
                         adapters={n: qmm.make_lora_adapters(v) for n, v in items.items()}, rank_max=64)
    ids = [t // m for t in range(T)]
    own_at = [lens[t // m] - m + t % m for t in range(T)]
    half.ids.copy_(torch.tensor(ids))
    half.pages.copy_(own)
    half.row_starts.copy_(torch.tensor(starts))
    half.kv_lens.copy_(torch.tensor(lens))
    half.positions.copy_(torch.tensor([prefix + j for j in own_at]))
    half.slots.copy_(torch.tensor([int(own[t // m, j // page]) * page + j % page for t, j in enumerate(own_at)]))
    half.X.copy_(rnd(T, width))
    Kp, Vp = Kc.double(), Vc.double()
    half.run()
    torch.cuda.synchronize()
    assert qmm.device_status() == 0
    X = half.X.double()
    y = {n: plain.lora(half.X, X @ dense[n].T, ids, items[n])[0] for n in "qkv"}
    q, _ = plain.norm_rope(y["q"].view(T, Hq, D), q_norm, 1e-6, cos_sin, half.positions, False)
    k, _ = plain.norm_rope(y["k"].view(T, Hk, D), k_norm, 1e-6, cos_sin, half.positions, False)
    Kp[half.slots], Vp[half.slots] = k, y["v"].view(T, Hk, D)
    O, _, _ = plain.attention(q, Kp, Vp, page, prefix_pages, prefix, own, lens, starts, D ** -0.5)
    want, _ = plain.lora(O.view(T, Hq * D), O.view(T, Hq * D) @ dense["o"].T, ids, items["o"])
    err = (half.Y.double() - want).abs() / want.square().mean(-1, keepdim=True).sqrt()
    assert bool((err.square().mean(-1).sqrt() <= 2.0 ** -5).all()) and err.max().item() <= 2.0 ** -3
