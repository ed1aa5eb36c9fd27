"""GPU test of a decoding step over a 4-bit cache as its parts are used together: the attention half (products, norm and
rotation into the cache, attention, o projection), the lm_head's product, and the tokens of the drafted rows, in one
captured graph.

The bounds.  The attention is compared with its 64-bit form over the values that the cache holds afterwards, and the chain
rounds to 16 bits twice besides the softmax weights (queries, O: 2^-8 of a value each): 2^-5 of the row's root mean square
covers the row's root mean square error, as each value of Y sums a few hundred errors of random sign, and four of those
any single one.  A stored value lies within half a step of the widest gap of its block (6 - 4 = 2 units of a scale that is a
sixth of the block's largest value to 2^-4), or is cut at 6 units: at most 0.18 of the block's largest, and the products'
fp32 sums (2^-12).  The tokens follow from the logits that were computed, by the definition."""
import pytest
import torch

import fp4_plain
import layer_plain as plain
from bit_quantized_skinny_gb300 import build_lib, inputs

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
SCALES = (0.01, 0.013)


@pytest.fixture(scope="module")
def qmm():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    build_lib.build()
    from bit_quantized_skinny_gb300 import qmm as q
    q.load()
    return q


@pytest.mark.parametrize("Hq,Hk,D,page,rows", [(8, 2, 64, 16, [3, 1, 4]), (10, 2, 128, 32, [8, 8, 8, 8])])
def test_steps_with_drafts(qmm, oracle_lib, Hq, Hk, D, page, rows):
    from bit_quantized_skinny_gb300.attention_half import AttentionHalf

    width, V, prefix, B, T = 512, 1024, 75, len(rows), sum(rows)
    shape = {"q": (Hq * D, width), "k": (Hk * D, width), "v": (Hk * D, width), "o": (width, Hq * D), "head": (V, width)}
    g = torch.Generator(device="cuda").manual_seed(7 + D)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    packed = {n: oracle_lib.pack(inputs.weights_f32(N, K, 80 + k)) for k, (n, (N, K)) in enumerate(shape.items())}
    dense = {n: torch.from_numpy(oracle_lib.dequant(packed[n], *shape[n])).cuda().double() for n in shape}
    weights = {n: torch.from_numpy(p).cuda() for n, p in packed.items()}
    lens = [20 + 13 * b + m for b, m in enumerate(rows)]           # own keys after the step
    starts = [sum(rows[:b]) for b in range(B + 1)]
    per_stream, n_pre = -(-(max(lens) + 30) // page), -(-prefix // page)
    n_pages = n_pre + B * per_stream + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    prefix_pages, own = order[:n_pre].contiguous(), order[n_pre:n_pre + B * per_stream].view(B, -1).contiguous()
    cache = []
    for scale in SCALES:
        code, s = fp4_plain.quantise((0.5 * rnd(n_pages * page, Hk, D)).double(), scale)
        cache.append(fp4_plain.pack(code, s, page))
    Kc, Vc = cache
    q_norm, k_norm = 1 + 0.1 * rnd(D), 1 + 0.1 * rnd(D)
    inv = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
    angle = torch.arange(512, dtype=torch.float64, device="cuda")[:, None] * inv
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
    half = AttentionHalf(weights, width, Hq, Hk, D, T, B, Kc, Vc, page, per_stream, q_norm, k_norm, cos_sin, prefix_pages,
                         prefix, kv_scales=SCALES)
    half.pages.copy_(own)
    half.row_starts.copy_(torch.tensor(starts))
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
    hidden, logits = torch.zeros(T, width, dtype=BF16, device="cuda"), torch.empty(T, V, device="cuda")
    uniform, fed, tokens, logprobs = torch.rand(T, generator=g, device="cuda"), i32(T), i32(T), torch.zeros(T, device="cuda")
    accepted, follows = i32(B), i32(B)
    T0, k0, p0, m0 = 0.8, 50, 0.9, 0.01
    column = lambda x, dtype=torch.float32: torch.full((T,), x, dtype=dtype, device="cuda")
    pick = qmm.make_sample(logits, uniform, tokens, temperature=column(T0), top_k=column(k0, torch.int32), top_p=column(p0),
                           min_p=column(m0), logprobs=logprobs, fed=fed, row_starts=half.row_starts, accepted=accepted,
                           next=follows)

    def step():
        half.run()
        hidden.copy_(half.Y)
        qmm.run(weights["head"], V, width, hidden, logits)
        qmm.sample(pick)

    def set_step(lens):
        pos, slots = [], []
        for b, (m, n) in enumerate(zip(rows, lens)):
            for j in range(n - m, n):
                pos.append(prefix + j)
                slots.append(int(own[b, j // page]) * page + j % page)
        half.positions.copy_(torch.tensor(pos))
        half.slots.copy_(torch.tensor(slots))
        half.kv_lens.copy_(torch.tensor(lens))
        half.X.copy_(rnd(T, width))
        uniform.copy_(torch.rand(T, generator=g, device="cuda"))

    def check(lens, before):
        X = half.X.double()
        y = {n: X @ dense[n].T for n in "qkv"}
        q, _ = plain.norm_rope(y["q"].view(T, Hq, D), q_norm, 1e-6, cos_sin, half.positions, False)
        k, _ = plain.norm_rope(y["k"].view(T, Hk, D), k_norm, 1e-6, cos_sin, half.positions, False)
        held = [fp4_plain.unpack(c, Hk, D, page, s) for c, s in zip((Kc, Vc), SCALES)]
        unwritten = torch.ones(n_pages * page, dtype=torch.bool, device="cuda")
        unwritten[half.slots] = False
        for now, was, want in zip(held, before, (k, y["v"].view(T, Hk, D))):
            assert torch.equal(now[unwritten], was[unwritten])
            block = want.unflatten(-1, (-1, 16)).abs().amax(-1).repeat_interleave(16, -1)
            assert bool(((now[half.slots] - want).abs() <= (0.18 + 2.0 ** -12) * block).all())
        O, _, _ = plain.attention(q, *held, page, prefix_pages, prefix, own, lens, starts, D ** -0.5)
        want = O.view(T, Hq * D) @ dense["o"].T
        err = (half.Y.double() - want).abs() / want.square().mean(-1, keepdim=True).sqrt()
        assert bool((err.square().mean(-1).sqrt() <= 2.0 ** -5).all()) and err.max().item() <= 2.0 ** -3
        f32 = lambda v: torch.tensor(v).item()
        clear = 0
        for t in range(T):
            token, logprob, margin = fp4_plain.sample(logits[t].double(), f32(T0), k0, f32(p0), f32(m0), uniform[t].item())
            if margin > 2.0 ** -36:
                clear += 1
                assert tokens[t].item() == token and abs(logprobs[t].item() - logprob) <= 2.0 ** -24 * (abs(logprob) + 1)
        assert clear >= 0.9 * T
        for b in range(B):
            n = 0
            while n + 1 < rows[b] and tokens[starts[b] + n] == fed[starts[b] + n + 1]:
                n += 1
            assert accepted[b].item() == n and follows[b].item() == tokens[starts[b] + n].item()

    set_step(lens)
    before = [fp4_plain.unpack(c, Hk, D, page, s) for c, s in zip((Kc, Vc), SCALES)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):               # the products' workspace is the stream's: one call before the capture
        step()
    torch.cuda.synchronize()
    check(lens, before)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for k in range(3):
        lens = [n + k + 1 for n in lens]
        set_step(lens)
        fed.copy_(tokens.roll(1))               # guesses: some of the tokens of the step before
        before = [fp4_plain.unpack(c, Hk, D, page, s) for c, s in zip((Kc, Vc), SCALES)]
        graph.replay()
        torch.cuda.synchronize()
        check(lens, before)
    # the drafts are what the rows give: all of them stand, and the last row's token follows
    fed[1:] = tokens[:-1]
    graph.replay()
    torch.cuda.synchronize()
    assert accepted.tolist() == [m - 1 for m in rows] and follows.tolist() == [tokens[s - 1].item() for s in starts[1:]]
    assert qmm.device_status() == 0


def test_a_wait_that_runs_out_is_reported(qmm):
    """With a bound far below a memory access's latency the first waits give up: the call ends, sets bit 0, and
    the next call (default bound) is right."""
    from test_gpu_attn_fp4 import Case
    c = Case([8] * 4, [90, 8, 500, 129], 2050, 10, 2, 128, 64)
    qmm.set_wait_limit(2, 50)
    try:
        c.run(qmm)
    finally:
        qmm.set_wait_limit(0, 0)
    assert qmm.device_status() & 1 and qmm.device_status() == 0
    c.run(qmm).check()
    assert qmm.device_status() == 0
