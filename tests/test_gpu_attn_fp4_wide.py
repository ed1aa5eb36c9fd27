"""GPU tests of qmm_attn_shared_fp4 with page lists as wide as a program with captured graphs has them, which is the form for few
rows of many keys: where the cache lies behind 4 GiB, over long streams, right behind the append that writes its keys, and inside
the attention half.  Every test asserts the form that it is for."""
import pytest
import torch

from bit_quantized_skinny_gb300 import build_lib, inputs
from test_gpu_attn_fp4 import BF16, F16, Case
from test_gpu_attn_fp4_forms import ROOM, expands, roomy
from test_gpu_launch_order import same_bits_without_waiting

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.fixture(scope="module")
def qmm():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    build_lib.build()
    from bit_quantized_skinny_gb300 import qmm as q
    q.load()
    return q


@pytest.mark.parametrize("D,page", [(128, 64), (64, 256)])
def test_cache_beyond_32_bit_offsets(qmm, D, page):
    """Pages behind the first 4 GiB of each cache, for the prefix, the own keys and the blocks that the joining launch looks at."""
    Hk = 8
    bytes_of_page = page * Hk * D * 9 // 16
    c = roomy(Case([2, 3], [150, 70], 200, 16, Hk, D, page))
    n_pages = (5 << 30) // bytes_of_page
    shift = n_pages - c.n_pages
    c.poke(c.V, 1, 68, 2, 1, 0x7F)                    # a NaN block that the last two rows of stream 1 see
    K, V = (torch.empty(n_pages * bytes_of_page, dtype=torch.uint8, device="cuda") for _ in range(2))
    K[shift * bytes_of_page:], V[shift * bytes_of_page:] = c.K, c.V
    O, lse, S = c.plain()
    c.K, c.V = K, V
    c.prefix_pages += shift
    c.pages += shift
    assert not expands(qmm, c)
    c.run(qmm)
    tolerance, nan = c.tolerance(O, S), O.isnan()
    tolerance[nan], O[nan] = 0.0, 0.0
    assert torch.equal(c.O.isnan(), nan) and bool(nan[3:, 4:6, 16:32].all()) and int(nan.sum()) == 2 * 2 * 16
    assert bool(((c.O.double().nan_to_num(0.0) - O).abs() <= tolerance).all())
    assert bool(((c.lse.double() - lse).abs() <= 2.0 ** -12).all())
    assert qmm.device_status() == 0


@pytest.mark.parametrize("rows,lens,prefix,Hq,Hk,D,page,dtype", [
    ([1, 1], [40000, 33001], 0, 10, 2, 128, 64, BF16),
    ([4] * 20, [1500 + 70 * k for k in range(20)], 6000, 20, 2, 64, 16, F16),
    ([5] * 8, [40 + 9 * k for k in range(8)], 9000, 40, 8, 128, 64, BF16),
    ([1] * 3, [9000, 1, 20000], 0, 64, 1, 128, 256, F16),
])
def test_long_streams_against_the_formula(qmm, rows, lens, prefix, Hq, Hk, D, page, dtype):
    c = roomy(Case(rows, lens, prefix, Hq, Hk, D, page, dtype))
    assert not expands(qmm, c)
    c.run(qmm).check()
    O, lse = c.O.clone(), c.lse.clone()
    c.run(qmm)
    assert torch.equal(c.O, O) and torch.equal(c.lse, lse) and qmm.device_status() == 0


@pytest.mark.parametrize("rows,lens,page", [([4, 8], [700, 90], 64), ([1, 1, 1], [3000, 17, 129], 16), ([12], [12], 16)])
def test_append_and_attention_without_waiting(qmm, rows, lens, page):
    """Every key that the attention reads is written by the call right ahead of it."""
    Hq, Hk, D, B, T = 10, 2, 128, len(rows), sum(rows)
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    per = -(-max(lens) // page)
    n_slots = B * per * page
    pages = torch.randperm(B * per, generator=g, device="cuda").int().view(B, per)
    wide = torch.cat([pages, torch.zeros(B, -(-ROOM // (4 * Hk * D * page * B)), dtype=torch.int32, device="cuda")], 1)
    Kc, Vc = (torch.zeros(qmm.kv_fp4_bytes(n_slots, Hk, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    N = sum(lens)
    slots = torch.cat([pages[b].long()[j // page] * page + j % page
                       for b, j in ((b, torch.arange(n, device="cuda")) for b, n in enumerate(lens))])
    Q, K, V = rnd(N, Hq, D), rnd(N, Hk, D), rnd(N, Hk, D)
    q_out = torch.empty(N, Hq, D, dtype=BF16, device="cuda")
    append = qmm.make_norm_rope_fp4(Q, K, V, None, None, None, None, slots, q_out, Kc, Vc, n_slots, page, 0.01, 0.01)
    O, lse = torch.empty(T, Hq, D, dtype=BF16, device="cuda"), torch.empty(T, Hq, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    attn = qmm.make_attn_fp4(q_out[:T], Kc, Vc, Hk, page, None, 0, wide, i32(lens), i32([sum(rows[:b]) for b in range(B + 1)]), O,
                             scale=D ** -0.5, k_scale=0.01, v_scale=0.01, lse=lse)
    need = qmm.attn_fp4_workspace_bytes(attn)
    assert 0 < need < ROOM                                       # no room for the keys in 16 bits
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    nothing = lambda: None
    same_bits_without_waiting([lambda: qmm.norm_rope_fp4(append), nothing, nothing, lambda: qmm.attn_shared_fp4(attn, ws)],
                              [Kc, Vc, q_out, O, lse])
    assert qmm.device_status() == 0


def test_attention_half_in_a_graph(qmm, oracle_lib):
    """The same steps of an attention half with page lists of what the streams need, and of what they may ever need: the same
    bytes in the cache, and Y apart by what two roundings of O to bf16 and of the weights to 16 bits come to: 2^-7 of a value of O
    each, of random sign over the sums of Y."""
    from bit_quantized_skinny_gb300.attention_half import AttentionHalf

    width, Hq, Hk, D, page, prefix, rows = 512, 10, 2, 128, 32, 75, [8, 1, 0, 5]
    B, T = len(rows), sum(rows)
    shape = {"q": (Hq * D, width), "k": (Hk * D, width), "v": (Hk * D, width), "o": (width, Hq * D)}
    weights = {n: torch.from_numpy(oracle_lib.pack(inputs.weights_f32(N, K, 60 + k))).cuda()
               for k, (n, (N, K)) in enumerate(shape.items())}
    g = torch.Generator(device="cuda").manual_seed(17)
    lens = [20 + 31 * b + m for b, m in enumerate(rows)]
    n_pre, per = -(-prefix // page), -(-(max(lens) + 8) // page)
    order = torch.randperm(n_pre + B * per, generator=g, device="cuda").int()
    prefix_pages, own = order[:n_pre].contiguous(), order[n_pre:].view(B, per)
    held = torch.randint(0, 256, (2, (n_pre + B * per) * page * Hk * D * 9 // 16), generator=g, device="cuda").to(torch.uint8) & 0xBF
    cos_sin = torch.ones(512, D, device="cuda") * 0.5 ** 0.5
    halves, graphs, side = [], [], torch.cuda.Stream()
    for more in (0, -(-ROOM // (4 * Hk * D * page * B))):
        Kc, Vc = held.clone()
        half = AttentionHalf(weights, width, Hq, Hk, D, T, B, Kc, Vc, page, per + more, torch.ones(D, device="cuda"),
                             torch.ones(D, device="cuda"), cos_sin, prefix_pages, prefix, kv_scales=(0.01, 0.013))
        half.pages.fill_(0)
        half.pages[:, :per] = own
        half.row_starts.copy_(torch.tensor([sum(rows[:b]) for b in range(B + 1)]))
        sums = 2 * T * Hq * (4 * D + 16) + 152 * 256 * (4 * D + 16) + 5 * 256
        assert (qmm.attn_fp4_workspace_bytes(half._attn) > sums) is (more == 0)
        halves.append((half, Kc, Vc))
    for step in range(3):
        X = torch.randn(T, width, generator=g, device="cuda")
        now = [n + step for n in lens]
        at = [(b, j) for b, (m, n) in enumerate(zip(rows, now)) for j in range(n - m, n)]
        for half, _, _ in halves:
            half.X.copy_(X)
            half.positions.copy_(torch.tensor([prefix + j for _, j in at]))
            half.slots.copy_(torch.tensor([int(own[b, j // page]) * page + j % page for b, j in at]))
            half.kv_lens.copy_(torch.tensor(now))
        torch.cuda.synchronize()
        if step == 0:
            for half, _, _ in halves:
                half.run(stream=side)                            # (the products' workspace is the stream's)
                side.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    half.run()
                graphs.append(graph)
        else:
            for graph in graphs:
                graph.replay()
        torch.cuda.synchronize()
        (a, Ka, Va), (b, Kb, Vb) = halves
        assert torch.equal(Ka, Kb) and torch.equal(Va, Vb)
        err = (a.Y.double() - b.Y.double()) / a.Y.double().square().mean(-1, keepdim=True).sqrt()
        assert bool((err.square().mean(-1).sqrt() <= 2.0 ** -6).all()) and bool(a.Y.isfinite().all())
    assert qmm.device_status() == 0
