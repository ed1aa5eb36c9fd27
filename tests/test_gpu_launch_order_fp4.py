"""GPU test of the 4-bit cache's calls behind each other with nothing between them, where the later launch starts while the
earlier one runs and reads what it writes: the bits are those of the same calls one at a time."""
import pytest
import torch

from bit_quantized_skinny_gb300 import build_lib
from test_gpu_launch_order import same_bits_without_waiting

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


@pytest.mark.parametrize("rows,lens,page", [([4, 8], [700, 90], 64), ([120, 80], [700, 90], 64), ([3000], [3000], 16)])
def test_append_attention_read_and_tokens(qmm, rows, lens, page):
    """Every key that the attention reads is written by the call ahead of it, with few rows a key and with many; and
    tokens from logits that a copy ahead of them writes."""
    Hq, Hk, D, B, T = 10, 2, 128, len(rows), sum(rows)
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    per = -(-max(lens) // page)
    n_slots = B * per * page
    pages = torch.randperm(B * per, generator=g, device="cuda").int().view(B, per)
    Kc, Vc = (torch.zeros(qmm.kv_fp4_bytes(n_slots, Hk, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    # the streams' keys are appended in one call of all lens, the rows' among them
    N = sum(lens)
    slots = torch.cat([pages[b].long()[j // page] * page + j % page
                       for b, j in ((b, torch.arange(n, device="cuda")) for b, n in enumerate(lens))])
    Q, K, V = rnd(N, Hq, D), rnd(N, Hk, D), rnd(N, Hk, D)
    q_out = torch.empty(N, Hq, D, dtype=BF16, device="cuda")
    positions = torch.arange(N, device="cuda").int()
    angle = torch.arange(N, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (
        -torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
    append = qmm.make_norm_rope_fp4(Q, K, V, None, None, cos_sin, positions, slots, q_out, Kc, Vc, n_slots, page, 0.01, 0.01)
    O, lse = torch.empty(T, Hq, D, dtype=BF16, device="cuda"), torch.empty(T, Hq, device="cuda")
    starts = torch.tensor([sum(rows[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
    attn = qmm.make_attn_fp4(q_out[:T], Kc, Vc, Hk, page, None, 0, pages, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                             starts, O, scale=D ** -0.5, k_scale=0.01, v_scale=0.01, lse=lse)
    ws = torch.empty(qmm.attn_fp4_workspace_bytes(attn), dtype=torch.uint8, device="cuda")
    K_out, V_out = torch.empty(N, Hk, D, device="cuda"), torch.empty(N, Hk, D, device="cuda")
    read = qmm.make_kv_fp4_read(Kc, Vc, K_out, V_out, n_slots, page, 0.01, 0.01, slots=slots)
    source = rnd(40, 32003) * 3
    logits, tokens = torch.empty_like(source), torch.empty(40, dtype=torch.int32, device="cuda")
    uniform = torch.rand(40, generator=g, device="cuda")
    pick = qmm.make_sample(logits, uniform, tokens, top_p=torch.full((40,), 0.9, device="cuda"))
    nothing = lambda: None
    same_bits_without_waiting(
        [lambda: qmm.norm_rope_fp4(append), nothing, nothing, lambda: qmm.attn_shared_fp4(attn, ws), nothing,
         lambda: qmm.kv_fp4_read(read), nothing, lambda: logits.copy_(source), lambda: qmm.sample(pick)],
        [Kc, Vc, q_out, O, lse, K_out, V_out, logits, tokens])
    assert qmm.device_status() == 0
