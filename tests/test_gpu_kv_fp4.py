"""GPU tests of qmm_norm_rope_fp4 and qmm_kv_fp4_read: the packed bytes are those of the definition, computed in
64 bits, byte for byte.  (A 64-bit result off by 2^-50 decides differently from the real number only where
that comes within 2^-50 of a border of binary32, of a code or of a scale: not among some 10^6 values.)"""
import pytest
import torch

import fp4_plain
import layer_plain as plain
from bit_quantized_skinny_gb300 import build_lib
from test_gpu_norm_rope import check, table

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
EPS = torch.tensor(1e-6, dtype=F32).item()   # as the call takes it


@pytest.fixture(scope="module")
def qmm():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    build_lib.build()
    from bit_quantized_skinny_gb300 import qmm as q
    q.load()
    return q


def written(cache, slots, code, s, page):
    """`cache` with codes and scales at `slots`."""
    Hk, D = code.shape[1:]
    pages = cache.clone().view(-1, Hk, page * (D // 2 + D // 16))
    two = (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)
    p, i = slots // page, slots % page
    h = torch.arange(Hk, device="cuda")
    for j in range(D // 2):
        pages[p[:, None], h, (i * (D // 2) + j)[:, None]] = two[..., j]
    for j in range(D // 16):
        pages[p[:, None], h, (page * (D // 2) + i * (D // 16) + j)[:, None]] = s[..., j].to(torch.uint8)
    return pages.flatten()


class Case:
    def __init__(self, qmm, T, Hq, Hk, D, rot, interleaved, src, dst, page, k_scale=0.04, v_scale=0.055, seed=0, spread=2.0):
        g = torch.Generator(device="cuda").manual_seed(seed + T + D)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
        # rows of a wider buffer: the q, k and v of one fused projection
        fused = (rnd(T, (Hq + 2 * Hk) * D + 8) * torch.exp(spread * rnd(T, 1))).to(src)
        self.Q = fused[:, :Hq * D].unflatten(1, (Hq, D))
        self.K = fused[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
        self.V = fused[:, (Hq + Hk) * D:(Hq + 2 * Hk) * D].unflatten(1, (Hk, D))
        self.qw, self.kw = 1 + 0.3 * rnd(D), 1 + 0.3 * rnd(D)
        self.cs, self.interleaved = (table(5000, rot) if rot else None), interleaved
        self.pos = torch.randint(0, 5000, (T,), generator=g, device="cuda").int()
        self.n_slots = -(-(T + 37) // page) * page
        self.slots = torch.randperm(self.n_slots, generator=g, device="cuda")[:T].clone()
        if T > 1:
            self.slots[T // 2] = -1      # a padding row
        self.page, self.scales = page, (k_scale, v_scale)
        self.Kc, self.Vc = (torch.randint(0, 256, (qmm.kv_fp4_bytes(self.n_slots, Hk, D),), generator=g, device="cuda",
                                          dtype=torch.uint8) for _ in range(2))
        self.out = torch.full((T, Hq, D), 5.0, dtype=dst, device="cuda")

    def args(self, qmm):
        return qmm.make_norm_rope_fp4(self.Q, self.K, self.V, self.qw, self.kw, self.cs, self.pos, self.slots, self.out,
                                      self.Kc, self.Vc, n_slots=self.n_slots, page_size=self.page, k_scale=self.scales[0],
                                      v_scale=self.scales[1], interleaved=self.interleaved)

    def want(self):
        live = self.slots >= 0
        y, _ = plain.norm_rope(self.K, self.kw, EPS, self.cs, self.pos, self.interleaved)
        k = fp4_plain.quantise(fp4_plain.f32(y), self.scales[0])
        v = fp4_plain.quantise(self.V.double(), self.scales[1])
        return [written(c, self.slots[live], code[live], s[live], self.page) for c, (code, s) in ((self.Kc, k), (self.Vc, v))]

    def run_and_check(self, qmm):
        want_k, want_v = self.want()
        qmm.norm_rope_fp4(self.args(qmm))
        torch.cuda.synchronize()
        assert qmm.device_status() == 0
        check(self.out, *plain.norm_rope(self.Q, self.qw, EPS, self.cs, self.pos, self.interleaved), self.Q.shape[2])
        assert torch.equal(self.Vc, want_v), f"{int((self.Vc != want_v).sum())} bytes of the values"
        assert torch.equal(self.Kc, want_k), f"{int((self.Kc != want_k).sum())} bytes of the keys"


@pytest.mark.parametrize("T,Hq,Hk,D,rot,interleaved,src,dst,page", [
    (1, 40, 8, 128, 128, False, F32, BF16, 64),
    (32, 40, 8, 128, 128, False, F32, BF16, 64),
    (7, 5, 1, 64, 64, True, F32, F16, 16),
    (33, 24, 3, 64, 32, True, BF16, F16, 16),
    (19, 3, 3, 64, 16, False, F16, BF16, 4096),
    (130, 6, 2, 256, 64, False, F32, BF16, 128),
    (11, 6, 2, 256, 256, True, BF16, BF16, 32),
    (9, 4, 2, 128, 48, False, F16, F16, 16),
    (9, 4, 2, 128, 0, False, F32, BF16, 256),
    (1500, 10, 2, 128, 128, False, F32, BF16, 64),
    (2311, 24, 3, 64, 32, True, BF16, F16, 16),
    (3001, 5, 1, 128, 128, False, F32, BF16, 64),
])
def test_bytes_of_the_definition(qmm, T, Hq, Hk, D, rot, interleaved, src, dst, page):
    Case(qmm, T, Hq, Hk, D, rot, interleaved, src, dst, page).run_and_check(qmm)


@pytest.mark.parametrize("k_scale,v_scale,spread", [(1.0, 1.0, 0.0), (2.0 ** -60, 2.0 ** 60, 0.0), (1e-3, 1e-3, 4.0),
                                                    (0.0123, 37.0, 6.0)])
def test_tensor_scales(qmm, k_scale, v_scale, spread):
    """Scales that saturate, that are subnormal E4M3 values, and blocks that round to nothing."""
    Case(qmm, 40, 4, 2, 128, 128, False, F32, BF16, 16, k_scale, v_scale, spread=spread).run_and_check(qmm)


def test_values_on_borders(qmm):
    """Values halfway between codes, and blocks whose largest value puts the scale halfway: ties go to even."""
    T, Hk, D, page = 64, 2, 64, 16
    c = Case(qmm, T, 2, Hk, D, 0, False, F32, BF16, page, k_scale=0.25, v_scale=0.25)
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], device="cuda")
    V = (borders[torch.arange(T * Hk * D, device="cuda") % 8] * (1 - 2 * (torch.arange(T * Hk * D, device="cuda") % 3 == 0))
         ).view(T, Hk, D).float()
    V[..., 0] = 6.0 * (1 + torch.arange(T, device="cuda")[:, None] / 16)     # scales 1, 17/16 (a tie), 9/8, ...
    c.V = (V * 0.25).contiguous()
    c.K = c.V.clone()
    c.run_and_check(qmm)


def test_special_values(qmm):
    T, Hk, D, page = 6, 2, 64, 16
    c = Case(qmm, T, 2, Hk, D, 64, False, F32, BF16, page)
    c.V = c.V.clone()
    c.K = c.K.clone()
    c.V[0, 0, 3], c.V[1, 1, 40], c.V[2, 0, 63] = float("nan"), float("inf"), -float("inf")
    c.V[3], c.K[3] = 0.0, 0.0
    c.K[4, 1, 7] = float("nan")
    c.K[5, 0] *= 1e25                    # squares beyond binary32: the definition is in real numbers
    c.K[5, 1] *= 1e-25
    c.slots = torch.arange(T, device="cuda")
    c.run_and_check(qmm)
    v = fp4_plain.unpack(c.Vc, Hk, D, page, c.scales[1])
    assert bool(v[0, 0, :16].isnan().all()) and bool(v[0, 0, 16:].isfinite().all()) and bool((v[3] == 0).all())


def test_same_bits_whatever_the_batch(qmm):
    c = Case(qmm, 300, 10, 2, 128, 128, False, F32, BF16, 64)
    c.slots = torch.randperm(c.n_slots, device="cuda")[:300].clone()
    c.Kc.zero_()
    c.Vc.zero_()
    qmm.norm_rope_fp4(c.args(qmm))
    k, v = c.Kc.clone(), c.Vc.clone()
    c.Kc.zero_()
    c.Vc.zero_()
    for t in range(300):
        one = slice(t, t + 1)
        qmm.norm_rope_fp4(qmm.make_norm_rope_fp4(c.Q[one], c.K[one], c.V[one], c.qw, c.kw, c.cs, c.pos[one], c.slots[one],
                                                 c.out[one], c.Kc, c.Vc, n_slots=c.n_slots, page_size=c.page,
                                                 k_scale=c.scales[0], v_scale=c.scales[1]))
    torch.cuda.synchronize()
    assert torch.equal(c.Kc, k) and torch.equal(c.Vc, v)


def test_without_keys_or_values(qmm):
    T, H, D, page = 5, 3, 128, 16
    Q, K = torch.randn(T, H, D, device="cuda"), torch.randn(T, 1, D, device="cuda")
    cs, pos = table(64, D), torch.arange(T, dtype=torch.int32, device="cuda")
    out = torch.empty(T, H, D, dtype=BF16, device="cuda")
    qmm.norm_rope_fp4(qmm.make_norm_rope_fp4(Q, None, None, None, None, cs, pos, None, out, None, None, n_slots=page,
                                             page_size=page))
    check(out, *plain.norm_rope(Q, None, EPS, cs, pos, False), D)
    Kc, slots = torch.zeros(qmm.kv_fp4_bytes(page, 1, D), dtype=torch.uint8, device="cuda"), torch.arange(T, device="cuda") + 2
    qmm.norm_rope_fp4(qmm.make_norm_rope_fp4(Q, K, None, None, None, cs, pos, slots, out, Kc, None, n_slots=page,
                                             page_size=page, k_scale=0.01))
    code, s = fp4_plain.quantise(fp4_plain.f32(plain.norm_rope(K, None, EPS, cs, pos, False)[0]), 0.01)
    assert torch.equal(Kc, written(torch.zeros_like(Kc), slots, code, s, page))


def test_indices_out_of_range_write_nothing(qmm):
    c = Case(qmm, 4, 2, 2, 128, 128, False, F32, BF16, 16)
    c.slots = torch.tensor([0, 1, 1 << 40, c.n_slots], device="cuda")
    kc = c.Kc.clone()
    good = c.slots < 2
    qmm.norm_rope_fp4(c.args(qmm))
    assert qmm.device_status() == 4 and qmm.device_status() == 0
    y, _ = plain.norm_rope(c.K, c.kw, EPS, c.cs, c.pos, False)
    code, s = fp4_plain.quantise(fp4_plain.f32(y), c.scales[0])
    assert torch.equal(c.Kc, written(kc, c.slots[good], code[good], s[good], c.page))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n,Hk,D,page", [(64, 8, 128, 64), (48, 3, 64, 16), (256, 1, 256, 256)])
def test_read(qmm, dtype, n, Hk, D, page):
    g = torch.Generator(device="cuda").manual_seed(n)
    rnd = lambda: torch.randint(0, 256, (qmm.kv_fp4_bytes(n, Hk, D),), generator=g, device="cuda", dtype=torch.uint8)
    scale = (0.037, 0.11)
    Kc, Vc = rnd(), rnd()
    for c in (Kc, Vc):     # scales are not negative; 127 is NaN
        c.view(-1, Hk, page * D * 9 // 16)[..., page * D // 2:] &= 127
    values = lambda c, s: fp4_plain.f32(fp4_plain.unpack(c, Hk, D, page, s)).float().to(dtype)
    same = lambda a, b: torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))
    K, V = (torch.full((n, Hk, D), 3.0, dtype=dtype, device="cuda") for _ in range(2))
    qmm.kv_fp4_read(qmm.make_kv_fp4_read(Kc, Vc, K, V, n_slots=n, page_size=page, k_scale=scale[0], v_scale=scale[1]))
    assert same(K, values(Kc, scale[0])) and same(V, values(Vc, scale[1]))
    slots = torch.randperm(n, generator=g, device="cuda")[:13].clone()
    slots[4] = -1
    K13 = torch.full((13, Hk, D), 3.0, dtype=dtype, device="cuda")
    qmm.kv_fp4_read(qmm.make_kv_fp4_read(Kc, None, K13, None, n_slots=n, page_size=page, k_scale=scale[0], slots=slots))
    assert bool((K13[4] == 3).all())
    rest = torch.arange(13, device="cuda") != 4
    assert same(K13[rest], K[slots[rest]])
    slots[2] = n
    qmm.kv_fp4_read(qmm.make_kv_fp4_read(Kc, None, K13, None, n_slots=n, page_size=page, slots=slots))
    assert qmm.device_status() == 4
    qmm.kv_fp4_read(qmm.make_kv_fp4_read(Kc, None, K13[:0], None, n_slots=n, page_size=page))


def test_other_stream_and_graph(qmm):
    c = Case(qmm, 8, 4, 2, 128, 128, False, F32, BF16, 16)
    want_k, want_v = c.want()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qmm.norm_rope_fp4(c.args(qmm), stream=side)
    side.synchronize()
    assert torch.equal(c.Kc, want_k) and torch.equal(c.Vc, want_v)
    args = c.args(qmm)
    values = torch.zeros(c.n_slots, 2, 128, dtype=BF16, device="cuda")
    read = qmm.make_kv_fp4_read(c.Kc, None, values, None, n_slots=c.n_slots, page_size=16, k_scale=c.scales[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmm.norm_rope_fp4(args)
        qmm.kv_fp4_read(read)
    c.pos += 17
    want_k, _ = c.want()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.Kc, want_k)
    live = c.slots[c.slots >= 0]
    want = fp4_plain.f32(fp4_plain.unpack(want_k, 2, 128, 16, c.scales[0])).float().to(BF16)
    assert torch.equal(values[live], want[live])


def test_cache_beyond_32_bit_offsets(qmm):
    Hk, D, page = 8, 128, 64
    n_slots = (5 << 30) // (Hk * D * 9 // 16) // page * page
    K, V = torch.randn(3, Hk, D, device="cuda"), torch.randn(3, Hk, D, device="cuda")
    Q = torch.randn(3, 1, D, device="cuda")
    Kc, Vc = (torch.zeros(qmm.kv_fp4_bytes(n_slots, Hk, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    slots = torch.tensor([n_slots - 1, n_slots // 2, 5], device="cuda")
    out = torch.empty(3, 1, D, dtype=BF16, device="cuda")
    qmm.norm_rope_fp4(qmm.make_norm_rope_fp4(Q, K, V, None, None, None, None, slots, out, Kc, Vc, n_slots=n_slots,
                                             page_size=page, k_scale=0.01, v_scale=0.01))
    Ko, Vo = (torch.empty(3, Hk, D, device="cuda") for _ in range(2))
    qmm.kv_fp4_read(qmm.make_kv_fp4_read(Kc, Vc, Ko, Vo, n_slots=n_slots, page_size=page, k_scale=0.01, v_scale=0.01,
                                         slots=slots))
    code, s = fp4_plain.quantise(V.double(), 0.01)
    scale = torch.tensor(fp4_plain.E4M3, dtype=torch.float64, device="cuda")[s].repeat_interleave(16, -1)
    grid = torch.tensor(fp4_plain.E2M1 + [-v for v in fp4_plain.E2M1], dtype=torch.float64, device="cuda")
    tensor_scale = torch.tensor(0.01).double().item()
    assert torch.equal(Vo, (grid[code] * scale * tensor_scale).float())
    assert qmm.device_status() == 0
