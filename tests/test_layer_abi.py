"""CPU tests of the attention half's entry points: what they refuse before any GPU work."""
import ctypes

import pytest

from bit_quantized_skinny_gb300 import build_lib

NULL, SHAPE, M_RANGE, ALIGN, BUFSIZE, COUNT, TYPE = 1, 2, 3, 4, 5, 8, 12


@pytest.fixture(scope="module")
def qmm():
    build_lib.build()
    from bit_quantized_skinny_gb300 import qmm as q
    q.load()
    return q


def norm_rope_args(qmm, **change):
    # addresses are never dereferenced: every call below fails its checks first
    a = qmm._NormRopeArgs(T=4, Hq=4, Hk=2, D=128, rot=128, interleaved=0, in_type=qmm.F32, out_type=qmm.BF16, eps=1e-6,
                          Q=16, K=16, V=16, ldq=512, ldk=256, ldv=256, q_weight=16, k_weight=16, cos_sin=16, max_pos=8,
                          positions=16, slots=16, Q_out=16, ldqo=512, K_cache=16, V_cache=16, n_slots=64)
    for k, v in change.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), SHAPE), (dict(Hq=0), SHAPE), (dict(Hk=-1), SHAPE), (dict(D=96), SHAPE), (dict(rot=8), SHAPE),
    (dict(rot=144), SHAPE), (dict(in_type=3), TYPE), (dict(out_type=0), TYPE), (dict(Q=None), NULL),
    (dict(K=None), NULL), (dict(slots=None), NULL), (dict(V_cache=None), NULL), (dict(cos_sin=None), NULL),
    (dict(positions=None), NULL), (dict(max_pos=0), SHAPE), (dict(ldq=511), SHAPE), (dict(ldv=255), SHAPE),
    (dict(n_slots=0), SHAPE), (dict(Q=24), ALIGN), (dict(ldk=257), ALIGN), (dict(Q_out=8), ALIGN),
    (dict(ldqo=516), ALIGN), (dict(q_weight=20), ALIGN), (dict(slots=12), ALIGN), (dict(positions=18), ALIGN),
])
def test_norm_rope_refusals(qmm, change, status):
    assert qmm.load().qmm_norm_rope(norm_rope_args(qmm, **change), None) == status


def test_norm_rope_without_rows(qmm):
    assert qmm.load().qmm_norm_rope(norm_rope_args(qmm, T=0), None) == 0
    assert qmm.load().qmm_norm_rope(None, None) == NULL


def attn_args(qmm, **change):
    a = qmm._AttnArgs(T=8, B=2, Hq=10, Hk=2, D=128, page_size=64, type=qmm.BF16, scale=0.1, Q=16, ldq=1280, K_cache=16,
                      V_cache=16, n_slots=640, prefix_pages=16, prefix_len=100, pages=16, pages_per_stream=4,
                      kv_lens=16, row_starts=16, O=16, ldo=1280, lse=16)
    for k, v in change.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), SHAPE), (dict(T=65537), SHAPE), (dict(scale=0.0), SHAPE), (dict(scale=float('nan')), SHAPE), (dict(scale=float('inf')), SHAPE), (dict(B=-1), SHAPE), (dict(B=1025), SHAPE), (dict(D=256), SHAPE),
    (dict(Hk=0), SHAPE), (dict(Hk=3), SHAPE), (dict(Hq=130, Hk=2, ldq=1 << 16, ldo=1 << 16), SHAPE),
    (dict(page_size=8), SHAPE), (dict(page_size=48, n_slots=480), SHAPE), (dict(page_size=8192, n_slots=8192), SHAPE),
    (dict(n_slots=100), SHAPE), (dict(n_slots=1 << 31), SHAPE), (dict(prefix_len=-1), SHAPE),
    (dict(prefix_len=1 << 30), SHAPE), (dict(pages_per_stream=1 << 24), SHAPE), (dict(ldq=1279), SHAPE),
    (dict(ldo=1272), SHAPE), (dict(type=0), TYPE), (dict(type=7), TYPE), (dict(Q=None), NULL), (dict(O=None), NULL),
    (dict(K_cache=None), NULL), (dict(row_starts=None), NULL), (dict(prefix_pages=None), NULL), (dict(pages=None), NULL),
    (dict(kv_lens=None), NULL), (dict(Q=24), ALIGN), (dict(ldq=1281), ALIGN), (dict(V_cache=8), ALIGN),
    (dict(lse=18), ALIGN), (dict(pages=18), ALIGN),
])
def test_attn_refusals(qmm, change, status):
    lib, a = qmm.load(), attn_args(qmm, **change)
    assert lib.qmm_attn_shared(a, 16, 1 << 40, None) == status
    if status in (SHAPE, TYPE):
        assert lib.qmm_attn_workspace_bytes(a) == 0


def test_attn_workspace(qmm):
    lib = qmm.load()
    need = lib.qmm_attn_workspace_bytes(attn_args(qmm))
    assert need > 0
    assert lib.qmm_attn_shared(attn_args(qmm), None, need, None) == NULL
    assert lib.qmm_attn_shared(attn_args(qmm), 16, need - 1, None) == BUFSIZE
    assert lib.qmm_attn_shared(attn_args(qmm), 24, need, None) == ALIGN
    assert lib.qmm_attn_shared(None, 16, need, None) == NULL
    assert lib.qmm_attn_shared(attn_args(qmm, T=0), None, 0, None) == 0


def lora_entries(qmm, **change):
    e = (qmm._LoraEntry * 2)()
    for k in range(2):
        e[k] = qmm._LoraEntry(16, 3, 16, 16, 16, 100, 512)
    for k, v in change.items():
        setattr(e[1], k, v)
    return e


@pytest.mark.parametrize("change,status", [
    (dict(adapters=None), NULL), (dict(X=None), NULL), (dict(Y0=None), NULL), (dict(Y=None), NULL), (dict(K=500), SHAPE),
    (dict(N=0), SHAPE), (dict(n_adapters=0), SHAPE), (dict(X=24), ALIGN), (dict(Y=18), ALIGN), (dict(adapters=20), ALIGN),
])
def test_lora_refusals(qmm, change, status):
    assert qmm.load().qmm_run_lora(lora_entries(qmm, **change), 2, 16, 4, 8, 16, 1 << 30, None) == status


def test_lora_refusals_of_the_call(qmm):
    lib, e = qmm.load(), lora_entries(qmm)
    need = lib.qmm_lora_workspace_bytes(e, 2, 4, 8)
    assert need > 0
    assert lib.qmm_run_lora(None, 2, 16, 4, 8, 16, need, None) == NULL
    assert lib.qmm_run_lora(e, 2, None, 4, 8, 16, need, None) == NULL
    assert lib.qmm_run_lora(e, 2, 16, 4, 8, None, need, None) == NULL
    assert lib.qmm_run_lora(e, 0, 16, 4, 8, 16, need, None) == COUNT
    assert lib.qmm_run_lora(e, 17, 16, 4, 8, 16, need, None) == COUNT
    assert lib.qmm_run_lora(e, 2, 16, 0, 8, 16, need, None) == M_RANGE
    assert lib.qmm_run_lora(e, 2, 16, 33, 8, 16, need, None) == M_RANGE
    assert lib.qmm_run_lora(e, 2, 16, 4, 0, 16, need, None) == SHAPE
    assert lib.qmm_run_lora(e, 2, 16, 4, 257, 16, need, None) == SHAPE
    assert lib.qmm_run_lora(e, 2, 16, 4, 8, 16, need - 1, None) == BUFSIZE
    assert lib.qmm_run_lora(e, 2, 18, 4, 8, 16, need, None) == ALIGN
    assert lib.qmm_lora_workspace_bytes(e, 0, 4, 8) == 0 and lib.qmm_lora_workspace_bytes(e, 2, 4, 300) == 0


def test_python_checks(qmm):
    import torch
    Q, out = torch.zeros(2, 4, 64), torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    for bad in (dict(Q=Q.double()), dict(Q_out=out[:1]), dict(Q=Q.transpose(1, 2)), dict(q_weight=torch.zeros(63)),
                dict(q_weight=torch.zeros(64).half())):
        kw = dict(Q=Q, K=None, V=None, q_weight=None, k_weight=None, cos_sin=None, positions=None, slots=None, Q_out=out,
                  K_cache=None, V_cache=None)
        with pytest.raises(qmm.QmmError):
            qmm.make_norm_rope(**dict(kw, **bad))
    K = torch.zeros(64, 2, 64, dtype=torch.bfloat16)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)
    kw = dict(Q=out, K_cache=K, V_cache=K, page_size=16, prefix_pages=i32(0), prefix_len=10, pages=i32(1)[None],
              kv_lens=i32(3), row_starts=i32(0, 2), O=out.clone(), scale=0.1)
    qmm.make_attn(**kw)
    for bad in (dict(V_cache=K[:32]), dict(row_starts=i32(0)), dict(kv_lens=torch.zeros(1)), dict(prefix_len=17),
                dict(O=Q), dict(K_cache=K.half()), dict(lse=torch.zeros(2, 3))):
        with pytest.raises(qmm.QmmError):
            qmm.make_attn(**dict(kw, **bad))


def test_python_checks_of_adapters(qmm):
    """What the adapters' calls read through raw pointers has the type, shape and layout that they take."""
    import torch
    bf16 = torch.bfloat16
    A, Bt = torch.zeros(8, 512, dtype=bf16), torch.zeros(8, 40, dtype=bf16)
    table = qmm.make_lora_adapters([(A, Bt, 1.0), (A[:3], Bt[:3], 0.5)])
    assert table.numel() == 2 * ctypes.sizeof(qmm._LoraAdapter)
    for bad in ([], [(A[:4], Bt, 1.0)], [(A.float(), Bt, 1.0)], [(A, Bt.half(), 1.0)], [(A[:, ::2], Bt, 1.0)],
                [(A, Bt.T.contiguous().T, 1.0)], [(A, Bt, 1.0), (A, torch.zeros(8, 48, dtype=bf16), 1.0)],
                [(A, Bt, 1.0), (torch.zeros(8, 256, dtype=bf16), Bt, 1.0)], [(A[0], Bt[0], 1.0)]):
        with pytest.raises(qmm.QmmError):
            qmm.make_lora_adapters(bad)
    X, Y = torch.zeros(4, 512, dtype=bf16), torch.zeros(4, 40)
    good = dict(adapters=table, X=X, Y0=Y, Y=Y, N=40, K=512)
    entries = qmm.make_lora_entries([tuple(good.values())])
    for bad in (dict(X=X.float()), dict(X=X[:, :256]), dict(X=torch.zeros(512, 4, dtype=bf16).T), dict(Y0=Y.half()),
                dict(Y=Y[:3]), dict(Y=torch.zeros(4, 41)), dict(Y0=torch.zeros(40, 4).T), dict(N=48), dict(K=256),
                dict(adapters=table.view(torch.int64)), dict(X=X[0])):
        with pytest.raises(qmm.QmmError):
            qmm.make_lora_entries([tuple(dict(good, **bad).values())])
    # an adapter's widths are those of its projection, also where X and Y fit another one
    with pytest.raises(qmm.QmmError):
        qmm.make_lora_entries([(table, X[:, :256].contiguous(), Y, Y, 40, 256)])
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    i32 = torch.zeros(4, dtype=torch.int32)
    for bad in (dict(ids=i32.long()), dict(ids=i32[:3]), dict(ids=torch.zeros(8, dtype=torch.int32)[::2]),
                dict(ids=torch.zeros(5, dtype=torch.int32), M=5)):
        kw = dict(dict(ids=i32, M=4), **bad)
        with pytest.raises(qmm.QmmError):
            qmm.run_lora(entries, kw["ids"], kw["M"], 8, ws, stream=0)


def test_python_checks_of_missing_tensors(qmm):
    import torch
    bf16, i32 = torch.bfloat16, lambda *v: torch.tensor(v, dtype=torch.int32)
    Q, K, out, cache = torch.zeros(2, 4, 64), torch.zeros(2, 1, 64), torch.zeros(2, 4, 64, dtype=bf16), torch.zeros(16, 1, 64, dtype=bf16)
    kw = dict(Q=Q, K=K, V=K, q_weight=None, k_weight=None, cos_sin=None, positions=None, slots=torch.arange(2), Q_out=out,
              K_cache=cache, V_cache=cache.clone())
    qmm.make_norm_rope(**kw)
    for name in ("K_cache", "V_cache"):
        with pytest.raises(qmm.QmmError):
            qmm.make_norm_rope(**dict(kw, **{name: None}))
    kw = dict(Q=out, K_cache=cache, V_cache=cache, page_size=16, prefix_pages=None, prefix_len=0, pages=i32(0)[None],
              kv_lens=i32(3), row_starts=i32(0, 2), O=out.clone(), scale=0.1)
    qmm.make_attn(**kw)
    for name in ("K_cache", "V_cache", "pages", "kv_lens", "row_starts", "O"):
        with pytest.raises(qmm.QmmError):
            qmm.make_attn(**dict(kw, **{name: None}))
