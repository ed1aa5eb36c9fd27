"""CPU tests of the 4-bit cache's and of sampling's entry points: what they refuse before any GPU work."""
import ctypes

import pytest

from bit_quantized_skinny_gb300 import build_lib
from test_layer_abi import ALIGN, BUFSIZE, NULL, SHAPE, TYPE, attn_args, norm_rope_args


@pytest.fixture(scope="module")
def qmm():
    build_lib.build()
    from bit_quantized_skinny_gb300 import qmm as q
    q.load()
    return q


def test_cache_bytes(qmm):
    assert qmm.kv_fp4_bytes(64, 8, 128) == 64 * 8 * 72 and qmm.kv_fp4_bytes(1, 1, 64) == 36 and qmm.kv_fp4_bytes(3, 2, 256) == 864
    for bad in ((0, 8, 128), (-1, 8, 128), (64, 0, 128), (64, 32768, 128), (64, 8, 96), (64, 8, 512), (1 << 40, 8, 128)):
        assert qmm.kv_fp4_bytes(*bad) == 0


def fp4_norm_rope(qmm, page_size=16, k_scale=1.0, v_scale=1.0, **change):
    a = qmm._NormRopeFp4Args(page_size=page_size, k_scale=k_scale, v_scale=v_scale)
    a.base = norm_rope_args(qmm, **change)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(page_size=8), SHAPE), (dict(page_size=48), SHAPE), (dict(page_size=8192), SHAPE), (dict(page_size=0), SHAPE),
    (dict(k_scale=0.0), SHAPE), (dict(v_scale=-1.0), SHAPE), (dict(k_scale=float("nan")), SHAPE), (dict(v_scale=float("inf")), SHAPE),
    (dict(k_scale=2.0 ** -61), SHAPE), (dict(n_slots=65), SHAPE), (dict(page_size=128), SHAPE), (dict(n_slots=0), SHAPE),
    (dict(T=-1), SHAPE), (dict(D=96), SHAPE), (dict(rot=8), SHAPE), (dict(in_type=3), TYPE), (dict(out_type=0), TYPE),
    (dict(Q=None), NULL), (dict(K=None), NULL), (dict(slots=None), NULL), (dict(V_cache=None), NULL), (dict(cos_sin=None), NULL),
    (dict(K_cache=24), ALIGN), (dict(Q=24), ALIGN), (dict(ldqo=516), ALIGN), (dict(positions=18), ALIGN),
])
def test_norm_rope_fp4_refusals(qmm, change, status):
    assert qmm.load().qmm_norm_rope_fp4(fp4_norm_rope(qmm, **change), None) == status


def test_norm_rope_fp4_without_rows(qmm):
    assert qmm.load().qmm_norm_rope_fp4(fp4_norm_rope(qmm, T=0), None) == 0
    assert qmm.load().qmm_norm_rope_fp4(None, None) == NULL


def read_args(qmm, **change):
    a = qmm._KvFp4ReadArgs(Hk=2, D=128, page_size=16, out_type=qmm.BF16, k_scale=1.0, v_scale=1.0, n_slots=64, K_cache=16,
                           V_cache=16, slots=16, n=5, K_out=16, V_out=16)
    for k, v in change.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(Hk=0), SHAPE), (dict(D=32), SHAPE), (dict(page_size=24), SHAPE), (dict(n_slots=0), SHAPE), (dict(n_slots=40), SHAPE),
    (dict(n=-1), SHAPE), (dict(n=65, slots=None), SHAPE), (dict(n=1 << 41), SHAPE), (dict(k_scale=0.0), SHAPE), (dict(out_type=5), TYPE),
    (dict(K_cache=None), NULL), (dict(K_out=None), NULL), (dict(V_cache=None), NULL), (dict(V_out=None), NULL),
    (dict(K_cache=8), ALIGN), (dict(K_out=8), ALIGN), (dict(V_out=4), ALIGN), (dict(slots=12), ALIGN),
])
def test_read_refusals(qmm, change, status):
    assert qmm.load().qmm_kv_fp4_read(read_args(qmm, **change), None) == status


def test_read_nothing(qmm):
    assert qmm.load().qmm_kv_fp4_read(read_args(qmm, n=0), None) == 0
    assert qmm.load().qmm_kv_fp4_read(None, None) == NULL


def fp4_attn(qmm, k_scale=1.0, v_scale=1.0, **change):
    a = qmm._AttnFp4Args(k_scale=k_scale, v_scale=v_scale)
    a.base = attn_args(qmm, **change)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(k_scale=0.0), SHAPE), (dict(v_scale=float("nan")), SHAPE), (dict(v_scale=2.0 ** 61), SHAPE), (dict(T=-1), SHAPE),
    (dict(T=65537), SHAPE), (dict(scale=0.0), SHAPE), (dict(B=1025), SHAPE), (dict(D=256), SHAPE), (dict(Hk=3), SHAPE),
    (dict(Hq=130, Hk=2, ldq=1 << 16, ldo=1 << 16), SHAPE), (dict(page_size=8), SHAPE), (dict(n_slots=100), SHAPE),
    (dict(prefix_len=-1), SHAPE), (dict(ldq=1279), SHAPE), (dict(type=0), TYPE), (dict(Q=None), NULL), (dict(O=None), NULL),
    (dict(K_cache=None), NULL), (dict(row_starts=None), NULL), (dict(prefix_pages=None), NULL), (dict(pages=None), NULL),
    (dict(kv_lens=None), NULL), (dict(Q=24), ALIGN), (dict(V_cache=8), ALIGN), (dict(lse=18), ALIGN),
])
def test_attn_fp4_refusals(qmm, change, status):
    lib, a = qmm.load(), fp4_attn(qmm, **change)
    assert lib.qmm_attn_shared_fp4(a, 16, 1 << 40, None) == status
    if status in (SHAPE, TYPE):
        assert lib.qmm_attn_fp4_workspace_bytes(a) == 0


def test_attn_fp4_workspace(qmm):
    lib = qmm.load()
    need = lib.qmm_attn_fp4_workspace_bytes(fp4_attn(qmm))
    assert need > 0
    assert lib.qmm_attn_shared_fp4(fp4_attn(qmm), None, need, None) == NULL
    assert lib.qmm_attn_shared_fp4(fp4_attn(qmm), 16, need - 1, None) == BUFSIZE
    assert lib.qmm_attn_shared_fp4(fp4_attn(qmm), 24, need, None) == ALIGN
    assert lib.qmm_attn_shared_fp4(None, 16, need, None) == NULL
    assert lib.qmm_attn_shared_fp4(fp4_attn(qmm, T=0), None, 0, None) == 0


def sample_args(qmm, **change):
    a = qmm._SampleArgs(T=4, V=100, type=qmm.F32, logits=16, ld=100, temperature=16, top_k=16, top_p=16, min_p=16, uniform=16,
                        tokens=16, logprobs=16, B=2, row_starts=16, fed=16, accepted=16, next=16)
    for k, v in change.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), SHAPE), (dict(T=65536), SHAPE), (dict(V=0), SHAPE), (dict(V=393217), SHAPE), (dict(ld=99), SHAPE), (dict(B=-1), SHAPE),
    (dict(B=1025), SHAPE), (dict(type=3), TYPE), (dict(logits=None), NULL), (dict(uniform=None), NULL), (dict(tokens=None), NULL),
    (dict(row_starts=None), NULL), (dict(fed=None), NULL), (dict(accepted=None), NULL), (dict(next=None), NULL),
    (dict(logits=18), ALIGN), (dict(logits=17, type=1), ALIGN), (dict(temperature=18), ALIGN), (dict(top_k=18), ALIGN),
    (dict(top_p=18), ALIGN), (dict(min_p=18), ALIGN), (dict(uniform=18), ALIGN), (dict(tokens=18), ALIGN), (dict(logprobs=18), ALIGN),
    (dict(row_starts=18), ALIGN), (dict(fed=18), ALIGN), (dict(accepted=18), ALIGN), (dict(next=18), ALIGN),
])
def test_sample_refusals(qmm, change, status):
    assert qmm.load().qmm_sample(sample_args(qmm, **change), None) == status


def test_sample_without_rows(qmm):
    assert qmm.load().qmm_sample(sample_args(qmm, T=0, B=0), None) == 0
    assert qmm.load().qmm_sample(None, None) == NULL


def test_python_checks(qmm):
    import torch
    f32, i32, u8 = torch.float32, torch.int32, torch.uint8
    Q, K = torch.zeros(2, 4, 128), torch.zeros(2, 2, 128)
    cache, short = torch.zeros(16 * 2 * 72, dtype=u8), torch.zeros(16 * 2 * 72 - 1, dtype=u8)
    out, slots = torch.zeros(2, 4, 128, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int64)
    make = lambda kc, vc, **k: qmm.make_norm_rope_fp4(Q, K, K, None, None, None, None, slots, out, kc, vc, n_slots=16, page_size=16, **k)
    for kc, vc, status in ((short, cache, BUFSIZE), (cache, None, NULL), (None, cache, NULL), (cache.view(torch.int8), cache, TYPE),
                           (cache, cache, SHAPE)):     # the last: not on a CUDA device
        with pytest.raises(qmm.QmmError) as e:
            make(kc, vc)
        assert e.value.status == status
    values = torch.zeros(4, 2, 128)
    read = lambda *a, **k: qmm.make_kv_fp4_read(*a, n_slots=16, page_size=16, **k)
    for a, k, status in (((cache, None, values, values), {}, NULL), ((cache, cache, values, values[:2]), {}, SHAPE),
                         ((short, cache, values, values), {}, BUFSIZE), ((cache, cache, values, values.half()), {}, TYPE),
                         ((cache, cache, values, values), dict(slots=slots), SHAPE), ((cache, cache, values.int(), values), {}, TYPE)):
        with pytest.raises(qmm.QmmError) as e:
            read(*a, **k)
        assert e.value.status == status
    ints = lambda *s: torch.zeros(*s, dtype=i32)
    q16 = Q.bfloat16()
    attn = lambda **k: qmm.make_attn_fp4(**{**dict(Q=q16, K_cache=cache, V_cache=cache, Hk=2, page_size=16, prefix_pages=ints(1),
                                                   prefix_len=9, pages=ints(1, 1), kv_lens=ints(1), row_starts=ints(2), O=q16,
                                                   scale=0.1), **k})
    for k, status in ((dict(K_cache=None), NULL), (dict(V_cache=short), SHAPE), (dict(K_cache=short, V_cache=short), BUFSIZE),
                      (dict(page_size=0), SHAPE), (dict(prefix_len=17), SHAPE), (dict(O=Q), TYPE), (dict(kv_lens=ints(2)), SHAPE),
                      (dict(K_cache=cache.view(torch.int8)), TYPE), (dict(lse=torch.zeros(2, 3)), SHAPE), ({}, SHAPE)):
        with pytest.raises(qmm.QmmError) as e:
            attn(**k)
        assert e.value.status == status, k
    x, u, tokens = torch.zeros(3, 50), torch.zeros(3), ints(3)
    sample = lambda **k: qmm.make_sample(**{**dict(logits=x, uniform=u, tokens=tokens), **k})
    drafts = dict(fed=ints(3), row_starts=ints(3), accepted=ints(2), next=ints(2))
    for k, status in ((dict(uniform=None), NULL), (dict(logits=x.int()), TYPE), (dict(logits=x[0]), SHAPE), (dict(logits=x.t()), SHAPE),
                      (dict(uniform=u[:2]), SHAPE), (dict(uniform=u.double()), TYPE), (dict(tokens=tokens.long()), TYPE),
                      (dict(top_k=u), TYPE), (dict(top_p=torch.zeros(6)[::2]), SHAPE), (dict(logprobs=u[:1]), SHAPE),
                      (dict(fed=ints(3)), NULL), ({**drafts, "fed": ints(2)}, SHAPE), ({**drafts, "next": ints(3)}, SHAPE),
                      ({**drafts, "row_starts": ints(2)}, SHAPE), ({**drafts, "accepted": u[:2]}, TYPE), (drafts, SHAPE), ({}, SHAPE)):
        with pytest.raises(qmm.QmmError) as e:
            sample(**k)
        assert e.value.status == status, k
