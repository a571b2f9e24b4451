"""The paged cache's entry points on the host: bad arguments are rejected
synchronously, before any GPU is touched; and the plain forms the GPU tests
compare with agree with each other on small cases."""
import math

import pytest
import torch

import sequence_depth_attention_gb300 as moda
from sequence_depth_attention_gb300 import binding
from sequence_depth_attention_gb300 import build as mbuild

import paged_common as pc

OK, INVALID, UNSUPPORTED, MISALIGNED, CUDA, TIMEOUT, NO_DEVICE = range(7)
# fake device addresses far apart: validation must not dereference anything
Q, K, V, ROPE, SEQ, POS, QO, KO, PK, PV, KS, VS, TAB, LENS, KD, VD, O, LSE, WS = (
    (i + 1) << 32 for i in range(19))


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return binding.load()


def cache(fmt=0, num_pages=8, page_size=16, Hk=2, d=64, B=3, max_pages=4, pk=PK, pv=PV, pks=None,
          pvs=None, table=TAB):
    return binding._PagedKv(fmt, num_pages, page_size, Hk, d, B, max_pages, pk, pv, pks, pvs, table)


BAD_CACHES = [
    (dict(fmt=2), INVALID), (dict(fmt=-1), INVALID), (dict(B=-1), INVALID),
    (dict(num_pages=0), INVALID), (dict(max_pages=0), INVALID), (dict(Hk=0), INVALID),
    (dict(pk=None), INVALID), (dict(pv=None), INVALID), (dict(table=None), INVALID),
    (dict(pks=KS, pvs=VS), INVALID), (dict(fmt=1), INVALID), (dict(fmt=1, pks=KS), INVALID),
    (dict(page_size=0), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED),
    (dict(page_size=256), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(d=0), UNSUPPORTED),
    (dict(num_pages=1 << 27), UNSUPPORTED), (dict(max_pages=1 << 27), UNSUPPORTED),
    (dict(pk=PK + 8), MISALIGNED), (dict(table=TAB + 2), MISALIGNED),
    (dict(fmt=1, pks=KS + 4, pvs=VS), MISALIGNED),
]


def append(lib, c=None, q=Q, k=K, v=V, qs=8 * 64, ks=8 * 64, vs=8 * 64, rope=ROPE, rows=64, rot=64,
           inter=0, seq=SEQ, pos=POS, N=5, Hq=4, qo=QO, ko=KO, **kw):
    return lib.moda_kv_append(q, k, v, qs, ks, vs, rope, rows, rot, inter, seq, pos, N, Hq,
                              cache(**kw) if c is None else c, qo, ko, None)


@pytest.mark.parametrize("kw,code", BAD_CACHES + [
    (dict(N=-1), INVALID), (dict(Hq=-1), INVALID), (dict(N=(1 << 24) + 1), UNSUPPORTED),
    (dict(Hq=5000), UNSUPPORTED), (dict(rot=-16), INVALID), (dict(rot=24), UNSUPPORTED),
    (dict(rot=80), UNSUPPORTED), (dict(rope=None), INVALID), (dict(rows=0), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(seq=None), INVALID), (dict(pos=None), INVALID), (dict(qo=None), INVALID),
    (dict(qs=4 * 64 - 8), INVALID), (dict(qs=4 * 64 + 4), INVALID), (dict(ks=64), INVALID),
    (dict(vs=129), INVALID), (dict(ks=1 << 40), UNSUPPORTED),
    (dict(q=Q + 2), MISALIGNED), (dict(rope=ROPE + 8), MISALIGNED), (dict(seq=SEQ + 1), MISALIGNED),
    (dict(ko=KO + 4), MISALIGNED),
    (dict(qo=Q), INVALID), (dict(ko=K + 64), INVALID), (dict(qo=KO), INVALID), (dict(k=PK), INVALID),
    (dict(ko=PV + 16), INVALID), (dict(table=PK), INVALID), (dict(seq=PV + 64), INVALID),
    (dict(v=PK), INVALID), (dict(v=PK - 512), INVALID),
])
def test_append_rejects(lib, kw, code):
    assert append(lib, **kw) == code
    assert lib.moda_last_error_detail().decode() != ""


def test_append_without_tokens_or_queries(lib):
    assert append(lib, N=0, k=None, v=None, seq=None) == OK
    # no queries, no rotation, no k_out, strides of a single token unused
    rc = append(lib, q=None, qo=None, Hq=0, ko=None, rope=None, rows=0, rot=0, N=1, ks=3, vs=5)
    assert rc in (OK, NO_DEVICE) if not torch.cuda.is_available() else True


def test_null_cache(lib):
    assert lib.moda_kv_append(Q, K, V, 512, 512, 512, ROPE, 64, 64, 0, SEQ, POS, 5, 4, None, QO, KO,
                              None) == INVALID
    assert lib.moda_kv_gather(None, SEQ, POS, 5, K, V, None) == INVALID
    assert lib.moda_decode_paged(Q, None, LENS, KD, VD, 512, 256, 64, 4, 4, 0.1, O, LSE, WS, 1 << 30,
                                 None) == INVALID


def gather(lib, seq=SEQ, pos=POS, N=5, k=K, v=V, **kw):
    return lib.moda_kv_gather(cache(**kw), seq, pos, N, k, v, None)


@pytest.mark.parametrize("kw,code", BAD_CACHES + [
    (dict(N=-1), INVALID), (dict(N=(1 << 24) + 1), UNSUPPORTED), (dict(seq=None), INVALID),
    (dict(pos=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(k=K + 8), MISALIGNED), (dict(pos=POS + 2), MISALIGNED), (dict(k=V), INVALID),
    (dict(k=PK + 32), INVALID), (dict(v=TAB), INVALID), (dict(k=SEQ), INVALID),
])
def test_gather_rejects(lib, kw, code):
    assert gather(lib, **kw) == code
    assert lib.moda_last_error_detail().decode() != ""


def test_gather_of_nothing(lib):
    assert gather(lib, N=0, k=None, v=None) == OK


def decode(lib, q=Q, lens=LENS, kd=KD, vd=VD, sb=2 * 4 * 64, sh=4 * 64, sl=64, Hq=4, L=4, scale=0.125,
           o=O, lse=LSE, ws=WS, wsb=None, **kw):
    c = cache(**kw)
    if wsb is None:
        wsb = lib.moda_decode_paged_workspace_bytes(4, 2, 64)
    return lib.moda_decode_paged(q, c, lens, kd, vd, sb, sh, sl, Hq, L, scale, o, lse, ws, wsb, None)


@pytest.mark.parametrize("kw,code", BAD_CACHES + [
    (dict(Hq=0), INVALID), (dict(Hq=5), INVALID), (dict(Hq=34), UNSUPPORTED), (dict(L=-1), INVALID),
    (dict(L=1025), UNSUPPORTED), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(B=1 << 23), UNSUPPORTED), (dict(q=None), INVALID), (dict(lens=None), INVALID),
    (dict(o=None), INVALID), (dict(ws=None), INVALID), (dict(kd=None), INVALID), (dict(vd=None), INVALID),
    (dict(sl=56), INVALID), (dict(sh=60), INVALID), (dict(sb=0), INVALID), (dict(sb=1 << 38), INVALID),
    (dict(wsb=0), INVALID), (dict(q=Q + 2), MISALIGNED), (dict(kd=KD + 8), MISALIGNED),
    (dict(ws=WS + 4), MISALIGNED), (dict(lens=LENS + 2), MISALIGNED), (dict(lse=LSE + 2), MISALIGNED),
    (dict(o=Q), INVALID), (dict(lse=O + 64), INVALID), (dict(ws=PK), INVALID), (dict(o=KD + 128), INVALID),
    (dict(o=LENS), INVALID), (dict(lse=TAB), INVALID),
])
def test_decode_rejects(lib, kw, code):
    assert decode(lib, **kw) == code
    assert lib.moda_last_error_detail().decode() != ""


def test_decode_empty_batch(lib):
    assert decode(lib, B=0, table=None, q=None, o=None, lens=None) == OK


def test_decode_workspace(lib):
    w = lib.moda_decode_paged_workspace_bytes
    assert w(16, 4, 128) > 0
    assert w(4, 4, 64) <= w(64, 4, 64) <= w(64, 4, 128)
    for bad in ((0, 4, 128), (6, 4, 128), (17 * 4, 4, 128), (4, 0, 128), (4, 4, 96)):
        assert w(*bad) == 0


def test_binding_refuses_mismatched_tensors():
    c = pc.Cache("bf16", [5], 2, 64, 16)
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):  # CPU tensors
        moda.moda_kv_append(None, x, x, *c.args(), i, i)
    with pytest.raises(TypeError):
        moda.moda_kv_gather([1], c.v, c.table, i, i)
    with pytest.raises(ValueError):
        moda.moda_decode_paged(x, *c.args(), i, 0.1)


# ------------------------------------------------- the plain forms themselves
def test_quantised_values_by_hand():
    x = torch.zeros(1, 32, dtype=torch.float64)
    x[0, :16] = torch.tensor([7.0, -7.0, 6.1, 5.0, 5.1, 3.5, 2.5, 2.6, 1.75, 1.25, 0.75, 0.25, 0.26, -0.25,
                              -0.74, 1.3])
    want = torch.tensor([6.0, -6, 6, 4, 6, 4, 2, 3, 2, 1, 1, 0, 0.5, 0, -0.5, 1.5])
    assert torch.equal(pc.mx4_quantised(x)[0, :16], want.double())
    assert torch.equal(pc.mx4_quantised(x * 2 ** -9), pc.mx4_quantised(x) * 2 ** -9)
    x[0, 0] = 7.001  # one scale up: 7.001 / 2 -> 4 halves
    assert pc.mx4_quantised(x)[0, 0] == 8.0 and pc.mx4_quantised(x)[0, 3] == 4.0
    assert pc.mx4_quantised(x)[0, 11] == 0.0
    x[0, 0] = math.inf
    assert pc.mx4_quantised(x).isnan().all()


def test_turned_is_a_rotation():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(4, 3, 64, generator=g, dtype=torch.float64)
    pos = torch.tensor([0, 1, 7, 30])
    for inter in (False, True):
        y = pc.turned(x, pc.rope_table(31, 32), pos, inter)
        assert torch.equal(y[0], x[0]) and torch.equal(y[..., 32:], x[..., 32:])
        assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1), rtol=1e-6)
    # complex form, half-split pairs
    rope = pc.rope_table(31, 64)[pos].double()
    z = torch.complex(x[..., :32], x[..., 32:]) * torch.complex(rope[:, :32], rope[:, 32:])[:, None]
    y = pc.turned(x, pc.rope_table(31, 64), pos, False)
    assert torch.allclose(y[..., :32], z.real) and torch.allclose(y[..., 32:], z.imag)


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
def test_decode_reference_against_one_softmax(fmt):
    lens = [0, 1, 19, 33]
    c = pc.Cache(fmt, lens, 2, 64, 16, seed=3)
    g = torch.Generator().manual_seed(4)
    q = torch.randn(4, 6, 64, generator=g).bfloat16()
    kd, vd = (torch.randn(4, 2, 5, 64, generator=g).bfloat16() for _ in range(2))
    o, lse, _, _ = pc.decode_reference(c, q, lens, kd, vd, 0.125)
    for b, n in enumerate(lens):
        for h in range(6):
            k = torch.cat((c.rows("k", b, n)[h // 3], kd[b, h // 3].double()))
            v = torch.cat((c.rows("v", b, n)[h // 3], vd[b, h // 3].double()))
            w = torch.softmax(k @ q[b, h].double() * 0.125, 0)
            assert torch.allclose(w @ v, o[b, h])
            assert abs(torch.log(torch.exp(k @ q[b, h].double() * 0.125).sum()) - lse[b, h]) < 1e-12


def test_append_rejects_too_many_rows(lib):
    # N * (Hq + 2 Hk) rows beyond 2^31 - 1
    assert append(lib, N=1 << 24, Hq=256, qs=256 * 64, ks=1 << 20, vs=1 << 20, Hk=2) == UNSUPPORTED


@pytest.mark.parametrize("call", [append, gather, decode])
def test_more_kv_heads_than_supported(lib, call):
    assert call(lib, Hk=4097, num_pages=1) == UNSUPPORTED
    assert "4097" in lib.moda_last_error_detail().decode()


def test_decode_rejects_a_scale_whose_log2_form_overflows(lib):
    assert decode(lib, scale=2.4e38) == INVALID
