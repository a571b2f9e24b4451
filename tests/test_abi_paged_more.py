"""Chunks of new tokens and selected pages on the host: bad arguments are refused
synchronously, before any GPU is touched; the extension and the Python code behind it pass
on the same arguments; and the plain forms that the GPU tests compare with agree with each
other on small cases."""
import ctypes
import itertools
import math

import pytest
import torch

import sequence_depth_attention_gb300 as moda
from sequence_depth_attention_gb300 import binding

import paged_chunk_common as cc
import paged_common as pc
import test_abi_paged as host
from test_abi_paged import (BAD_CACHES, INVALID, KD, LENS, LSE, MISALIGNED, NO_DEVICE, O, OK, PK, POS, PV, Q, SEQ, TAB,
                            UNSUPPORTED, VD, WS, cache, lib)  # noqa: F401 (lib is a fixture)
from test_abi_paged_args import (D, HK, HQ, L, N, PAGE, PAGES, B, STREAM, WORKSPACE, bad, bf, c_type, f32, i32,
                                 ways)  # noqa: F401 (ways is a fixture)
from test_abi_paged_args import cache as tensors

STARTS, MEANS, PAGES_AT, ROWS = ((i + 40) << 32 for i in range(4))


def prefill(lib, q=Q, qs=4 * 64, starts=STARTS, lens=LENS, kd=KD, vd=VD, sl=5 * 2 * 64, st=2 * 64, sh=64, N=5, Hq=4,
            L=4, scale=0.125, o=O, lse=LSE, ws=WS, wsb=None, **kw):
    if wsb is None:
        wsb = lib.moda_prefill_paged_workspace_bytes(4, 2, 64)
    return lib.moda_prefill_paged(q, qs, cache(**kw), starts, lens, kd, vd, sl, st, sh, N, Hq, L, scale, o, lse, ws,
                                  wsb, None)


def means(lib, seq=SEQ, pos=POS, N=5, m=MEANS, **kw):
    return lib.moda_page_means(cache(**kw), seq, pos, N, m, None)


def select(lib, q=Q, m=MEANS, seq=SEQ, pos=POS, N=5, Hq=4, S=3, sink=1, recent=1, pages=PAGES_AT, rows=ROWS, **kw):
    return lib.moda_select_pages(q, m, cache(**kw), seq, pos, N, Hq, S, sink, recent, pages, rows, None)


def selected(lib, q=Q, pages=PAGES_AT, rows=ROWS, N=5, S=3, kd=KD, vd=VD, st=2 * 4 * 64, sh=4 * 64, sl=64, Hq=4, L=4,
             scale=0.125, o=O, lse=LSE, ws=WS, wsb=None, **kw):
    if wsb is None:
        wsb = lib.moda_decode_paged_workspace_bytes(4, 2, 64)
    return lib.moda_decode_selected(q, cache(**kw), pages, rows, N, S, kd, vd, st, sh, sl, Hq, L, scale, o, lse, ws, wsb,
                                    None)


@pytest.mark.parametrize("kw,code", BAD_CACHES + [
    (dict(N=-1), INVALID), (dict(N=(1 << 24) + 1), UNSUPPORTED), (dict(Hq=0), INVALID), (dict(Hq=5), INVALID),
    (dict(Hq=34), UNSUPPORTED), (dict(L=-1), INVALID), (dict(L=1025), UNSUPPORTED), (dict(scale=0.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=2.4e38), INVALID),
    (dict(N=1 << 24, Hk=64, Hq=512, qs=1 << 20), UNSUPPORTED), (dict(Hk=4097, num_pages=1), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(starts=None), INVALID), (dict(lens=None), INVALID), (dict(o=None), INVALID),
    (dict(ws=None), INVALID), (dict(kd=None), INVALID), (dict(vd=None), INVALID),
    (dict(qs=4 * 64 - 8), INVALID), (dict(qs=4 * 64 + 4), INVALID), (dict(qs=1 << 38), INVALID),
    (dict(sl=56), INVALID), (dict(sh=60), INVALID), (dict(st=0), INVALID), (dict(st=-128), INVALID),
    (dict(sl=1 << 38), INVALID), (dict(wsb=0), INVALID),
    (dict(q=Q + 2), MISALIGNED), (dict(kd=KD + 8), MISALIGNED), (dict(ws=WS + 4), MISALIGNED),
    (dict(starts=STARTS + 2), MISALIGNED), (dict(lens=LENS + 2), MISALIGNED), (dict(lse=LSE + 2), MISALIGNED),
    (dict(o=Q), INVALID), (dict(lse=O + 64), INVALID), (dict(ws=PK), INVALID), (dict(o=KD + 128), INVALID),
    (dict(o=LENS), INVALID), (dict(lse=TAB), INVALID), (dict(o=STARTS), INVALID), (dict(o=VD - 64), INVALID),
])
def test_prefill_rejects(lib, kw, code):  # noqa: F811
    assert prefill(lib, **kw) == code
    assert lib.moda_last_error_detail().decode() != ""


@pytest.mark.parametrize("kw,code", BAD_CACHES + [
    (dict(N=-1), INVALID), (dict(N=(1 << 24) + 1), UNSUPPORTED), (dict(seq=None), INVALID), (dict(pos=None), INVALID),
    (dict(m=None), INVALID), (dict(m=MEANS + 8), MISALIGNED), (dict(pos=POS + 2), MISALIGNED),
    (dict(m=PK + 32), INVALID), (dict(m=TAB), INVALID), (dict(m=SEQ), INVALID), (dict(m=PV), INVALID),
])
def test_means_rejects(lib, kw, code):  # noqa: F811
    assert means(lib, **kw) == code
    assert lib.moda_last_error_detail().decode() != ""


@pytest.mark.parametrize("kw,code", BAD_CACHES + [
    (dict(N=-1), INVALID), (dict(N=(1 << 24) + 1), UNSUPPORTED), (dict(Hq=0), INVALID), (dict(Hq=5), INVALID),
    (dict(Hq=34), UNSUPPORTED), (dict(S=0), INVALID), (dict(S=1), INVALID), (dict(sink=-1), INVALID),
    (dict(recent=0), INVALID), (dict(sink=2, recent=2), INVALID), (dict(sink=2**31 - 1, recent=2**31 - 1), INVALID),
    (dict(max_pages=32769), UNSUPPORTED), (dict(N=1 << 24, Hk=64, Hq=512), UNSUPPORTED),
    (dict(S=2**31 - 1), UNSUPPORTED), (dict(q=None), INVALID), (dict(m=None), INVALID), (dict(seq=None), INVALID),
    (dict(pos=None), INVALID), (dict(pages=None), INVALID), (dict(rows=None), INVALID), (dict(q=Q + 2), MISALIGNED),
    (dict(m=MEANS + 8), MISALIGNED), (dict(pages=PAGES_AT + 2), MISALIGNED), (dict(rows=ROWS + 1), MISALIGNED),
    (dict(pages=Q), INVALID), (dict(rows=MEANS), INVALID), (dict(pages=SEQ), INVALID), (dict(rows=PAGES_AT), INVALID),
    (dict(rows=TAB), INVALID),
])
def test_select_rejects(lib, kw, code):  # noqa: F811
    assert select(lib, **kw) == code
    assert lib.moda_last_error_detail().decode() != ""


# what selected pages do not need of a cache: its sequences
SEQUENCES = [x for x in BAD_CACHES if set(x[0]) & {"B", "max_pages", "table"}]


@pytest.mark.parametrize("kw,code", [x for x in BAD_CACHES if x not in SEQUENCES] + [
    (dict(N=-1), INVALID), (dict(S=0), INVALID), (dict(N=1 << 23), UNSUPPORTED), (dict(Hq=0), INVALID),
    (dict(Hq=5), INVALID), (dict(Hq=34), UNSUPPORTED), (dict(L=-1), INVALID), (dict(L=1025), UNSUPPORTED),
    (dict(scale=-1.0), INVALID), (dict(S=1 << 27), UNSUPPORTED), (dict(N=1 << 20, S=1 << 24), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(pages=None), INVALID), (dict(rows=None), INVALID), (dict(o=None), INVALID),
    (dict(ws=None), INVALID), (dict(kd=None), INVALID), (dict(vd=None), INVALID), (dict(sl=56), INVALID),
    (dict(sh=60), INVALID), (dict(st=0), INVALID), (dict(wsb=0), INVALID), (dict(q=Q + 2), MISALIGNED),
    (dict(kd=KD + 8), MISALIGNED), (dict(ws=WS + 4), MISALIGNED), (dict(pages=PAGES_AT + 2), MISALIGNED),
    (dict(rows=ROWS + 2), MISALIGNED), (dict(o=Q), INVALID), (dict(lse=O + 64), INVALID), (dict(ws=PK), INVALID),
    (dict(o=PAGES_AT), INVALID), (dict(lse=ROWS), INVALID),
])
def test_selected_rejects(lib, kw, code):  # noqa: F811
    assert selected(lib, **kw) == code
    assert lib.moda_last_error_detail().decode() != ""


def test_calls_without_work(lib):  # noqa: F811
    assert prefill(lib, N=0, q=None, o=None) == OK
    assert prefill(lib, B=0, table=None, q=None, o=None, lens=None) == OK
    assert means(lib, N=0, m=None) == OK
    assert select(lib, N=0, q=None, pages=None) == OK
    assert selected(lib, N=0, q=None, o=None) == OK
    for call in (lib.moda_prefill_paged_workspace_bytes,):
        assert call(16, 4, 128) > 0 and call(16, 4, 64) <= call(16, 4, 128)
        for none in ((0, 4, 128), (6, 4, 128), (17 * 4, 4, 128), (4, 0, 128), (4, 4, 96)):
            assert call(*none) == 0


def test_null_cache(lib):  # noqa: F811
    assert lib.moda_prefill_paged(Q, 256, None, STARTS, LENS, KD, VD, 640, 128, 64, 5, 4, 4, 0.1, O, LSE, WS, 1 << 30,
                                  None) == INVALID
    assert lib.moda_page_means(None, SEQ, POS, 5, MEANS, None) == INVALID
    assert lib.moda_select_pages(Q, MEANS, None, SEQ, POS, 5, 4, 3, 1, 1, PAGES_AT, ROWS, None) == INVALID
    assert lib.moda_decode_selected(Q, None, PAGES_AT, ROWS, 5, 3, KD, VD, 512, 256, 64, 4, 4, 0.1, O, LSE, WS, 1 << 30,
                                    None) == INVALID


def test_calls_that_pass_validation_end_at_the_device(lib):  # noqa: F811
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for call in (prefill, means, select, selected):
        assert call(lib) == NO_DEVICE
    assert prefill(lib, kd=None, vd=None, L=0, lse=None, N=1, qs=3) == NO_DEVICE
    for kw, _ in SEQUENCES:
        assert selected(lib, **kw) == NO_DEVICE


# ------------------------------------------------------ tensors to the library
def arguments(call, mx4):
    c = tensors(mx4)
    scales = {n: c.pop(n) for n in ("k_scales", "v_scales")}
    pool = {n: c[n] for n in ("k_pages", "v_pages")}
    if call == "prefill":
        return dict(q=bf(N, HQ + 2, D)[:, :HQ], **c, q_starts=i32(B + 1), seq_lens=i32(B), scale=0.3,
                    kd=bf(L, N, HK + 1, D)[:, :, :HK], vd=bf(L, N, HK + 1, D)[:, :, :HK], **scales, o=bf(N, HQ, D),
                    lse=f32(N, HQ), workspace=f32(99), want_lse=False)
    if call == "means":
        return dict(**c, seq=i32(N), pos=i32(N), means=bf(PAGES, HK, D), **scales)
    if call == "select":
        return dict(q=bf(N, HQ, D), means=bf(PAGES, HK, D), **c, seq=i32(N), pos=i32(N), S=3, sink=1, recent=2,
                    **scales, pages=i32(N, HK, 3), rows=i32(N, HK))
    return dict(q=bf(N, HQ, D), **pool, pages=i32(N, HK, 3), rows=i32(N, HK), scale=0.3,
                kd=bf(N, L, HK, D).transpose(1, 2), vd=bf(N, L, HK, D).transpose(1, 2), **scales, o=bf(N, HQ, D),
                lse=f32(N, HQ), workspace=f32(99), want_lse=False)


SLOW = dict(prefill=moda.moda_prefill_paged, means=moda.moda_page_means, select=moda.moda_select_pages,
            selected=moda.moda_decode_selected)
OUTS = dict(prefill=("o", "lse"), means=(), select=("pages", "rows"), selected=("o", "lse"))
NAMES = dict(prefill="moda_prefill_paged", means="moda_page_means", select="moda_select_pages",
             selected="moda_decode_selected")
CALLS = list(itertools.product(SLOW, (False, True)))


@pytest.fixture
def more(ways):  # noqa: F811
    """The recorder and the extension of `ways` with the later functions too."""
    rec, ext = ways
    real = rec.lib
    for name in NAMES.values():
        rec.c[name] = c_type(real, name)(rec.keep)
        setattr(rec, name, rec.keep)
    size = "moda_prefill_paged_workspace_bytes"
    rec.c[size] = c_type(real, size)(lambda *shape: WORKSPACE)
    setattr(rec, size, lambda *shape: WORKSPACE)
    order = ("moda_prefill_paged", size, "moda_page_means", "moda_select_pages", "moda_decode_selected")
    ext.more(*(ctypes.cast(rec.c[n], ctypes.c_void_p).value for n in order))
    return rec, ext


def both(rec, ext, call, a):
    rec.seen = None
    fast = getattr(ext, call)(*a.values())
    assert (fast is None) == (rec.seen is None)
    fast, rec.seen = (rec.seen if fast is not None else None), None
    try:
        SLOW[call](**a)
        slow = rec.seen
    except Exception as e:  # noqa: BLE001
        slow = e
    return fast, slow


@pytest.mark.parametrize("call,mx4", CALLS)
def test_a_full_call_takes_the_extension(more, call, mx4):
    rec, ext = more
    fast, slow = both(rec, ext, call, arguments(call, mx4))
    assert fast is not None and fast == slow and fast[-1] == STREAM
    gone = dict(prefill=(("kd", "vd"), ("lse",)), selected=(("kd", "vd"), ("kd", "vd", "lse"))).get(call, ())
    for names in gone:
        fast, slow = both(rec, ext, call, dict(arguments(call, mx4), **dict.fromkeys(names)))
        assert fast is not None and fast == slow, names


@pytest.mark.parametrize("call,mx4", CALLS)
def test_what_the_extension_takes_the_checks_take_alike(more, call, mx4):
    rec, ext = more
    base = arguments(call, mx4)
    took = 0
    for name, t in base.items():
        for x in (bad(t) if isinstance(t, torch.Tensor) else (None, 0, 1, 2.5, "x", True, bf(1), bf(2))):
            if x is None and name in OUTS[call] + ("workspace",):
                continue  # made
            fast, slow = both(rec, ext, call, dict(base, **{name: x}))
            if fast is not None:
                took += 1
                assert fast == slow, (name, x)
    assert took >= 1
    for a, b in ((("kd", "vd"),) if "kd" in base else ()) + ((("q", "o"),) if "o" in base else ()):
        for x, y in zip(bad(base[a]), bad(base[b])):
            fast, slow = both(rec, ext, call, dict(base, **{a: x, b: y}))
            assert fast is None or fast == slow, (a, b, x, y)


@pytest.mark.parametrize("call,mx4", CALLS)
def test_missing_outputs_are_made(more, call, mx4):
    rec, ext = more
    full = arguments(call, mx4)
    gone = OUTS[call] + (("workspace",) if "workspace" in full else ())
    for names in itertools.chain.from_iterable(itertools.combinations(gone, i) for i in range(1, len(gone) + 1)):
        for wanted in (True, False) if "want_lse" in full else (None,):
            a = dict(full, **dict.fromkeys(names))
            if wanted is not None:
                a["want_lse"] = wanted
            fast, slow = getattr(ext, call)(*a.values()), SLOW[call](**a)
            for x, y, n in zip(fast, slow, OUTS[call]):
                if n == "lse" and not wanted and n in names:
                    assert x is None and y is None
                else:
                    assert x.shape == y.shape and x.dtype == y.dtype and x.is_contiguous()
                    assert (x is a[n]) == (y is a[n]) == (n not in names)


@pytest.mark.parametrize("call,mx4", CALLS)
def test_the_binding_takes_the_extension_and_raises_its_status(more, monkeypatch, call, mx4):
    rec, ext = more
    monkeypatch.setattr(binding, "_paged", ext)
    monkeypatch.setattr(binding, "_paged_cache", None)  # the checks behind it are not reached
    a = arguments(call, mx4)
    out = SLOW[call](**a)
    assert out is a["means"] if call == "means" else all(x is a[n] for x, n in zip(out, OUTS[call]))
    rec.status = 3
    with pytest.raises(moda.ModaError, match="recorded"):
        SLOW[call](**a)


@pytest.mark.parametrize("call,mx4", CALLS)
def test_what_is_no_tensor(more, call, mx4):
    rec, _ = more
    base = arguments(call, mx4)
    for name, t in base.items():
        if not isinstance(t, torch.Tensor):
            continue
        for x in ([1.0], 3, "x"):
            rec.seen = None
            with pytest.raises(TypeError, match=name):
                SLOW[call](**dict(base, **{name: x}))
            assert rec.seen is None


@pytest.mark.parametrize("call,mx4", CALLS)
def test_needed_tensors_may_not_be_none(more, call, mx4):
    rec, _ = more
    base = arguments(call, mx4)
    free = set(OUTS[call]) | {"workspace", "kd", "vd", "k_scales", "v_scales"}
    for name, t in base.items():
        if isinstance(t, torch.Tensor) and name not in free:
            rec.seen = None
            with pytest.raises((TypeError, ValueError, AttributeError)):
                SLOW[call](**dict(base, **{name: None}))
            assert rec.seen is None


# ------------------------------------------------------- the plain forms themselves
@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
def test_prefill_reference_is_the_decode_of_each_token(fmt):
    lens, new, d = [19, 33, 5], [4, 0, 5], 64
    c = pc.Cache(fmt, lens, 2, d, 16, seed=3)
    g = torch.Generator().manual_seed(4)
    starts = [0, 4, 4, 9]
    q = torch.randn(9, 6, d, generator=g).bfloat16()
    kd, vd = (torch.randn(3, 9, 2, d, generator=g).bfloat16() for _ in range(2))
    o, lse, to, tl = cc.prefill_reference(c, q, starts, lens, kd, vd, 0.125)
    for n, (b, t) in enumerate([(0, 15), (0, 16), (0, 17), (0, 18), (2, 0), (2, 1), (2, 2), (2, 3), (2, 4)]):
        one = pc.Cache(fmt, lens, 2, d, 16, seed=3)
        one.table = one.table[b : b + 1]
        want = pc.decode_reference(one, q[n : n + 1], [t + 1], kd[:, n].transpose(0, 1)[None],
                                   vd[:, n].transpose(0, 1)[None], 0.125)
        assert torch.allclose(o[n], want[0][0], rtol=1e-12) and torch.allclose(lse[n], want[1][0], rtol=1e-12)
        # three half steps of bf16, of values of at most 12 (6 at a block scale of 2), and
        # what scores are off by: 2 * 68 * 2^-24 * 0.125 * sum|q k|, below another half step
        top = max(c.rows("v", b, lens[b]).abs().max().item(), vd.abs().max().item())
        assert top <= 12 and (to[n] > 0).all() and (to[n] < 4 * pc.HALF_BF16 * top).all() and (tl[n] < 1e-2).all()


def test_selection_by_hand():
    c = pc.Cache("bf16", [16 * 6 + 3], 1, 64, 16)
    means = torch.zeros(c.num_pages, 1, 64, dtype=torch.bfloat16)
    for i, x in enumerate([9.0, 1.0, 5.0, math.nan, 5.0, 7.0, 100.0]):
        means[c.table[0, i].long(), 0, 0] = x
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    q[0, 0, 0], q[0, 1, 0] = 1.0, 0.5
    at = (torch.tensor([0]), torch.tensor([16 * 6 + 2]))
    for S, sink, recent, want, rows in ((2, 0, 1, [0, 6], 19), (4, 1, 1, [0, 2, 5, 6], 51), (3, 0, 3, [4, 5, 6], 35),
                                        (6, 0, 1, [0, 1, 2, 4, 5, 6], 83), (9, 1, 1, [0, 1, 2, 3, 4, 5, 6], 99)):
        pages, r = cc.selection(c, q, means, *at, S, sink, recent)
        assert pages[0, 0].tolist() == c.table[0, want].tolist() + [-1] * (S - len(want))
        assert r[0, 0] == rows


def test_a_planted_mistake_does_not_pass():
    """The bounds on o are tight enough to show one key less, or another's slots, in some head
    of every token (a single key may weigh next to nothing in one head)."""
    lens, starts, d = [40], [0, 8], 64
    c = pc.Cache("bf16", lens, 1, d, 16)
    g = torch.Generator().manual_seed(5)
    q = torch.randn(8, 4, d, generator=g).bfloat16()
    kd, vd = (torch.randn(2, 8, 1, d, generator=g).bfloat16() for _ in range(2))
    o, _, to, _ = cc.prefill_reference(c, q, starts, lens, kd, vd, 0.125)
    off = cc.prefill_reference(c, q[:7], [0, 7], [39], kd[:, 1:], vd[:, 1:], 0.125)[0]  # the next token's slots
    assert ((off - o[:7]).abs() > to[:7]).flatten(1).any(1).all()
    late = cc.prefill_reference(c, q[1:], [0, 7], [39], kd[:, 1:], vd[:, 1:], 0.125)[0]  # without the own row
    assert ((late - o[1:]).abs() > to[1:]).flatten(1).any(1).all()
