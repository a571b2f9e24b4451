"""The paged calls' two ways from tensors to the library: the extension module
for calls that are as they should be, and the Python code behind it that
checks, allocates and refuses. Both are run on CPU tensors against functions
that only record what they are given: what the first accepts, the second
passes on with the same arguments."""
import ctypes
import importlib.machinery
import importlib.util
import itertools
import shutil

import pytest
import torch

import sequence_depth_attention_gb300 as moda
from sequence_depth_attention_gb300 import binding
from sequence_depth_attention_gb300 import build as mbuild

STREAM = 0x5150
WORKSPACE = 4096


def c_type(lib, name):
    f = getattr(lib, name)
    return ctypes.CFUNCTYPE(f.restype, *f.argtypes)


def plain(x):
    """An argument as a callback or a call has it, as a comparable value."""
    if isinstance(x, ctypes._Pointer):
        x = x.contents
    if isinstance(x, binding._PagedKv):
        return tuple(getattr(x, n) or 0 for n, _ in x._fields_)
    if isinstance(x, float):
        return ctypes.c_float(x).value
    return x or 0


class Recorder:
    """moda_kv_append, moda_kv_gather and moda_decode_paged that return
    `status` and keep the arguments of their last call."""

    def __init__(self, lib):
        self.status, self.seen, self.lib = 0, None, lib
        self.c = {}
        for name in ("moda_kv_append", "moda_kv_gather", "moda_decode_paged"):
            self.c[name] = c_type(lib, name)(self.keep)
            setattr(self, name, self.keep)
        name = "moda_decode_paged_workspace_bytes"
        self.c[name] = c_type(lib, name)(lambda *shape: WORKSPACE)

    def keep(self, *args):
        self.seen = tuple(plain(a) for a in args)
        return self.status

    def moda_decode_paged_workspace_bytes(self, Hq, Hk, d):
        return WORKSPACE

    def moda_last_error_detail(self):
        return b"recorded"


@pytest.fixture
def ways(tmp_path, monkeypatch):
    """(recorder, extension): binding.py with the recorder for the library, the
    CPU for the current device, and a copy of the extension (which keeps what
    it was set up with) that calls the recorder too."""
    mbuild.build()
    lib = binding.load()
    rec = Recorder(lib)
    path = shutil.copy(binding._EXT, tmp_path / "paged_py.so")
    loader = importlib.machinery.ExtensionFileLoader("paged_py", str(path))
    ext = importlib.util.module_from_spec(importlib.util.spec_from_loader("paged_py", loader))
    loader.exec_module(ext)
    ext.setup(torch.Tensor, lambda: -1, lambda dev: STREAM,
              *(ctypes.cast(f, ctypes.c_void_p).value for f in rec.c.values()))
    monkeypatch.setattr(binding, "_lib", rec)
    monkeypatch.setattr(binding, "_paged", None)
    monkeypatch.setattr(binding, "_current_device", lambda: -1)
    monkeypatch.setattr(binding, "_raw_stream", lambda stream, dev: STREAM)
    return rec, ext


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def f32(*shape):
    return torch.zeros(shape, dtype=torch.float32)


N, B, HQ, HK, D, PAGES, PAGE, L = 5, 3, 8, 2, 64, 7, 16, 3


def cache(mx4):
    if mx4:
        return dict(k_pages=u8(PAGES, HK, PAGE, D // 2), v_pages=u8(PAGES, HK, PAGE, D // 2),
                    block_table=i32(B, 4), k_scales=u8(PAGES, HK, PAGE, D // 32),
                    v_scales=u8(PAGES, HK, PAGE, D // 32))
    return dict(k_pages=bf(PAGES, HK, PAGE, D), v_pages=bf(PAGES, HK, PAGE, D), block_table=i32(B, 4),
                k_scales=None, v_scales=None)


def arguments(call, mx4):
    c = cache(mx4)
    if call == "append":
        fused = bf(N, HQ + 2 * HK, D)
        return dict(q=fused[:, :HQ], k=fused[:, HQ:HQ + HK], v=fused[:, HQ + HK:], **c, seq=i32(N),
                    pos=i32(N), rope=f32(32, 32), interleaved=True, q_out=bf(N, HQ, D),
                    k_out=bf(N, HK, D), want_k_out=False)
    if call == "gather":
        return dict(**c, seq=i32(N), pos=i32(N), k=bf(N, HK, D), v=bf(N, HK, D))
    return dict(q=bf(B, HQ, D), **c, seq_lens=i32(B), scale=0.3, kd=bf(B, L, HK, D).transpose(1, 2),
                vd=bf(B, L, HK, D).transpose(1, 2), o=bf(B, HQ, D), lse=f32(B, HQ), workspace=f32(99),
                want_lse=False)


ORDER = dict(
    append=("q", "k", "v", "k_pages", "v_pages", "block_table", "seq", "pos", "rope", "interleaved",
            "k_scales", "v_scales", "q_out", "k_out", "want_k_out"),
    gather=("k_pages", "v_pages", "block_table", "seq", "pos", "k_scales", "v_scales", "k", "v"),
    decode=("q", "k_pages", "v_pages", "block_table", "seq_lens", "scale", "kd", "vd", "k_scales",
            "v_scales", "o", "lse", "workspace", "want_lse"))
SLOW = dict(append=moda.moda_kv_append, gather=moda.moda_kv_gather, decode=moda.moda_decode_paged)
OUTS = dict(append=("q_out", "k_out"), gather=("k", "v"), decode=("o", "lse"))


def both(rec, ext, call, a):
    """(what the extension passed on, or None; what binding.py did, or its
    exception)."""
    rec.seen = None
    fast = getattr(ext, call)(*(a[n] for n in ORDER[call]))
    assert (fast is None) == (rec.seen is None)
    if fast is not None:
        assert len(fast) == 2 and all(x is a[n] or a[n] is None for x, n in zip(fast, OUTS[call]))
    fast, rec.seen = rec.seen, None
    try:
        SLOW[call](**a)
        slow = rec.seen
    except Exception as e:  # noqa: BLE001 (the refusals' types are tested elsewhere)
        slow = e
    return fast, slow


CALLS = list(itertools.product(("append", "gather", "decode"), (False, True)))


@pytest.mark.parametrize("call,mx4", CALLS)
def test_a_full_call_takes_the_extension(ways, call, mx4):
    rec, ext = ways
    fast, slow = both(rec, ext, call, arguments(call, mx4))
    assert fast is not None and fast == slow and fast[-1] == STREAM


@pytest.mark.parametrize("call,mx4", CALLS)
def test_optional_arguments_may_be_missing(ways, call, mx4):
    rec, ext = ways
    gone = dict(append=(("rope",), ("q", "q_out"), ("k_out",), ("q", "q_out", "k_out", "rope")), gather=(),
                decode=(("kd", "vd"), ("lse",), ("kd", "vd", "lse")))[call]
    for names in gone:
        a = dict(arguments(call, mx4), **dict.fromkeys(names))
        fast, slow = both(rec, ext, call, a)
        assert fast is not None and fast == slow, names


def bad(t):
    """Tensors in t's place: most must not get through, some may."""
    yield None
    yield 3
    yield t.to(torch.float64)
    yield t.to(torch.int64)
    yield t.to("meta")
    yield t[..., :-1]
    yield t[..., :-1].contiguous()
    yield t[:-1].contiguous()
    yield t[:0].contiguous()
    yield t.unsqueeze(0)
    yield t[0] if t.dim() else t
    yield t.expand(2, *t.shape)
    yield torch.zeros((*t.shape[:-1], 2 * t.shape[-1]), dtype=t.dtype)[..., ::2]
    yield torch.zeros((*t.shape[:-1], 2 * t.shape[-1]), dtype=t.dtype)[..., :t.shape[-1]]
    yield t[:1].expand(t.shape)
    if t.dim() > 1:
        yield t.transpose(0, 1)
        yield t.transpose(0, 1).contiguous()
        yield t.transpose(-1, -2).contiguous().transpose(-1, -2)
        yield torch.cat([t, t], 1)
        yield t[:, :1]
        yield torch.cat([t, t], 0)[::2]


@pytest.mark.parametrize("call,mx4", CALLS)
def test_what_the_extension_takes_the_checks_take_alike(ways, call, mx4):
    rec, ext = ways
    base = arguments(call, mx4)
    took = 0
    for name, t in base.items():
        for x in (bad(t) if isinstance(t, torch.Tensor) else (None, 0, 1, 2.5, "x", True, bf(1), bf(2))):
            if x is None and name in OUTS[call] + ("workspace",):
                continue  # made: see test_missing_outputs_are_made
            fast, slow = both(rec, ext, call, dict(base, **{name: x}))
            if fast is not None:
                took += 1
                assert fast == slow, (name, x)
    assert took >= 2


@pytest.mark.parametrize("call", ("append", "decode"))
def test_pairs_changed_together(ways, call):
    rec, ext = ways
    base = arguments(call, False)
    pairs = dict(append=(("k", "v"), ("q", "q_out"), ("seq", "pos")), decode=(("kd", "vd"), ("q", "o")))
    for a, b in pairs[call]:
        for x, y in zip(bad(base[a]), bad(base[b])):
            fast, slow = both(rec, ext, call, dict(base, **{a: x, b: y}))
            assert fast is None or fast == slow, (a, b, x, y)


@pytest.mark.parametrize("call,mx4", CALLS)
def test_missing_outputs_are_made(ways, call, mx4):
    """Outputs and a workspace that are not given: as in the Python path but
    for where they are."""
    rec, ext = ways
    want = dict(append="want_k_out", gather=None, decode="want_lse")[call]
    full = arguments(call, mx4)
    gone = OUTS[call] + (("workspace",) if call == "decode" else ())
    for names in itertools.chain.from_iterable(itertools.combinations(gone, i) for i in range(1, len(gone) + 1)):
        a = dict(full, **dict.fromkeys(names))
        for wanted in (True, False) if want else (None,):
            if want:
                a[want] = wanted
            rec.seen = None
            fast = getattr(ext, call)(*(a[n] for n in ORDER[call]))
            assert fast is not None and rec.seen is not None
            seen, rec.seen = rec.seen, None
            slow = SLOW[call](**a)
            left_out = want and not wanted and OUTS[call][1] in names
            for i, (x, y, n) in enumerate(zip(fast, slow, OUTS[call])):
                if i == 1 and left_out:
                    assert x is None and y is None
                else:
                    assert x.shape == y.shape and x.dtype == y.dtype and x.is_contiguous()
                    assert (x is a[n]) == (y is a[n]) == (n not in names)
                    assert x.data_ptr() in seen and y.data_ptr() in rec.seen
            new = {t.data_ptr() for t in (*fast, *slow) if t is not None}
            differ = [i for i, (x, y) in enumerate(zip(seen, rec.seen)) if x != y]
            assert all(seen[i] in new or call == "decode" and i == len(seen) - 3 for i in differ)
            if call == "decode":  # the workspace's size
                assert seen[-2] == rec.seen[-2] == (WORKSPACE if "workspace" in names else 99 * 4)


@pytest.mark.parametrize("call,mx4", CALLS)
def test_the_binding_takes_the_extension_and_raises_its_status(ways, monkeypatch, call, mx4):
    rec, ext = ways
    monkeypatch.setattr(binding, "_paged", ext)
    a = arguments(call, mx4)
    monkeypatch.setattr(binding, "_paged_cache", None)  # the checks behind it are not reached
    out = SLOW[call](**a)
    assert all(x is a[n] for x, n in zip(out, OUTS[call])) and rec.seen is not None
    rec.status = 3
    with pytest.raises(moda.ModaError, match="recorded"):
        SLOW[call](**a)


def test_wrong_counts_of_arguments_are_no_call(ways):
    rec, ext = ways
    assert ext.append() is None and ext.gather(1) is None and ext.decode(*range(20)) is None
    assert rec.seen is None
