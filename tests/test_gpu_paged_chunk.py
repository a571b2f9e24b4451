"""Chunks of new tokens over the paged cache on the GPU, against fp64 forms
(tests/paged_chunk_common.py), at the sizes and masks where they can go wrong."""
import math

import pytest
import torch

import sequence_depth_attention_gb300 as moda
from sequence_depth_attention_gb300 import build as mbuild

import paged_chunk_common as cc
import paged_common as pc

pytestmark = pytest.mark.gpu
INVALID = 1


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mbuild.build()
    moda.load()


def settled(want=0):
    torch.cuda.synchronize()
    assert moda.moda_get_device_error() == want


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def chunk(fmt, new, past, Hq, Hk, d, L, page, pad=0, seed=1, gap=0, q_mul=1.0, **kw):
    """A cache of past[b] + new[b] rows, queries and depth slots of the new tokens; tokens
    of no sequence and the gaps between tokens hold NaN."""
    lens = [n + p for n, p in zip(new, past)]
    c = pc.Cache(fmt, lens, Hk, d, page, seed=seed, device="cuda", **kw)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    N = starts[-1] + pad
    g = torch.Generator().manual_seed(seed + 1)
    x = torch.full((N, Hq * d + gap), math.nan, dtype=torch.bfloat16)
    x[: starts[-1], : Hq * d] = (torch.randn(starts[-1], Hq * d, generator=g) * q_mul).bfloat16()
    x = x.cuda()
    q = x[:, : Hq * d].view(N, Hq, d)
    kd = vd = None
    if L:
        kd, vd = (torch.randn(L, N, Hk, d, generator=g).bfloat16().cuda() for _ in range(2))
        kd[:, starts[-1] :] = math.nan
        vd[:, starts[-1] :] = math.nan
    return c, q, starts, lens, kd, vd


def run(c, q, starts, lens, kd, vd, scale, want=0, **kw):
    N, Hq, d = q.shape
    o = torch.full((N, Hq, d), 3.5, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((N, Hq), 3.5, dtype=torch.float32, device="cuda")
    got = moda.moda_prefill_paged(q, *c.args(), i32(starts), i32(lens), scale, kd=kd, vd=vd, o=o, lse=lse,
                                  **c.scales(), **kw)
    settled(want)
    assert got[0] is o and got[1] is lse
    return o, lse


def check(c, q, starts, lens, kd, vd, scale, o, lse):
    wo, wl, to, tl = cc.prefill_reference(c, q, starts, lens, kd, vd, scale)
    n = starts[-1]
    eo = (o[:n].double() - wo[:n]).abs() - to[:n]
    el = (lse[:n].double() - wl[:n]).abs() - tl[:n]
    assert (eo <= 0).all(), f"o off by {eo.max().item():.3e} more than its bound"
    assert (el <= 0).all(), f"lse off by {el.max().item():.3e} more than its bound"
    assert (o[n:] == 3.5).all() and (lse[n:] == 3.5).all()


CHUNKS = [
    # fmt, new tokens, rows before them, Hq, Hk, d, L, page, padding, gap
    ("bf16", [1], [0], 4, 1, 128, 0, 16, 0, 0),
    ("bf16", [5], [696], 16, 4, 128, 46, 64, 0, 0),
    ("bf16", [32], [0], 4, 1, 128, 4, 128, 0, 0),
    ("bf16", [33, 0, 1, 7], [127, 50, 128, 0], 16, 4, 128, 24, 32, 3, 8),
    ("bf16", [129, 64], [1, 129], 2, 2, 128, 3, 64, 1, 0),
    ("bf16", [300], [40], 32, 2, 128, 0, 16, 0, 16),
    ("bf16", [9, 18, 2], [260, 0, 1000], 6, 2, 128, 5, 16, 2, 0),
    ("bf16", [20], [77], 5, 1, 128, 33, 32, 0, 0),
    ("bf16", [1] * 40, list(range(0, 400, 10)), 8, 8, 128, 1, 16, 0, 0),
    ("bf16", [65, 3], [600, 4], 64, 8, 64, 64, 16, 0, 8),
    ("bf16", [17, 130, 1], [0, 130, 255], 16, 1, 64, 7, 32, 5, 0),
    ("bf16", [11], [300], 14, 2, 64, 0, 128, 0, 0),
    ("mx4", [1], [0], 4, 1, 128, 0, 16, 0, 0),
    ("mx4", [5], [696], 16, 4, 128, 46, 64, 0, 0),
    ("mx4", [33, 0, 1, 7], [127, 50, 128, 0], 16, 4, 128, 24, 32, 3, 8),
    ("mx4", [129, 64], [1, 129], 2, 2, 128, 3, 64, 1, 0),
    ("mx4", [300], [40], 32, 2, 128, 0, 128, 0, 0),
    ("mx4", [9, 18, 2], [260, 0, 1000], 6, 2, 128, 5, 16, 2, 0),
    ("mx4", [65, 3], [600, 4], 64, 8, 64, 64, 16, 0, 8),
    ("mx4", [17, 130, 1], [0, 130, 255], 16, 1, 64, 7, 32, 5, 0),
]


@pytest.mark.parametrize("case", CHUNKS, ids=lambda c: "-".join(map(str, c[:1] + c[3:])) + f"-{len(c[1])}x{max(c[1])}")
def test_chunks(case):
    fmt, new, past, Hq, Hk, d, L, page, pad, gap = case
    x = chunk(fmt, new, past, Hq, Hk, d, L, page, pad, gap=gap)
    o, lse = run(*x, d ** -0.5)
    check(*x, d ** -0.5, o, lse)


# ------------------------------------------------------- what is not to be seen
def plant(c, b, row, which, value, hk=0, col=5):
    """`value` in one element of a row (bf16), or its block of 32 as NaN (4-bit)."""
    page = c.table[b, row // c.page].item()
    if c.fmt == "bf16":
        getattr(c, which)[page, hk, row % c.page, col] = value
    else:
        getattr(c, which + "s")[page, hk, row % c.page, col // 32] = 255


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("d", [64, 128])
def test_later_rows_have_no_influence(fmt, which, d):
    """A NaN in one token's key or value: the tokens before it are what they were, bit for
    bit, and the others are what a NaN makes of them."""
    new, past, Hk, G, L = [150, 9, 40], [20, 250, 0], 2, 4, 5
    x = chunk(fmt, new, past, Hk * G, Hk, d, L, 16)
    c, q, starts, lens, kd, vd = x
    clean, clean_lse = run(*x, d ** -0.5)
    for b, t in ((0, 100), (1, 255), (2, 0), (2, 39)):  # the token at row t of sequence b
        c2 = pc.Cache(fmt, lens, Hk, d, 16, seed=1, device="cuda")
        plant(c2, b, t, which, math.nan if (b, t) != (1, 255) else math.inf, hk=1)
        o, lse = run(c2, *x[1:], d ** -0.5)
        first = starts[b] + t - past[b]
        hit = torch.zeros_like(o, dtype=torch.bool)
        cols = slice(None) if which == "k" else slice(5, 6) if fmt == "bf16" else slice(0, 32)
        hit[first : starts[b + 1], G:, cols] = True
        assert torch.equal(o[~hit], clean[~hit])
        assert not torch.isfinite(o[hit]).any() if which == "v" else (fmt == "bf16" or torch.isnan(o[hit]).all())
        if which == "k":
            assert torch.equal(lse[: first], clean_lse[: first]) and torch.equal(lse[:, :G], clean_lse[:, :G])
        else:
            assert torch.equal(lse, clean_lse)


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_other_tokens_slots_have_no_influence(fmt, value):
    new, past, Hk, G, d, L = [70, 3], [5, 400], 2, 2, 128, 9
    x = chunk(fmt, new, past, Hk * G, Hk, d, L, 32, pad=2)
    clean, clean_lse = run(*x, d ** -0.5)
    c, q, starts, lens, kd, vd = x
    for token, slot, hk in ((0, 0, 0), (33, 8, 1), (69, 3, 0), (71, 5, 1)):
        v2 = vd.clone()
        v2[slot, token, hk, 100] = value
        o, lse = run(c, q, starts, lens, kd, v2, d ** -0.5)
        hit = torch.zeros_like(o, dtype=torch.bool)
        hit[token, hk * G : (hk + 1) * G, 100] = True
        n = starts[-1]
        assert torch.equal(o[:n][~hit[:n]], clean[:n][~hit[:n]]) and torch.equal(lse, clean_lse)
        want = torch.full_like(o[hit], value)
        assert torch.equal(torch.nan_to_num(o[hit], nan=7.0), torch.nan_to_num(want, nan=7.0))


def test_infinite_values_of_seen_rows():
    """An infinity that all tokens see, one that some see, and both signs in a column."""
    x = chunk("bf16", [64], [300], 4, 1, 128, 2, 16)
    c, q, starts, lens, kd, vd = x
    plant(c, 0, 10, "v", math.inf, col=3)
    plant(c, 0, 320, "v", -math.inf, col=3)
    plant(c, 0, 340, "v", -math.inf, col=77)
    o, _ = run(*x, 128 ** -0.5)
    assert (o[:20, :, 3] == math.inf).all() and torch.isnan(o[20:, :, 3]).all()
    assert torch.isfinite(o[:40, :, 77]).all() and (o[40:, :, 77] == -math.inf).all()
    rest = torch.ones(128, dtype=torch.bool, device="cuda")
    rest[[3, 77]] = False
    assert torch.isfinite(o[..., rest]).all()
