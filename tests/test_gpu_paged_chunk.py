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


# ---------------------------------------------------------------- hard scores
@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["large", "rising", "falling", "one", "jump in a block", "low depth"])
def test_scores_of_any_size(fmt, d, kind):
    """References that rise within a tile, a block and half a block; weights that vanish."""
    new, past, Hk, G, L = [40, 3], [500, 777], 2, 4, 6
    x = chunk(fmt, new, past, Hk * G, Hk, d, L, 16, q_mul=12.0 if kind == "large" else 1.0)
    c, q, starts, lens, kd, vd = x
    if kind != "large":
        # keys along one direction, whose factor makes the score of each row
        n = torch.arange(c.max_pages * 16, device="cuda", dtype=torch.float32)
        factor = dict(rising=n / 40, falling=-n / 40, one=torch.where(n == 300, 40.0, 0.0))
        factor["jump in a block"] = torch.where(n % 128 == 100, n / 20, 0.0)
        factor["low depth"] = torch.zeros_like(n)
        f = factor[kind]
        q.copy_((torch.randn(q.shape, generator=torch.Generator().manual_seed(2)) * 0.3).to(q))
        q[..., 0] = 8.0
        q[starts[-1]:] = math.nan
        if kd is not None:
            kd[..., 0] = -30.0 if kind == "low depth" else 0.0
        for b in range(len(lens)):
            for p in range(-(-lens[b] // 16)):
                page, fp = c.table[b, p].long(), f[p * 16 : p * 16 + 16]
                if fmt == "bf16":
                    c.k[page, :, :, 0] = torch.where(c.k[page, :, :, 0].isnan(), c.k[page, :, :, 0], fp.to(c.k))
                else:  # the block's first value 4 * 2^E with its sign
                    e = torch.where(fp == 0, torch.zeros_like(fp), torch.log2(fp.abs().clamp(min=1e-3))).round().clamp(-6, 4)
                    byte = (e - 2 + 127).to(torch.uint8)
                    c.ks[page, :, :, 0] = torch.where(c.ks[page, :, :, 0] == 255, c.ks[page, :, :, 0], byte)
                    c.k[page, :, :, 0] = torch.where(fp < 0, 14, 6).to(torch.uint8) + (c.k[page, :, :, 0] & 0x10)
    o, lse = run(*x, d ** -0.5)
    assert torch.isfinite(o[: starts[-1]]).all()
    check(*x, d ** -0.5, o, lse)


# ------------------------------------------------------------ how it is called
def test_a_single_token_is_a_decode():
    lens = [1, 700, 129, 5000]
    c, q, starts, _, kd, vd = chunk("bf16", [1] * 4, [n - 1 for n in lens], 16, 4, 128, 9, 64)
    o, lse = run(c, q, starts, lens, kd, vd, 0.1)
    want, wl = moda.moda_decode_paged(q, *c.args(), i32(lens), 0.1, kd=kd.permute(1, 2, 0, 3), vd=vd.permute(1, 2, 0, 3))
    settled()
    _, _, to, tl = cc.prefill_reference(c, q, starts, lens, kd, vd, 0.1)
    assert ((o.double() - want.double()).abs() <= 2 * to).all() and ((lse.double() - wl.double()).abs() <= 2 * tl).all()


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
def test_long_contexts_are_split(fmt):
    """More blocks than SMs, by far, for a few rows, and a table wider than the batch needs."""
    x = chunk(fmt, [3, 1, 0, 20], [30000, 0, 0, 9000], 16, 1, 128, 2, 128, width=400)
    o, lse = run(*x, 128 ** -0.5)
    check(*x, 128 ** -0.5, o, lse)


def test_depth_slots_at_any_strides():
    c, q, starts, lens, kd, vd = chunk("bf16", [9, 30], [100, 4], 8, 2, 64, 5, 32)
    o, lse = run(c, q, starts, lens, kd, vd, 0.125)
    for order in ((2, 1, 0, 3), (1, 2, 0, 3), (1, 0, 2, 3)):  # memory order of [L, N, Hk]
        back = [order.index(i) for i in range(4)]
        k2, v2 = (t.permute(order).contiguous().permute(back) for t in (kd, vd))
        o2, lse2 = run(c, q, starts, lens, k2, v2, 0.125)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    wide = [torch.full((5, q.shape[0], 4, 80), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for w, t in zip(wide, (kd, vd)):
        w[:, :, 1:3, 8:72] = t
    o2, lse2 = run(c, q, starts, lens, *(w[:, :, 1:3, 8:72] for w in wide), 0.125)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_tokens_of_no_sequence():
    """Tokens before the first sequence's and behind the last one's, and sequences without."""
    c, q, starts, lens, kd, vd = chunk("bf16", [5, 0, 12], [60, 9, 3], 4, 2, 128, 3, 16, pad=4)
    full, full_lse = run(c, q, starts, lens, kd, vd, 0.1)
    some = [5, 5, 5, 17]  # the first sequence's five tokens belong to none
    o, lse = run(c, q, some, lens, kd, vd, 0.1)
    assert (o[:5] == 3.5).all() and (o[17:] == 3.5).all() and (lse[:5] == 3.5).all()
    _, _, to, tl = cc.prefill_reference(c, q, starts, lens, kd, vd, 0.1)
    assert ((o[5:17].double() - full[5:17].double()).abs() <= 2 * to[5:17]).all()
    o, lse = run(c, q, [0, 0, 0, 0], lens, kd, vd, 0.1)
    assert (o == 3.5).all() and (lse == 3.5).all()


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
def test_bad_indexes_are_left_out_and_latched(fmt):
    c, q, starts, lens, kd, vd = chunk(fmt, [5, 8, 12], [60, 9, 3], 4, 2, 128, 3, 16)
    whole, _ = run(c, q, starts, lens, kd, vd, 0.1)
    _, _, to, _ = cc.prefill_reference(c, q, starts, lens, kd, vd, 0.1)

    def others(o, first, last):
        keep = torch.ones(q.shape[0], dtype=torch.bool, device="cuda")
        keep[first:last] = False
        assert ((o.double() - whole.double()).abs()[keep] <= 2 * to[keep]).all()
        return o[~keep]

    for bad in (7, -1, c.max_pages * 16 + 1):  # fewer rows than tokens, none, more than the table's
        o, _ = run(c, q, starts, [lens[0], bad, lens[2]], kd, vd, 0.1, want=INVALID)
        assert (others(o, 5, 13) == 3.5).all()
    for s in ([0, 5, 13, 26], [0, 5, 13, 12], [-3, 5, 13, 25]):  # beyond N, falling, before 0
        o, _ = run(c, q, s, lens, kd, vd, 0.1, want=INVALID)
        at = (13, 25) if s[0] == 0 else (0, 5)
        assert (others(o, *at) == 3.5).all()
    for bad in (c.num_pages, -1, 2**31 - 1):  # a page that is not in the pool
        was = c.table[1, 0].item()
        c.table[1, 0] = bad
        others(run(c, q, starts, lens, kd, vd, 0.1, want=INVALID)[0], 5, 13)
        c.table[1, 0] = was
    o, _ = run(c, q, starts, lens, kd, vd, 0.1)
    assert torch.equal(o, whole)


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
def test_captured_calls_follow_their_inputs(fmt):
    """One capture, replayed with other lengths, tables, queries; two graphs with a
    workspace each at once."""
    x = chunk(fmt, [30, 2, 9], [200, 900, 0], 8, 2, 128, 4, 32, pad=3)
    c, q, starts, lens, kd, vd = x
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    need = moda.moda_prefill_paged_workspace_bytes(8, 2, 128) // 4
    st, ln = i32(starts), i32(lens)
    outs, graphs = [], []
    for s in (s1, s2):
        o = torch.full_like(q, 3.5).contiguous()
        lse = torch.full(q.shape[:2], 3.5, device="cuda")
        ws = torch.empty(need, device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            moda.moda_prefill_paged(q, *c.args(), st, ln, 0.1, kd=kd, vd=vd, o=o, lse=lse, workspace=ws, **c.scales())
        outs.append((o, lse, ws))
        graphs.append(g)
    for new, rows in (([30, 2, 9], lens), ([1, 20, 8], [100, 620, 9]), ([41, 0, 0], [60, 0, 0])):
        sts = [0, new[0], new[0] + new[1], sum(new)]
        st.copy_(i32(sts))
        ln.copy_(i32(rows))
        q.copy_(torch.randn_like(q))
        for o, lse, _ in outs:
            o.fill_(3.5)
            lse.fill_(3.5)
        torch.cuda.synchronize()
        for g, s in zip(graphs, (s1, s2)):
            with torch.cuda.stream(s):
                for _ in range(3):
                    g.replay()
        settled()
        for o, lse, _ in outs:
            check(c, q, sts, rows, kd, vd, 0.1, o, lse)
            assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])


def test_a_stream_of_its_own():
    x = chunk("bf16", [30, 2], [200, 900], 8, 2, 128, 4, 32)
    c, q, starts, lens, kd, vd = x
    want, wl = run(*x, 0.1)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream, 0):
        o, lse = moda.moda_prefill_paged(q, *c.args(), i32(starts), i32(lens), 0.1, kd=kd, vd=vd, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(lse, wl)
    assert moda.moda_prefill_paged(q, *c.args(), i32(starts), i32(lens), 0.1, kd=kd, vd=vd, want_lse=False)[1] is None
    settled()


def test_the_same_call_gives_the_same_bits():
    x = chunk("mx4", [70, 5, 300], [3000, 9000, 0], 16, 2, 128, 12, 16)
    first = run(*x, 0.1)
    for _ in range(5):
        again = run(*x, 0.1)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


# ------------------------------------------------------------ as a server does
@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
def test_a_prompt_in_pieces_then_selected_decoding(fmt):
    """Prompts of three sequences come in pieces: append, summaries, attention of the piece
    over all that the cache holds. Then steps of one token each that attend to selected
    pages. Each step against fp64 forms over the cache as it is."""
    Hq, Hk, d, L, page, S = 8, 2, 64, 3, 16, 6
    pieces = [[40, 0, 7], [100, 33, 1], [1, 60, 0]]
    total = [sum(p[b] for p in pieces) + 12 for b in range(3)]
    c = pc.Cache(fmt, [0, 0, 0], Hk, d, page, spare=sum(-(-n // page) for n in total), fill="nan", device="cuda",
                 width=max(-(-n // page) for n in total))
    order = torch.randperm(c.num_pages, generator=torch.Generator().manual_seed(3)).to(torch.int32)
    at = 0
    for b, n in enumerate(total):
        held = -(-n // page)
        c.table[b, :held] = order[at : at + held].cuda()
        at += held
    means = torch.full((c.num_pages, Hk, d), math.nan, dtype=torch.bfloat16, device="cuda")
    rope = pc.rope_table(max(total), 32).cuda()
    g = torch.Generator().manual_seed(4)
    lens = [0, 0, 0]

    def step(new):
        N = sum(new)
        qkv = torch.randn(N, (Hq + 2 * Hk) * d, generator=g).bfloat16().cuda()
        q, k, v = (qkv[:, a * d : b * d].view(N, -1, d) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))
        seq = i32([b for b in range(3) for _ in range(new[b])])
        pos = i32([t for b in range(3) for t in range(lens[b], lens[b] + new[b])])
        q, _ = moda.moda_kv_append(q, k, v, *c.args(), seq, pos, rope=rope, **c.scales())
        moda.moda_page_means(*c.args(), seq, pos, means, **c.scales())
        for b in range(3):
            lens[b] += new[b]
        return q, seq, pos, N

    for new in pieces:
        q, _, _, N = step(new)
        kd, vd = (torch.randn(L, N, Hk, d, generator=g).bfloat16().cuda() for _ in range(2))
        starts = [0, new[0], new[0] + new[1], N]
        o, lse = run(c, q, starts, lens, kd, vd, d ** -0.5)
        check(c, q, starts, lens, kd, vd, d ** -0.5, o, lse)
    for _ in range(12):
        q, seq, pos, N = step([1, 1, 1])
        # (the summaries of pages that are not full are never read: they are still NaN)
        pages, rows = moda.moda_select_pages(q, means, *c.args(), seq, pos, S, sink=1, recent=1, **c.scales())
        settled()
        want = cc.selection(c, q, means, seq.cpu(), pos.cpu(), S, 1, 1)
        assert torch.equal(pages.cpu(), want[0]) and torch.equal(rows.cpu(), want[1])
        kd, vd = (torch.randn(N, Hk, L, d, generator=g).bfloat16().cuda() for _ in range(2))
        o, lse = moda.moda_decode_selected(q, c.k, c.v, pages, rows, d ** -0.5, kd=kd, vd=vd, **c.scales())
        settled()
        wo, wl, to, tl = cc.selected_reference(c, q, pages, rows, kd, vd, d ** -0.5)
        assert ((o.double() - wo).abs() <= to).all() and ((lse.double() - wl).abs() <= tl).all()


# ------------------------------ small heads: each half of a block's keys by itself
def test_halves_of_a_block_that_hold_nothing():
    """One to 70 rows and no depth slots: the second 64 keys are none or few."""
    new, past = [5, 64, 65, 1, 6], [0, 0, 0, 63, 64]
    x = chunk("bf16", new, past, 16, 2, 64, 0, 16)
    o, lse = run(*x, 64 ** -0.5)
    check(*x, 64 ** -0.5, o, lse)


@pytest.mark.parametrize("loud", [0, 1])
@pytest.mark.parametrize("new,past", [([40], [500]), ([3, 20], [30000, 9000])])
def test_halves_of_a_block_far_apart(loud, new, past):
    """Scores of one half of every 128 keys are some 20 times the other's."""
    c, q, starts, lens, kd, vd = chunk("bf16", new, past, 8, 1, 64, 3, 64)
    for b, n in enumerate(lens):
        for i in range(-(-n // 64)):
            if i % 2 == loud:
                c.k[c.table[b, i].long()] *= 20
    o, lse = run(c, q, starts, lens, kd, vd, 64 ** -0.5)
    check(c, q, starts, lens, kd, vd, 64 ** -0.5, o, lse)


def test_infinite_values_of_seen_rows_in_small_heads():
    x = chunk("bf16", [64], [300], 4, 1, 64, 2, 16)
    c, q, starts, lens, kd, vd = x
    plant(c, 0, 10, "v", math.inf, col=3)
    plant(c, 0, 320, "v", -math.inf, col=3)
    plant(c, 0, 340, "v", -math.inf, col=61)
    o, _ = run(*x, 64 ** -0.5)
    assert (o[:20, :, 3] == math.inf).all() and torch.isnan(o[20:, :, 3]).all()
    assert torch.isfinite(o[:40, :, 61]).all() and (o[40:, :, 61] == -math.inf).all()
    rest = torch.ones(64, dtype=torch.bool, device="cuda")
    rest[[3, 61]] = False
    assert torch.isfinite(o[..., rest]).all()


def test_small_heads_captured_and_replayed():
    """Other lengths behind the captured addresses: other tiles, shares and joins."""
    new, past = [30, 2, 9], [200, 900, 0]
    c, q, starts, lens, kd, vd = chunk("bf16", new, past, 8, 2, 64, 4, 32)
    s, n = i32(starts), i32(lens)
    o = torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(q.shape[:2], dtype=torch.float32, device="cuda")
    work = torch.zeros(moda.moda_prefill_paged_workspace_bytes(8, 2, 64) // 4, dtype=torch.float32, device="cuda")

    def call():
        moda.moda_prefill_paged(q, *c.args(), s, n, 64 ** -0.5, kd=kd, vd=vd, o=o, lse=lse, workspace=work)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for m, rows in (([30, 2, 9], lens), ([41, 0, 0], [60, 0, 0]), ([20, 20, 1], [100, 620, 6])):
        starts = [0, m[0], m[0] + m[1], sum(m)]
        s.copy_(i32(starts))
        n.copy_(i32(rows))
        torch.cuda.synchronize()
        graph.replay()
        settled()
        check(c, q, starts, rows, kd, vd, 64 ** -0.5, o, lse)
