"""Page summaries, the choice of pages by them and the attention over chosen pages on the
GPU, against plain fp64 forms (tests/paged_chunk_common.py)."""
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


def normal(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


# ----------------------------------------------------------------- summaries
@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,Hk,lens", [(16, 1, [16]), (16, 3, [1, 15, 16, 17, 32, 160]), (32, 8, [64, 31, 100]),
                                          (64, 4, [64, 701]), (128, 2, [128, 127, 513, 256])])
def test_means(fmt, d, page, Hk, lens):
    c = pc.Cache(fmt, lens, Hk, d, page, seed=3, device="cuda")
    # every row of the second half of each sequence, in no order, among padding
    at = [(b, t) for b, n in enumerate(lens) for t in range(n // 2, n)] + [(-1, page - 1)] * 3
    order = torch.randperm(len(at), generator=torch.Generator().manual_seed(1)).tolist()
    seq, pos = i32([at[i][0] for i in order]), i32([at[i][1] for i in order])
    means = torch.full((c.num_pages, Hk, d), 3.5, dtype=torch.bfloat16, device="cuda")
    got = moda.moda_page_means(*c.args(), seq, pos, means, **c.scales())
    settled()
    assert got is means
    want = cc.page_means(c)
    filled = torch.zeros(c.num_pages, dtype=torch.bool, device="cuda")
    for b, t in at:
        if b >= 0 and t % page == page - 1:
            filled[c.table[b, t // page].long()] = True
    assert (means[~filled] == 3.5).all()
    # one rounding to bf16, and page sums in fp32 of magnitudes' mean
    mags = (c.k.double() if fmt == "bf16" else pc.mx4_values(c.k, c.ks)).abs().mean(2)
    err = (means.double() - want).abs()[filled]
    assert (err <= (pc.HALF_BF16 * want.abs() + page * 2 * pc.HALF_FP32 * mags)[filled]).all()


def test_means_of_large_and_small_values():
    """Sums that fp32 could not hold, values next to zero, infinities and NaN, a page
    named twice."""
    c = pc.Cache("bf16", [64], 1, 64, 16, fill=None, device="cuda")
    ids = c.table[0].long()
    c.k[ids[0]] = 3e38
    c.k[ids[1]] = 2e-39
    c.k[ids[2], 0, 5, 7] = math.inf
    c.k[ids[3], 0, 2, 9] = math.nan
    means = torch.zeros(c.num_pages, 1, 64, dtype=torch.bfloat16, device="cuda")
    moda.moda_page_means(*c.args(), i32([0, 0, 0, 0, 0]), i32([15, 31, 47, 63, 15]), means)
    settled()
    assert (means[ids[0]] == c.k[ids[0], 0, 0, 0]).all()
    assert (means[ids[1]].double() - 2e-39).abs().max() < 2e-39 * 2 ** -6
    assert means[ids[2], 0, 7] == math.inf and torch.isfinite(means[ids[2], 0]).sum() == 63
    assert torch.isnan(means[ids[3], 0, 9]) and torch.isfinite(means[ids[3], 0]).sum() == 63


# --------------------------------------------------------------------- choice
def bare(lens, Hk, d, page, seed=3):
    """A table of pages without rows, for calls that read none."""
    c = pc.Cache("bf16", [0], Hk, d, page, seed=seed)
    held = [-(-n // page) for n in lens]
    c.lens, c.num_pages, c.max_pages = lens, sum(held) + 2, max(1, max(held))
    c.table = torch.full((len(lens), c.max_pages), -7, dtype=torch.int32)
    order = torch.randperm(c.num_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    at = 0
    for b, n in enumerate(held):
        c.table[b, :n] = order[at : at + n]
        at += n
    c.table = c.table.cuda()
    c.k = c.v = torch.zeros(c.num_pages, Hk, page, d, dtype=torch.bfloat16, device="cuda")
    return c


def choose(c, q, means, seq, pos, S, sink, recent, want=0):
    N = q.shape[0]
    pages = torch.full((N, c.Hk, S), 99, dtype=torch.int32, device="cuda")
    rows = torch.full((N, c.Hk), 99, dtype=torch.int32, device="cuda")
    got = moda.moda_select_pages(q, means, *c.args(), seq, pos, S, sink=sink, recent=recent, pages=pages, rows=rows)
    settled(want)
    assert got[0] is pages and got[1] is rows
    return pages.cpu(), rows.cpu()


def compare(c, q, means, seq, pos, S, sink, recent):
    got = choose(c, q, means, seq, pos, S, sink, recent)
    want = cc.selection(c, q, means, seq.cpu(), pos.cpu(), S, sink, recent)
    assert torch.equal(got[1], want[1])
    assert torch.equal(got[0], want[0])


SELECTIONS = [
    # lens, Hq, Hk, d, page, S, sink, recent, padding
    ([1], 4, 1, 128, 16, 1, 0, 1, 0),
    ([65536], 16, 4, 128, 64, 32, 1, 2, 0),
    ([700, 1, 64, 65, 2000, 16], 16, 4, 128, 16, 8, 1, 2, 2),
    ([5000] * 3, 64, 4, 64, 16, 17, 0, 1, 1),
    ([900, 901], 7, 7, 64, 32, 5, 2, 3, 0),
    ([3000, 12], 12, 1, 128, 16, 64, 2, 2, 0),
    ([16 * 32768], 2, 1, 64, 16, 100, 1, 1, 0),
    ([4000 + 37 * i for i in range(60)], 8, 2, 128, 128, 9, 0, 1, 4),
    ([33 * 16], 3, 1, 64, 16, 32, 0, 32, 0),
    ([40 * 16, 7], 4, 4, 128, 16, 39, 0, 1, 0),
]


@pytest.mark.parametrize("case", SELECTIONS, ids=lambda c: f"{len(c[0])}x{max(c[0])}-" + "-".join(map(str, c[1:])))
def test_selection(case):
    lens, Hq, Hk, d, page, S, sink, recent, pad = case
    c = bare(lens, Hk, d, page)
    seq = i32(list(range(len(lens))) + [-1] * pad)
    pos = i32([n - 1 for n in lens] + [0] * pad)
    compare(c, normal(len(lens) + pad, Hq, d, seed=4), normal(c.num_pages, Hk, d, seed=5), seq, pos, S, sink, recent)


def test_selection_of_a_chunk():
    """Several tokens of a sequence, each with the pages up to its own."""
    c = bare([1000, 300], 2, 128, 16)
    at = [(0, t) for t in range(930, 1000)] + [(1, t) for t in (0, 15, 16, 250, 299)]
    compare(c, normal(len(at), 8, 128, seed=6), normal(c.num_pages, 2, 128, seed=7), i32([a for a, _ in at]),
            i32([t for _, t in at]), 6, 1, 2)


@pytest.mark.parametrize("pages", [20, 100, 1000, 5000])
@pytest.mark.parametrize("kind", ["equal", "zeros", "two kinds", "tiny differences", "nan", "infinite", "overflow",
                                  "underflow", "signed zeros"])
def test_selection_among_close_scores(kind, pages):
    """Scores that are equal, that fp32 cannot tell apart, or that are no numbers: the
    order is that of the fp64 scores, then that of the pages."""
    Hk, G, d, page = 2, 4, 64, 16
    c = bare([pages * page - 3], Hk, d, page)
    q, means = normal(1, Hk * G, d, seed=8), normal(c.num_pages, Hk, d, seed=9)
    g = torch.Generator().manual_seed(10)
    if kind == "equal":
        means[:] = means[0]
    elif kind == "zeros":
        q[:, G:] = 0
        means[:, 0] = 0
    elif kind == "two kinds":
        means[:] = torch.where((torch.rand(c.num_pages, 1, 1, generator=g) < 0.5).cuda(), means[0], means[1])
    elif kind == "tiny differences":  # in an element that counts for 2^-40 of the score
        means[:] = means[0]
        q[..., 11] = 2.0 ** -40
        means[..., 11] = torch.randint(-40, 41, (c.num_pages, Hk), generator=g).bfloat16().cuda()
    elif kind == "nan":
        means[torch.rand(c.num_pages, generator=g).cuda() < 0.3, :, 5] = math.nan
        q[0, G + 1, 3] = math.nan
    elif kind == "infinite":
        means[torch.rand(c.num_pages, generator=g).cuda() < 0.1, 0, 5] = math.inf
        means[torch.rand(c.num_pages, generator=g).cuda() < 0.1, 1, 6] = -math.inf
    elif kind == "overflow":  # products that fp32 cannot hold
        q *= 2.0 ** 100
        means *= 2.0 ** 90
    elif kind == "underflow":
        q *= 2.0 ** -90
        means *= 2.0 ** -90
    else:
        q[:] = 0
        means[:] = torch.where((torch.rand(c.num_pages, 1, 1, generator=g) < 0.5).cuda(), means, -means)
    for S, sink, recent in ((7, 0, 1), (16, 2, 3)):
        compare(c, q, means, i32([0]), i32([pages * page - 4]), S, sink, recent)


# ------------------------------------------------------------------ attention
ATTENDS = [
    # fmt, rows of each (token, head), Hq, Hk, d, L, page, S
    ("bf16", [[1]], 4, 1, 128, 0, 16, 1),
    ("bf16", [[2048, 2001, 1990, 65]], 16, 4, 128, 48, 64, 32),
    ("bf16", [[0, 5], [33, 0], [17, 16]], 6, 2, 64, 0, 16, 4),
    ("bf16", [[100, 128], [1, 2], [0, 0]], 32, 2, 128, 5, 32, 4),
    ("mx4", [[1]], 4, 1, 128, 0, 16, 1),
    ("mx4", [[1024, 1001, 17, 64], [0, 16, 15, 500]], 32, 4, 128, 24, 16, 64),
    ("mx4", [[0, 5], [33, 0], [17, 16]], 6, 2, 64, 0, 16, 4),
    ("mx4", [[100, 128], [1, 2], [0, 0]], 32, 2, 64, 5, 32, 4),
    ("bf16", [[1000 + 7 * i + j for j in range(8)] for i in range(50)], 16, 8, 128, 3, 128, 12),
    ("mx4", [[1000 + 7 * i + j for j in range(8)] for i in range(50)], 16, 8, 128, 3, 128, 12),
]


@pytest.mark.parametrize("case", ATTENDS, ids=lambda c: "-".join(map(str, c[:1] + c[2:])) + f"-{len(c[1])}")
@pytest.mark.parametrize("layer_major", [False, True])
def test_attention_over_selected_pages(case, layer_major):
    fmt, rows, Hq, Hk, d, L, page, S = case
    N = len(rows)
    g = torch.Generator().manual_seed(11)
    # a sequence per (token, head) whose pages are spread over a pool; what none owns is NaN
    flat = [r for x in rows for r in x]
    c = pc.Cache(fmt, flat, 1, d, page, seed=12, width=S, device="cuda")
    extra = -c.num_pages % Hk  # whole pages of Hk row blocks
    def pool(x):
        if x is None:
            return None
        x = torch.cat((x, x[:1].expand(extra, -1, -1, -1))) if extra else x
        return x.reshape(-1, Hk, *x.shape[2:])
    pages = c.table.view(N, Hk, S)
    k, v, ks, vs = (pool(x) for x in (c.k, c.v, c.ks, c.vs))
    q = torch.randn(N, Hq, d, generator=g).bfloat16().cuda()
    kd = vd = None
    if L:
        kd, vd = (torch.randn(N, Hk, L, d, generator=g).bfloat16().cuda() for _ in range(2))
        if layer_major:  # as the layers write them
            kd, vd = (x.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3) for x in (kd, vd))
    o, lse = moda.moda_decode_selected(q, k, v, pages, i32(rows), d ** -0.5, kd=kd, vd=vd, k_scales=ks, v_scales=vs)
    settled()
    whole = pc.Cache(fmt, [0], Hk, d, page)
    whole.k, whole.v, whole.ks, whole.vs = k, v, ks, vs
    wo, wl, to, tl = cc.selected_reference(whole, q, pages, torch.tensor(rows), kd, vd, d ** -0.5)
    assert ((o.double() - wo).abs() <= to).all()
    empty = wl == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    assert ((lse.double() - wl).abs()[~empty] <= tl[~empty]).all()


def test_bad_indexes_are_latched():
    Hk, d, page = 2, 64, 16
    c = bare([100, 300], Hk, d, page)
    q, means = normal(4, 8, d, seed=20), normal(c.num_pages, Hk, d, seed=21)
    good = choose(c, q[:2], means, i32([0, 1]), i32([99, 299]), 5, 1, 1)
    # sequences and rows that are not there: no pages; the others as they were
    for seq, pos in (([0, 1, 2, 0], [99, 299, 5, -1]), ([0, 1, -2, 1], [99, 299, 5, c.max_pages * page])):
        got = choose(c, q, means, i32(seq), i32(pos), 5, 1, 1, want=INVALID)
        assert torch.equal(got[0][:2], good[0]) and torch.equal(got[1][:2], good[1])
        assert (got[0][2:] == -1).all() and (got[1][2:] == 0).all()
    # pages that are not in the pool: chosen last, and given as -1
    was = c.table.clone()
    for bad in (c.num_pages, -1, 2**31 - 1):
        c.table[1, 3:15] = bad
        pages, rows = choose(c, q[:2], means, i32([0, 1]), i32([99, 299]), 5, 1, 1, want=INVALID)
        assert torch.equal(pages[0], good[0][0]) and (pages[1] >= 0).all() and (rows == good[1]).all()
        pages, _ = choose(c, q[:2], means, i32([0, 1]), i32([99, 299]), 18, 1, 1, want=INVALID)
        assert ((pages[1] == -1).sum(-1) == 11).all()  # 19 pages, of which 12 are not there: one is left out
        c.table.copy_(was)
    fresh = torch.full((c.num_pages, Hk, d), 3.5, dtype=torch.bfloat16, device="cuda")
    c.table[0, 0] = c.num_pages
    moda.moda_page_means(*c.args(), i32([0, 1, 5, 1]), i32([15, 31, 15, 1 << 20]), fresh)
    settled(INVALID)
    touched = (fresh != 3.5).flatten(1).any(1).nonzero().flatten().tolist()
    assert touched == [int(was[1, 1])]
    x = normal(1, 4, 64, seed=22)
    k = v = normal(3, 2, 16, 64, seed=23)
    for pages, rows in (([[[6, 1], [1, 2]]], [[20, 30]]), ([[[0, 1], [1, -1]]], [[20, 30]]), ([[[0, 1], [1, 2]]], [[33, -1]])):
        moda.moda_decode_selected(x, k, v, i32(pages), i32(rows), 0.1)
        settled(INVALID)


def test_captured_selection_and_attention():
    """Captured together, replayed with other tokens and rows; a batch padded to its
    captured size."""
    Hq, Hk, d, page, S = 8, 2, 128, 16, 7
    lens = [900, 20, 333, 1]
    c = pc.Cache("bf16", lens, Hk, d, page, seed=24, device="cuda")
    means = cc.page_means(c).bfloat16()
    means[torch.isnan(means)] = 0
    q = normal(6, Hq, d, seed=25)
    seq, pos = i32([0, 1, 2, 3, -1, -1]), i32([n - 1 for n in lens] + [0, 0])
    need = moda.moda_decode_paged_workspace_bytes(Hq, Hk, d) // 4
    pages, rows = torch.zeros(6, Hk, S, dtype=torch.int32, device="cuda"), torch.zeros(6, Hk, dtype=torch.int32, device="cuda")
    o, lse, ws = torch.zeros_like(q), torch.zeros(6, Hq, device="cuda"), torch.empty(need, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        moda.moda_select_pages(q, means, *c.args(), seq, pos, S, sink=1, recent=2, pages=pages, rows=rows)
        moda.moda_decode_selected(q, c.k, c.v, pages, rows, 0.1, o=o, lse=lse, workspace=ws)
    for s, t in (([0, 1, 2, 3, -1, -1], [899, 19, 332, 0, 0, 0]), ([2, -1, 0, 0, 0, 1], [100, 7, 500, 300, 15, 16])):
        seq.copy_(i32(s))
        pos.copy_(i32(t))
        q.copy_(torch.randn_like(q))
        torch.cuda.synchronize()
        for _ in range(2):
            g.replay()
        settled()
        want = cc.selection(c, q, means, seq.cpu(), pos.cpu(), S, 1, 2)
        assert torch.equal(pages.cpu(), want[0]) and torch.equal(rows.cpu(), want[1])
        wo, wl, to, tl = cc.selected_reference(c, q, pages, rows, None, None, 0.1)
        assert ((o.double() - wo).abs() <= to).all()
        some = wl > -math.inf
        assert torch.equal(lse == -math.inf, ~some) and ((lse.double() - wl).abs()[some] <= tl[some]).all()


def test_streams_of_their_own():
    Hk, d, page = 2, 64, 16
    c = pc.Cache("bf16", [500], Hk, d, page, seed=26, device="cuda")
    q, means = normal(1, 8, d, seed=27), normal(c.num_pages, Hk, d, seed=28)
    pages, rows = choose(c, q, means, i32([0]), i32([499]), 6, 1, 1)
    want, wl = moda.moda_decode_selected(q, c.k, c.v, pages.cuda(), rows.cuda(), 0.1)
    filled = moda.moda_page_means(*c.args(), i32([0]), i32([15]), torch.zeros_like(means))
    settled()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream, 0):
        got = moda.moda_select_pages(q, means, *c.args(), i32([0]), i32([499]), 6, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got[0].cpu(), pages) and torch.equal(got[1].cpu(), rows)
        o, lse = moda.moda_decode_selected(q, c.k, c.v, *got, 0.1, stream=stream)
        m = moda.moda_page_means(*c.args(), i32([0]), i32([15]), torch.zeros_like(means), stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(lse, wl) and torch.equal(m, filled)
    assert moda.moda_decode_selected(q, c.k, c.v, pages.cuda(), rows.cuda(), 0.1, want_lse=False)[1] is None
