"""Single rows of V in the outputs of chunks and of attention over selected pages, under bounds
that a row, a page, a block or a partial result too few or in another's place does not pass
(tests/paged_chunk_tight.py, tests/paged_tight.py); and what a NaN key makes of its readers."""
import math

import pytest
import torch

import sequence_depth_attention_gb300 as moda
import paged_chunk_common as cc
import paged_chunk_tight as tight
import paged_common as pc
import paged_tight
from test_gpu_paged_chunk import _built, chunk, i32, plant, run, settled  # noqa: F401 (_built is a fixture)

pytestmark = pytest.mark.gpu
FORMATS = pytest.mark.parametrize("fmt,d", [(f, d) for f in ("bf16", "mx4") for d in (64, 128)])

CHUNKS = [  # new tokens, rows before them, Hq, Hk, L, page
    ([5], [696], 16, 4, 46, 64),
    ([40, 3], [500, 9000], 16, 1, 5, 16),
    ([130, 1, 33], [20, 255, 4000], 8, 2, 3, 32),
    ([3, 1, 20], [30000, 0, 9000], 16, 1, 2, 128),
    ([9, 18], [260, 1000], 6, 2, 0, 16),
]


@FORMATS
@pytest.mark.parametrize("case", CHUNKS, ids=lambda c: f"{len(c[0])}x{max(c[1])}-" + "-".join(map(str, c[2:])))
def test_single_rows_of_chunks(fmt, d, case):
    new, past, Hq, Hk, L, page = case
    for seed in (1, 2, 3):
        c, q, starts, lens, kd, vd = x = chunk(fmt, new, past, Hq, Hk, d, L, page, seed=seed)
        tight.single(c, lens, vd, seed)
        want = cc.prefill_reference(*x, d ** -0.5)[0]
        tol = tight.bound(want, q, c, starts, lens, kd, d ** -0.5)
        o, _ = run(*x, d ** -0.5)
        assert ((o.double() - want).abs() <= tol).all()


@FORMATS
@pytest.mark.parametrize("new,past,Hq,L,page", [
    ([3, 1, 20], [30000, 0, 9000], 16, 2, 128), ([200], [1900], 4, 0, 16), ([7, 9], [65536, 100], 2, 33, 64)])
def test_every_row_of_chunks_counts_once(fmt, d, new, past, Hq, L, page):
    c, q, starts, lens, kd, vd = x = chunk(fmt, new, past, Hq, 1, d, L, page)
    q[:] = 0
    if L:
        kd[:] = 0
    for first in range(0, max(lens), 32 * d):
        tight.counted(c, lens, vd, first)
        o, lse = run(*x, d ** -0.5)
        want, tol = (t.cuda() for t in tight.counts(d, starts, lens, L, first))
        assert ((o.double() - want).abs() <= tol).all()
    n = torch.cat([torch.arange(b - m, b) for b, m in zip(lens, new)]) + 1 + L
    assert ((lse.double().cpu() - n.double().log()[:, None]).abs() <= 2.0 ** -19 * (1 + n.double().log()[:, None])).all()


SELECTED = [  # tokens, Hk, G, rows, L, page
    (4, 2, 4, 500, 3, 16), (1, 4, 8, 256, 24, 64), (16, 4, 8, 1024, 5, 16), (40, 2, 16, 2048, 0, 32),
    (2, 1, 3, 100, 1, 128),
]


@FORMATS
@pytest.mark.parametrize("case,shown", [(c, s) for c in SELECTED for s in ("rows", "slots") if c[4] or s == "rows"],
                         ids=lambda x: x if isinstance(x, str) else "-".join(map(str, x)))
def test_single_rows_of_selected_pages(fmt, d, case, shown):
    N, Hk, G, n, L, page = case
    c = pc.Cache(fmt, [n] * (N * Hk), 1, d, page, seed=21, device="cuda", spare=2 * Hk)
    if shown == "rows":
        row = paged_tight.single_rows(c, 22)
        assert (row >= 0).sum() == n  # every row has a column
    else:
        tight.clear(c)
    g = torch.Generator().manual_seed(23)
    q = (torch.randn(N, Hk * G, d, generator=g) * (1 if fmt == "bf16" else 0.5)).bfloat16().cuda()
    kd = vd = None
    if L:
        kd, vd = (torch.randn(N, Hk, L, d, generator=g).bfloat16().cuda() for _ in range(2))
        of = torch.randint(0, L, (N, Hk, 1, d), generator=g).cuda()
        at = torch.arange(L, device="cuda")[:, None] == of
        vd = torch.where(at & (shown == "slots"), vd.abs() + 1, 0.0).bfloat16()
    # the pool's row blocks in pages of Hk blocks
    extra = -c.num_pages % Hk
    pool = [None if x is None else torch.cat((x, x[:1].expand(extra, -1, -1, -1))).reshape(-1, Hk, *x.shape[2:])
            for x in (c.k, c.v, c.ks, c.vs)]
    S = c.max_pages
    o, _ = moda.moda_decode_selected(q, pool[0], pool[1], c.table.view(N, Hk, S), i32([[n] * Hk] * N), d ** -0.5, kd=kd,
                                     vd=vd, k_scales=pool[2], v_scales=pool[3])
    settled()
    flat = [None if x is None else x.reshape(N * Hk, 1, L, d) for x in (kd, vd)]
    qs = q.view(N * Hk, G, d)
    for b in range(N * Hk):
        want, tol = paged_tight.one(c, b, n, qs, *flat, d ** -0.5)
        got = o.view(N * Hk, G, d)[b].double()
        assert ((got - want[0]).abs() <= tol[0]).all()
        assert (want[0] > 0).any()


# ------------------------------------------------------------------ NaN keys
def within(o, lse, wo, wl, to, tl, where):
    """Values, not bits: rows of a warp raise their reference together."""
    assert ((o.double() - wo).abs() <= to)[where].all() and ((lse.double() - wl).abs() <= tl)[where].all()


@FORMATS
def test_a_nan_key_is_seen_by_its_readers_alone(fmt, d):
    new, past, Hk, G, L = [150, 9, 40], [20, 250, 0], 2, 4, 5
    x = chunk(fmt, new, past, Hk * G, Hk, d, L, 16)
    c, q, starts, lens, kd, vd = x
    wo, wl, to, tl = cc.prefill_reference(*x, d ** -0.5)
    for b, t in ((0, 3), (0, 100), (0, 169), (1, 255), (2, 0), (2, 39)):
        for hk in range(Hk):
            c2 = pc.Cache(fmt, lens, Hk, d, 16, seed=1, device="cuda")
            plant(c2, b, t, "k", math.nan, hk=hk)
            o, lse = run(c2, *x[1:], d ** -0.5)
            hit = torch.zeros_like(lse, dtype=torch.bool)
            hit[starts[b] + max(0, t - past[b]) : starts[b + 1], hk * G : (hk + 1) * G] = True
            assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
            within(o, lse, wo, wl, to, tl, ~hit)
    for token, slot, hk in ((0, 0, 0), (33, 4, 1), (198, 2, 1)):  # of a token's own slots
        k2 = kd.clone()
        k2[slot, token, hk, d - 1] = math.nan
        o, lse = run(c, q, starts, lens, k2, vd, d ** -0.5)
        hit = torch.zeros_like(lse, dtype=torch.bool)
        hit[token, hk * G : (hk + 1) * G] = True
        assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
        within(o, lse, wo, wl, to, tl, ~hit)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [math.inf, -math.inf])
def test_an_infinite_key_is_seen_by_its_readers_alone(d, value):
    """A score of +infinity makes a NaN of its reader; one of -infinity is no weight, as if the
    key were not there."""
    new, past, Hk, G, L = [150, 9], [20, 250], 2, 4, 5
    x = chunk("bf16", new, past, Hk * G, Hk, d, L, 16)
    c, q, starts, lens, kd, vd = x
    wo, wl, to, tl = cc.prefill_reference(*x, d ** -0.5)
    for b, t in ((0, 100), (1, 255)):
        c2 = pc.Cache("bf16", lens, Hk, d, 16, seed=1, device="cuda")
        plant(c2, b, t, "k", value, hk=1)
        o, lse = run(c2, *x[1:], d ** -0.5)
        reads = torch.zeros_like(lse, dtype=torch.bool)
        reads[starts[b] + t - past[b] : starts[b + 1], G:] = True
        sign = q[..., 5].double() * value  # of the score
        within(o, lse, wo, wl, to, tl, ~reads)
        assert torch.isnan(o[reads & (sign > 0)]).all()
        gone = reads & (sign < 0)
        # the key's weight taken from the softmax without it
        k = c.rows("k", b, lens[b])[1, t]
        p = torch.exp((q.double() * k).sum(-1) * d ** -0.5 - wl)[..., None]
        v = c.rows("v", b, lens[b])[1, t]
        left = (wo - p * v) / (1 - p)
        assert (sign[reads] != 0).all() and gone.any() and (p[gone] < 0.5).all()
        # (the bounds without it: of weights and sums as much larger)
        assert ((o.double() - left).abs() <= (to + pc.HALF_BF16 * left.abs()) / (1 - p))[gone].all()
        assert ((lse.double() - (wl + torch.log1p(-p[..., 0]))).abs() <= 2 * tl)[gone].all()
