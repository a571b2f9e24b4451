"""Inputs over which an attention output shows single rows of V, and bounds on it that hold the
chunks over the paged cache to the arithmetic that include/moda.h states. Over random values of
both signs an output is small beside the sum of its terms' errors, and a few hundred rows of
tens of thousands are lost in it; here no two terms cancel.

single     a column of V has one row (or one depth slot) that is not zero: its output is one
           weight times one value, off by
             the weight's rounding to bf16                    2^-8
             the output's                                     2^-8   (2^-15: their product, and more)
             the score's, ds = (d + 4) 2^-24 scale |q| |k|, for the weight and the sum of weights,
             2^-19 each for the fast exponential and rescaling
             fp32 sums of n weights                           n 2^-23
           all of the value itself
counted    all scores are 0, so that all weights are 1, and values are 0 or 1: an output is a count
           over a number of rows, both whole numbers below 2^24; it is rounded once, 2^-8, and
           the reciprocal and the product in fp32 take 2^-22. Row r has its 1 in column r % d, and
           of all rows those of a window of 32 d have one, so that a row more or less changes a
           column by 1 / 33 at least."""
from __future__ import annotations

import torch

import paged_common as pc

LEAST = 2.0 ** -90  # far above what underflows, far below any value here


def write(cache, b, h, rows, cols, values):
    """Elements (rows[i], cols[i]) of V of sequence b, KV head h; values: bf16 pages' values, or
    4-bit codes (in bytes that are 0 there)."""
    page, off = cache.table[b].long()[rows // cache.page], rows % cache.page
    if cache.fmt == "bf16":
        cache.v[page, h, off, cols] = values.to(cache.v)
    else:
        for half in (0, 1):
            of = cols % 2 == half
            cache.v[page[of], h, off[of], cols[of] // 2] += values[of].to(torch.uint8) << (4 * half)


def clear(cache):
    """Zeros in all rows of V that sequences own."""
    if cache.fmt == "bf16":
        cache.v[~cache.v.isnan()] = 0
    else:
        cache.v[:] = 0
        cache.vs[cache.vs != 255] = 127


def single(cache, lens, vd, seed):
    """V and vd [L,N,Hk,d] (in place) with one row, or slot of every token, a column of a (sequence, KV
    head) that is not zero: row [B,Hk,d], n + l for slot l."""
    B, Hk, d, L = len(lens), cache.Hk, cache.d, 0 if vd is None else vd.shape[0]
    g = torch.Generator().manual_seed(seed)
    dev = cache.v.device
    clear(cache)
    row = torch.zeros(B, Hk, d, dtype=torch.int64)
    if L:
        vd[~vd.isnan()] = 0
    for h in range(Hk):
        slot = torch.rand(d, generator=g) < (0.2 if L else 0.0)  # of every sequence alike: vd is by token
        of = torch.randint(0, max(1, L), (d,), generator=g)
        if L:
            vd[of[slot].to(dev), :, h, slot.nonzero().flatten().to(dev)] = 1.5
        for b, n in enumerate(lens):
            r = torch.randint(0, n, (d,), generator=g)
            r[: d // 4] = torch.randint(max(0, n - 130), n, (d // 4,), generator=g)  # around the border
            row[b, h] = torch.where(slot, n + of, r)
            cols = (~slot).nonzero().flatten()
            if cache.fmt == "bf16":
                values = torch.rand(len(cols), generator=g) + 1
            else:
                values = torch.randint(1, 8, (len(cols),), generator=g)
            write(cache, b, h, r[cols].to(dev), cols.to(dev), values.to(dev))
    return row


def bound(o, q, cache, starts, lens, kd, scale):
    """Of the outputs o [N,Hq,d] fp64 (paged_chunk_common.prefill_reference) over values of `single`."""
    N, Hq, d = q.shape
    Hk, L = cache.Hk, 0 if kd is None else kd.shape[0]
    tol = torch.full_like(o, float("nan"))
    for b, n in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        if hi == lo:
            continue
        qn = q[lo:hi].double().norm(dim=-1).view(hi - lo, Hk, -1)
        kn = cache.rows("k", b, n).norm(dim=-1).amax(-1)[None].expand(hi - lo, -1)
        if L:
            kn = torch.maximum(kn, kd[:, lo:hi].double().norm(dim=-1).amax(0))
        ds = ((d + 4) * 2.0 ** -24 * scale * qn * kn[..., None]).view(hi - lo, Hq, 1)
        rel = 2 * pc.HALF_BF16 + 2.0 ** -15 + 2 * (ds + 2.0 ** -19) + (n + L) * 2.0 ** -23
        tol[lo:hi] = rel * o[lo:hi].abs() + LEAST
    return tol


def counted(cache, lens, vd, first):
    """Ones in column r % d of the rows from `first` on, 32 d of them; depth slot l has one in
    column l."""
    d, dev = cache.d, cache.v.device
    clear(cache)
    for b, n in enumerate(lens):
        r = torch.arange(min(first, n), min(first + 32 * d, n), device=dev)
        for h in range(cache.Hk):
            write(cache, b, h, r, r % d, torch.ones_like(r) if cache.fmt == "bf16" else torch.full_like(r, 2))
    if vd is not None:
        vd[~vd.isnan()] = 0
        for l in range(vd.shape[0]):
            vd[l, :, :, l] = torch.where(vd[l, :, :, l].isnan(), vd[l, :, :, l], torch.ones_like(vd[l, :, :, l]))


def counts(d, starts, lens, L, first):
    """(outputs [N,1,d] fp64, bounds) of `counted` at scores of 0."""
    c = torch.arange(d)
    o = torch.zeros(starts[-1], 1, d, dtype=torch.float64)
    for b, n in enumerate(lens):
        for i in range(starts[b], starts[b + 1]):
            t = n - (starts[b + 1] - i)  # the token's row
            upto = lambda x: (x - c + d - 1).clamp(min=0) // d  # rows r < x with r % d == c
            rows = upto(min(max(t + 1, first), first + 32 * d)) - upto(first)
            o[i, 0] = (rows + (c < L)).double() / (t + 1 + L)
    return o, o * (pc.HALF_BF16 + 2.0 ** -21)
