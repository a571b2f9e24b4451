"""The bounds of tests/paged_chunk_tight.py reject outputs of planted mistakes."""
import pytest
import torch

import paged_chunk_common as cc
import paged_chunk_tight as tight
import paged_common as pc


def case(fmt, new, past, d=64, Hk=2, G=2, L=3, seed=1):
    lens = [n + p for n, p in zip(new, past)]
    c = pc.Cache(fmt, lens, Hk, d, 16, seed=seed)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(starts[-1], Hk * G, d, generator=g).bfloat16()
    kd, vd = (torch.randn(L, starts[-1], Hk, d, generator=g).bfloat16() for _ in range(2))
    return c, q, starts, lens, kd, vd


def outside(got, want, tol):
    return ~((got - want).abs() <= tol)


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
@pytest.mark.parametrize("seed", [1, 2])
def test_single_rows(fmt, seed):
    c, q, starts, lens, kd, vd = x = case(fmt, [6, 3], [300, 40], seed=seed)
    row = tight.single(c, lens, vd, seed)
    want = cc.prefill_reference(*x, 0.125)[0]
    tol = tight.bound(want, *(x[i] for i in (1, 0, 2, 3, 4)), 0.125)
    # every column is one weight times one value
    G = q.shape[1] // c.Hk
    for n in range(starts[-1]):
        b = 0 if n < starts[1] else 1
        t = lens[b] - (starts[b + 1] - n)
        seen = (row[b] <= t) | (row[b] >= lens[b])
        assert ((want[n].view(c.Hk, G, -1) > 0) == seen[:, None]).all()
    assert (tol[want > 0] / want[want > 0] < 2.1 * 2 * pc.HALF_BF16).all()

    def changed(f):
        """Which outputs f's change of V moves out of their bounds, and which it moves at all."""
        kept = c.v.clone()
        f()
        got = cc.prefill_reference(*x, 0.125)[0]
        c.v.copy_(kept)
        return outside(got, want, tol), got != want

    pages = c.table[0].long()
    blocks = lambda i: pages[8 * i : 8 * i + 8]  # 128 rows
    for i in (0, 1):
        out, moved = changed(lambda: c.v.index_fill_(0, blocks(i), 0))  # a block left out
        assert moved.any() and torch.equal(out, moved)
    for i, j in ((0, 1), (2, 9), (5, 18)):  # a page in another's place: other weights
        out, moved = changed(lambda: c.v.index_copy_(0, pages[[i, j]], c.v[pages[[j, i]]].clone()))
        assert moved.any() and out.sum() > 0.9 * moved.sum()
    out, moved = changed(lambda: c.v.copy_(c.v.roll(1, 2)))  # a row further
    assert out.sum() > 0.9 * moved.sum() > 0
    # another token's slots, another slot's key
    slot = (row >= torch.tensor(lens)[:, None, None]).repeat_interleave(G, 1)[0].expand(starts[1], -1, -1)
    assert slot.any()
    for other in (kd.roll(1, 1), kd.roll(1, 0)):
        got = cc.prefill_reference(c, q, starts, lens, other, vd, 0.125)[0]
        assert outside(got, want, tol)[: starts[1]][slot].float().mean() > 0.9
    # a partial result lost in a join: its weights stay in the sum, its O does not
    scaled = want * (1 - 2.0 ** -5)
    assert torch.equal(outside(scaled, want, tol), want > 0)


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
@pytest.mark.parametrize("first", [0, 2048, 4096])
def test_counted_rows(fmt, first):
    c, q, starts, lens, kd, vd = x = case(fmt, [3, 1, 2], [5000, 0, 130], Hk=1, G=1)
    q.zero_()
    tight.counted(c, lens, vd, first)
    want, tol = tight.counts(c.d, starts, lens, 3, first)
    assert torch.allclose(cc.prefill_reference(*x, 0.125)[0], want, rtol=1e-12, atol=0)
    pages = c.table[0].long()
    for at in (first // 16, min(len(pages), (first + 2048) // 16) - 9):  # a page, a block of 128 rows, a row
        for f in (lambda: c.v.index_fill_(0, pages[at : at + 1], 0), lambda: c.v.index_fill_(0, pages[at : at + 8], 0),
                  lambda: c.v[pages[at], :, 3].zero_()):
            kept = c.v.clone()
            f()
            got = cc.prefill_reference(*x, 0.125)[0]
            c.v.copy_(kept)
            out, moved = outside(got, want, tol), outside(got, want, want * 1e-12)
            assert moved[: starts[1]].any() and torch.equal(out, moved)
