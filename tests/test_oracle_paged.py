"""The bounds of paged_tight.py on the CPU: they hold the fp64 values themselves, and
mistakes planted in those do not pass."""
import pytest
import torch

import paged_common as pc
import paged_tight as pt


def queries(B, Hq, d, seed):
    return torch.randn(B, Hq, d, generator=torch.Generator().manual_seed(seed)).bfloat16()


@pytest.mark.parametrize("fmt,n", [("bf16", 64), ("bf16", 1000), ("mx4", 64)])
def test_a_row_left_out_is_seen(fmt, n):
    """Among random values, as far as a worst-case bound on their sum shows one."""
    c = pc.Cache(fmt, [n], 1, 128, 16, seed=1)
    if fmt == "mx4":
        c.ks[c.ks != 255] -= 2  # scores of about 1
    q = queries(1, 2, 128, 2)
    o, tol = pt.one(c, 0, n, q, None, None, 128 ** -0.5)
    v = c.rows("v", 0, n)
    for j in list(range(0, n, max(1, n // 61))) + [n - 1]:
        less = v.clone()
        less[:, j] = 0
        wrong, _ = pt.one(c, 0, n, q, None, None, 128 ** -0.5, v=less)
        assert ((wrong - o).abs() > tol).any(), j


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
@pytest.mark.parametrize("n", [4097, 9003])
def test_any_single_row_left_out_is_seen(fmt, n):
    d, Hk = 128, 2
    B = -(-n // (Hk * d))
    c = pc.Cache(fmt, [n] * B, Hk, d, 32, seed=3)
    row = pt.single_rows(c, 4)
    q = queries(B, 2 * Hk, d, 5)
    for b in range(B):
        o, tol = pt.one(c, b, n, q, None, None, d ** -0.5)
        assert (o.abs() > tol).all(1)[row[b] >= 0].all()


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
@pytest.mark.parametrize("n", [1000, 4097, 9003])
def test_exchanged_rows_are_seen(fmt, n):
    """Single rows at a time: nearly every exchange of a row with one of its
    neighbours, of the next tile or of the next unit (only weights that are alike within
    o's own rounding may pass)."""
    d, Hk = 128, 2
    B = -(-n // (Hk * d))
    c = pc.Cache(fmt, [n] * B, Hk, d, 32, seed=3)
    row = pt.single_rows(c, 4)
    q = queries(B, 2 * Hk, d, 5)
    seen = dict.fromkeys((1, 2, 8, 16, 32, 64), 0)
    for b in range(B):
        o, tol = pt.one(c, b, n, q, None, None, d ** -0.5)
        v = c.rows("v", b, n)
        for by in seen:
            to = torch.arange(n) ^ by
            to = torch.where(to < n, to, torch.arange(n))
            wrong, _ = pt.one(c, b, n, q, None, None, d ** -0.5, v=v[:, to])
            seen[by] += int(((wrong - o).abs() > tol).any(1)[row[b] >= 0].sum())
    assert all(x > 0.95 * n for x in seen.values()), seen


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
def test_single_rows_hold_every_row_once(fmt):
    n, d, Hk = 700, 64, 2
    c = pc.Cache(fmt, [n] * 6, Hk, d, 16, seed=6)
    row = pt.single_rows(c, 7)
    assert sorted(row[row >= 0].tolist()) == list(range(n))
    for b in range(6):
        v = c.rows("v", b, n)
        there = v != 0
        assert torch.equal(there.sum(1), (row[b] >= 0).long())
        h, col = (row[b] >= 0).nonzero(as_tuple=True)
        assert there[h, row[b][h, col], col].all()


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
def test_weights_of_fewer_bits_are_seen(fmt):
    """Weights rounded to bf16 once, where two parts (bf16 pages) or fp16 (4-bit
    pages) are promised, pass the bound of neither, with values of one sign."""
    n, d, Hk = 300, 64, 2
    c = pc.Cache(fmt, [n], Hk, d, 16, seed=8)
    if fmt == "bf16":
        c.v = c.v.abs()
    else:
        c.v = c.v & 0x77
        c.ks[c.ks != 255] -= 2
    q = queries(1, 4, d, 9)
    o, tol = pt.one(c, 0, n, q, None, None, d ** -0.5)
    k, v = pt.keys_values(c, 0, n, None, None)
    z = q[0].double().view(Hk, -1, d) @ k.transpose(1, 2) * d ** -0.5
    p = torch.exp(z - z.amax(-1, keepdim=True))
    wrong = torch.stack([(p * (1 + s * pc.HALF_BF16)) @ v / p.sum(-1, keepdim=True) for s in (-1, 1)])
    # the bound itself is mostly o's own rounding: without it
    left = tol - pc.HALF_BF16 * o.abs()
    assert ((wrong - o).abs() > left).all()
