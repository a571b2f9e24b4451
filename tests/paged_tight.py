"""Bounds on the paged decode's output that hold it to the arithmetic that
include/moda.h states, and inputs that show each row of V by itself.

Beside the values of an fp64 pass (test after test compares with them):

  a weight     2^-16 in two bf16 parts (bf16 pages, depth slots), 2^-11 in fp16
               (4-bit pages); where fp16 holds it to less, 2^-31 of the largest
               product of weight and block scale, times codes of at most 6
  a score      ds = (d + 4) 2^-24 scale sum |q k|, absolutely: d products added in fp32;
               2^-19 more for the fast exponential and for rescalings
  a sum        "at least single precision" a step, 2^-23. The rows of a segment go
               to four warps at least in turn, so that an accumulator of n rows takes
               n / 4 steps; twice that where a weight comes in two parts: n 2^-24.
               The sum of weights has fewer
  o            rounded to bf16 once: 2^-8 of the value
"""
from __future__ import annotations

import torch

import paged_common as pc

STEP = 2.0 ** -24


def keys_values(cache, b, n, kd, vd):
    k, v = cache.rows("k", b, n), cache.rows("v", b, n)
    if kd is not None:
        k, v = torch.cat((k, kd[b].double()), 1), torch.cat((v, vd[b].double()), 1)
    return k, v


def one(cache, b, n, q, kd, vd, scale, v=None):
    """fp64 (o [Hk, G, d], its bound) of sequence b with n rows; v in place of its values."""
    Hk, d = cache.Hk, q.shape[-1]
    qb = q[b].double().view(Hk, -1, d)
    k, held = keys_values(cache, b, n, kd, vd)
    v = held if v is None else v
    z = qb @ k.transpose(1, 2) * scale
    p = torch.softmax(z, -1)
    o = p @ v
    ds = ((d + 4) * STEP * scale * (qb.abs() @ k.abs().transpose(1, 2))).amax(-1, keepdim=True)
    rel = torch.full((k.shape[1],), 2.0 ** -16, dtype=torch.float64, device=q.device)
    if cache.fmt == "mx4":
        rel[:n] = pc.HALF_FP16
    a = v.abs()
    tol = pc.HALF_BF16 * o.abs() + (p * rel) @ a + (2 * (ds + 2.0 ** -19) + k.shape[1] * STEP) * (p @ a)
    tol += k.shape[1] * 2.0 ** -126 * a.amax(dim=(1, 2))[:, None, None]
    if cache.fmt == "mx4" and n:
        w = p[..., :n] * cache.block_scales("v", b, n)[:, None]
        tol += n * 6 * 2.0 ** -31 * w.amax(-1, keepdim=True)
    return o, tol


def single_rows(cache, seed):
    """Values of the cache's sequences, all of one length n, such that a column
    of a head has one row that is not zero, and (with n rows at most in all columns
    of all heads and sequences) every row has a column. Returns row [B, Hk, d], -1 for
    columns of nothing."""
    B, Hk, d, n = len(cache.lens), cache.Hk, cache.d, cache.lens[0]
    assert B * Hk * d >= n and all(m == n for m in cache.lens)
    g = torch.Generator().manual_seed(seed)
    row = torch.full((B * Hk * d,), -1, dtype=torch.int64)
    row[torch.randperm(B * Hk * d, generator=g)[:n]] = torch.randperm(n, generator=g)
    row = row.view(B, Hk, d)
    dev = cache.v.device
    b, h, c = (x.to(dev) for x in (row >= 0).nonzero(as_tuple=True))
    r = row.to(dev)[b, h, c]
    page, off = cache.table.long()[b, r // cache.page], r % cache.page
    if cache.fmt == "bf16":
        owned = ~cache.v.isnan()
        cache.v[owned] = 0
        cache.v[page, h, off, c] = (torch.rand(n, generator=g) + 1).bfloat16().to(dev)
    else:
        owned = cache.vs != 255
        cache.v[owned.any(-1)] = 0
        cache.vs[owned] = 1  # what a block of zeros is stored under
        cache.ks[cache.ks != 255] -= 2  # scores of about 1: no row without weight
        code = torch.randint(2, 8, (n,), generator=g, dtype=torch.uint8).to(dev)
        # (two columns of a byte may both be this row's)
        for half in (0, 1):
            of = c % 2 == half
            cache.v[page[of], h[of], off[of], c[of] // 2] |= code[of] << (4 * half)
        cache.vs[page, h, off, c // 32] = 126
    return row.to(dev)
