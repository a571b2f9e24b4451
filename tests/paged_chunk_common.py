"""Plain fp64 forms of the operators over chunks of new tokens and over selected pages,
and inputs for their tests. Written from the operators' definitions; nothing here calls
the library."""
from __future__ import annotations

import math

import torch

import paged_common as pc


def attention(q, k, v, seen, scale, mx4_products=None):
    """fp64 (o, lse, tol_o, tol_lse) of queries q[R,d] over keys and values [n,d] (both
    fp64, or [R,n,d] where every query has its own), of which row r sees `seen[r]`.

    The bounds are those of paged_common.decode_reference: scores are sums of d products
    in fp32, a weight is rounded once to bf16 and carries 2^-20 for the fast exponential
    and for rescaling, sums of n terms are in fp32, a weight below 2^-126 of the largest
    may count as 0, and o is rounded to bf16. mx4_products [R,n]: the probabilities'
    factors of the products that the 4-bit decode holds in fp16 (block scales)."""
    R, d = q.shape
    if k.dim() == 2:
        k, v = k[None], v[None]
    hidden = ~seen
    k = torch.where(hidden[..., None], 0.0, k)  # whatever it holds
    v = torch.where(hidden[..., None], 0.0, v)
    z = (q[:, None] * k).sum(-1) * scale
    z = z.masked_fill(hidden, -math.inf)
    n = seen.sum(-1)
    lse = torch.logsumexp(z, -1) if z.shape[-1] else torch.full((R,), -math.inf, dtype=torch.float64, device=q.device)
    some = n > 0
    p = torch.where(some[:, None], torch.exp(z - torch.where(some, lse, 0.0)[:, None]), 0.0)
    o = (p[:, None] @ v)[:, 0]
    a = (p[:, None] @ v.abs())[:, 0]
    ds = ((d + 4) * 2.0 ** -24 * scale * (q.abs()[:, None] * k.abs()).sum(-1)).masked_fill(hidden, 0.0)
    ds = ds.amax(-1) if ds.shape[-1] else torch.zeros_like(lse)
    rel = pc.HALF_BF16 + ds + 2.0 ** -20
    tol_o = pc.HALF_BF16 * o.abs() + (2 * rel + n * 2.0 ** -23)[:, None] * a
    if v.shape[1]:
        tol_o += (n * 2.0 ** -126)[:, None] * v.abs().amax(dim=(1, 2))[:, None]
    if mx4_products is not None and z.shape[-1]:
        tol_o += (n * 6 * 2.0 ** -32 * (p * mx4_products).amax(-1))[:, None]
    tol_lse = ds + n * 2.0 ** -24 + torch.where(some, lse, 0.0).abs() * 2.0 ** -22 + 2.0 ** -19
    return o, lse, tol_o, tol_lse


def prefill_reference(cache, q, q_starts, lens, kd, vd, scale):
    """attention() for the tokens q_starts[b] .. q_starts[b+1]-1 of each sequence, its last
    rows; kd, vd [L,N,Hk,d] or None. Rows of tokens of no sequence come back as NaN."""
    N, Hq, d = q.shape
    Hk = cache.Hk
    G = Hq // Hk
    f64 = dict(dtype=torch.float64, device=q.device)
    o, tol_o = (torch.full((N, Hq, d), math.nan, **f64) for _ in range(2))
    lse, tol_lse = (torch.full((N, Hq), math.nan, **f64) for _ in range(2))
    for b, n in enumerate(lens):
        lo, hi = q_starts[b], q_starts[b + 1]
        m = hi - lo
        if m == 0:
            continue
        t = torch.arange(n - m, n, device=q.device)
        k, v = cache.rows("k", b, n), cache.rows("v", b, n)
        step = max(1, int(3e7 // (G * d * (n + 1))))
        for i0 in range(0, m, step):
            here = slice(lo + i0, min(hi, lo + i0 + step))
            c = here.stop - here.start
            for h in range(Hk):
                heads = slice(h * G, (h + 1) * G)
                kk, vv = k[h][None].expand(c, -1, -1), v[h][None].expand(c, -1, -1)
                seen = torch.arange(n, device=q.device) <= t[i0 : i0 + c, None]
                if kd is not None:
                    kk = torch.cat((kk, kd[:, here, h].double().transpose(0, 1)), 1)
                    vv = torch.cat((vv, vd[:, here, h].double().transpose(0, 1)), 1)
                    seen = torch.cat((seen, torch.ones(c, kd.shape[0], dtype=torch.bool, device=q.device)), 1)
                args = [x.repeat_interleave(G, 0) for x in (kk, vv, seen)]
                got = attention(q[here, heads].double().reshape(-1, d), *args, scale)
                for to, x in zip((o, lse, tol_o, tol_lse), got):
                    to[here, heads] = x.view(c, G, *x.shape[1:])
    return o, lse, tol_o, tol_lse


def page_means(cache):
    """[num_pages,Hk,d] fp64: every page's mean key."""
    k = cache.k.double() if cache.fmt == "bf16" else pc.mx4_values(cache.k, cache.ks)
    return k.mean(2)


def selection(cache, q, means, seq, pos, S, sink, recent):
    """(pages[N,Hk,S], rows[N,Hk]) of moda_select_pages, scores in fp64 by a sum from the
    first element to the last."""
    N, Hk = q.shape[0], cache.Hk
    G, d = q.shape[1] // Hk, q.shape[2]
    q, means, table = q.double().cpu(), means.double().cpu(), cache.table.cpu()
    pages = torch.full((N, Hk, S), -1, dtype=torch.int32)
    rows = torch.zeros((N, Hk), dtype=torch.int32)
    for n in range(N):
        b, t = int(seq[n]), int(pos[n])
        if b < 0:
            continue
        m = t // cache.page + 1
        ids = table[b, :m].long()
        for h in range(Hk):
            score = torch.full((m,), -math.inf, dtype=torch.float64)
            for g in range(G):
                s = (q[n, h * G + g] * means[ids, h]).sum(-1)
                score = torch.where(torch.isnan(s), score, torch.maximum(score, s))
            always = [i for i in range(m) if i < sink or i >= m - recent] if m > S else list(range(m))
            rest = sorted(set(range(m)) - set(always), key=lambda i: (-score[i].item(), i))
            keep = sorted(always + rest[: max(0, S - len(always))])
            pages[n, h, : len(keep)] = (ids[keep] * Hk + h).int()
            rows[n, h] = (len(keep) - 1) * cache.page + t % cache.page + 1
    return pages, rows


def selected_reference(cache, q, pages, rows, kd, vd, scale):
    """attention() for every (token, KV head) over the first rows[n,hk] rows of its row
    blocks; kd, vd [N,Hk,L,d] or None."""
    N, Hq, d = q.shape
    Hk = cache.Hk
    G = Hq // Hk
    outs = [], [], [], []
    for n in range(N):
        for h in range(Hk):
            r = int(rows[n, h])
            ids = pages[n, h, : -(-r // cache.page)].long()
            kv = []
            for x, s in ((cache.k, cache.ks), (cache.v, cache.vs)):
                x = x.flatten(0, 1)[ids]
                x = x.double() if s is None else pc.mx4_values(x, s.flatten(0, 1)[ids])
                kv.append(x.reshape(-1, d)[:r] if r else torch.zeros(0, d, dtype=torch.float64, device=q.device))
            scales = None
            if cache.fmt == "mx4" and r:
                scales = torch.exp2(cache.vs.flatten(0, 1)[ids].double() - 127).amax(-1).reshape(-1)[:r]
                scales = torch.cat((scales, scales.new_zeros(0 if kd is None else kd.shape[2])))[None]
            if kd is not None:
                kv = [torch.cat((x, y[n, h].double())) for x, y in zip(kv, (kd, vd))]
            seen = torch.ones(G, kv[0].shape[0], dtype=torch.bool, device=q.device)
            got = attention(q[n, h * G : (h + 1) * G].double(), *kv, seen, scale, mx4_products=scales)
            for to, x in zip(outs, got):
                to.append(x)
    return tuple(torch.cat(x).view(N, Hq, *x[0].shape[1:]) for x in outs)
