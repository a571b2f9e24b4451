"""Plain fp64 forms of the paged cache's operators and inputs for their tests.
Written from the operators' definitions; nothing here calls the library."""
from __future__ import annotations

import math

import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2
HALF_FP16 = torch.finfo(torch.float16).eps / 2
HALF_FP32 = torch.finfo(torch.float32).eps / 2


class Cache:
    """A pool of pages with random rows and a table of randomly placed pages.
    lens: rows of each sequence that must have pages. fill: what every row
    that no sequence owns holds ("nan": NaN, and scale bytes of NaN)."""

    least_rows = 0  # columns of the table for as many rows at least

    def __init__(self, fmt, lens, Hk, d, page, seed=0, width=None, spare=2, fill="nan", device="cpu"):
        g = torch.Generator().manual_seed(seed)
        self.fmt, self.Hk, self.d, self.page, self.lens = fmt, Hk, d, page, list(lens)
        held = [-(-n // page) for n in lens]
        self.num_pages = sum(held) + spare
        self.max_pages = (max(1, max(held, default=0), -(-self.least_rows // page)) if width is None
                          else width)
        order = torch.randperm(self.num_pages, generator=g).to(torch.int32)
        # entries past a sequence's end name no page at all
        self.table = torch.full((len(lens), self.max_pages), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(held):
            self.table[b, :n] = order[at : at + n]
            at += n
        shape = (self.num_pages, Hk, page, d)
        if fmt == "bf16":
            self.k = torch.randn(shape, generator=g).bfloat16()
            self.v = torch.randn(shape, generator=g).bfloat16()
            self.ks = self.vs = None
        else:
            self.k, self.v = (torch.randint(0, 256, (*shape[:3], d // 2), generator=g,
                                            dtype=torch.uint8) for _ in range(2))
            self.ks, self.vs = (torch.randint(124, 129, (*shape[:3], d // 32), generator=g,
                                              dtype=torch.uint8) for _ in range(2))
        if fill == "nan":
            owned = torch.zeros(self.num_pages, page, dtype=torch.bool)
            for b, n in enumerate(lens):
                for p in range(held[b]):
                    owned[self.table[b, p], : min(page, n - p * page)] = True
            free = ~owned[:, None, :].expand(-1, Hk, -1)
            if fmt == "bf16":
                self.k[free] = math.nan
                self.v[free] = math.nan
            else:
                self.ks[free] = 255
                self.vs[free] = 255
        for n in ("table", "k", "v", "ks", "vs"):
            t = getattr(self, n)
            if t is not None:
                setattr(self, n, t.to(device))

    def args(self):
        return (self.k, self.v, self.table)

    def scales(self):
        return dict(k_scales=self.ks, v_scales=self.vs)

    def bits(self):
        return [t.clone() for t in (self.k, self.v, self.ks, self.vs) if t is not None]

    def rows(self, which, b, n):
        """[Hk, n, d] fp64: the first n rows of sequence b."""
        ids = self.table[b, : -(-n // self.page)].long()
        x = getattr(self, which)[ids]
        x = x.double() if self.fmt == "bf16" else mx4_values(x, getattr(self, which + "s")[ids])
        return x.transpose(0, 1).reshape(self.Hk, -1, self.d)[:, :n]

    def block_scales(self, which, b, n):
        """[Hk, n] fp64: the largest block scale of each of the first n rows."""
        ids = self.table[b, : -(-n // self.page)].long()
        s = torch.exp2(getattr(self, which + "s")[ids].double() - 127).amax(-1)
        return s.transpose(0, 1).reshape(self.Hk, -1)[:, :n]


def mx4_values(codes, scales):
    """fp64 values of 4-bit rows; a scale byte of 255 is NaN."""
    lut = torch.cat((E2M1, -E2M1)).to(codes.device)
    x = torch.stack((lut[(codes & 15).long()], lut[(codes >> 4).long()]), -1).flatten(-2)
    s = torch.exp2(scales.double() - 127)
    s = torch.where(scales == 255, torch.full_like(s, math.nan), s)
    return (x.reshape(*scales.shape, 32) * s.unsqueeze(-1)).reshape(x.shape)


def mx4_quantised(x):
    """The values that 4-bit rows hold for fp64 rows x[..., d]."""
    blk = x.reshape(-1, 32)
    big = blk.abs().amax(1)
    fine = torch.isfinite(big)
    E = torch.full_like(big, -126.0)
    for e in range(-125, 126):  # the smallest 2^E whose sevenfold reaches the largest magnitude
        E = torch.where(fine & (big > 7 * 2.0 ** (e - 1)), torch.full_like(E, float(e)), E)
    t = blk.abs() / torch.exp2(E)[:, None]
    lut = E2M1.to(x.device)
    gap = (t[..., None] - lut).abs()
    best = gap.amin(-1, keepdim=True)
    tied = gap == best
    even = torch.tensor([1, 0, 1, 0, 1, 0, 1, 0], dtype=torch.bool, device=x.device)
    pick = torch.where((tied & even).any(-1), (tied & even).int().argmax(-1), tied.int().argmax(-1))
    y = torch.copysign(lut[pick], blk) * torch.exp2(E)[:, None]
    y = torch.where(fine[:, None], y, torch.full_like(y, math.nan))
    return y.reshape(x.shape)


def turned(x, rope, pos, interleaved):
    """x[N,H,d] in fp64 with its pairs turned by row pos[n] of rope[P,rot]."""
    x = x.double().clone()
    half = rope.shape[1] // 2
    c, s = (t[:, None] for t in rope[pos.long()].double().split(half, 1))
    i = torch.arange(half, device=x.device)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = x[..., lo], x[..., hi]
    x[..., lo], x[..., hi] = a * c - b * s, b * c + a * s
    return x


def rope_table(P, rot, base=10000.0):
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(P, dtype=torch.float64)[:, None] * f
    return torch.cat((a.cos(), a.sin()), 1).float()


def decode_reference(cache, q, lens, kd, vd, scale):
    """fp64 (o, lse, tol_o, tol_lse) of the paged decode, and how far a kernel
    that follows the documented arithmetic may be from them.

    A score is a sum of d products in fp32: off by at most ds = (d + 4) 2^-24
    scale sum|q k| (absolutely, so exp of it relatively). A probability is
    rounded once to bf16 (2^-8), at worst, and carries 2^-20 for the fast
    exponential and the rescaling by powers of the running maximum's steps.
    o divides the weighted sum by the sum of weights, each off by that much,
    and is rounded to bf16; both sums add n + L terms in fp32.
    What rounding relative to the value does not cover is underflow. In fp32 a
    weight exp(z - max z) below 2^-126 may become 0: with the sum of weights at
    least 1, o is off by at most n 2^-126 max|v|. Over 4-bit pages a weight
    times its block scale is held in fp16 with the largest of all at 2^7 or
    more, so it is off by 2^-25 there, 2^-32 of the largest product of
    probability and block scale, times codes of at most 6."""
    B, Hq, d = q.shape
    Hk = cache.Hk
    out = [], [], [], []
    for b in range(B):
        qb = q[b].double().view(Hk, Hq // Hk, d)
        k, v = cache.rows("k", b, lens[b]), cache.rows("v", b, lens[b])
        if kd is not None:
            k, v = torch.cat((k, kd[b].double()), 1), torch.cat((v, vd[b].double()), 1)
        n = k.shape[1]
        if n == 0:
            zero = torch.zeros_like(qb)
            lse = torch.full(qb.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
            for got, x in zip(out, (zero, lse, zero, torch.zeros_like(lse))):
                got.append(x.reshape(Hq, -1) if x.dim() == 3 else x.reshape(Hq))
            continue
        z = qb @ k.transpose(1, 2) * scale
        lse = torch.logsumexp(z, -1)
        p = torch.exp(z - lse[..., None])
        o, a = p @ v, p @ v.abs()
        ds = ((d + 4) * 2.0 ** -24 * scale * (qb.abs() @ k.abs().transpose(1, 2))).amax(-1)
        rel = HALF_BF16 + ds + 2.0 ** -20
        tol_o = HALF_BF16 * o.abs() + (2 * rel + n * 2.0 ** -23)[..., None] * a
        tol_o += n * 2.0 ** -126 * v.abs().amax(dim=(1, 2))[:, None, None]
        if cache.fmt == "mx4" and lens[b]:
            w = p[..., : lens[b]] * cache.block_scales("v", b, lens[b])[:, None]
            tol_o += n * 6 * 2.0 ** -32 * w.amax(-1, keepdim=True)
        tol_lse = ds + n * 2.0 ** -24 + lse.abs() * 2.0 ** -22 + 2.0 ** -19
        for got, x in zip(out, (o, lse, tol_o, tol_lse)):
            got.append(x.reshape(Hq, -1) if x.dim() == 3 else x.reshape(Hq))
    return tuple(torch.stack(x) for x in out)
