"""Decode over 4-bit pages whose values' scales lie far apart: what a row counts
for in the softmax has nothing to do with how large its values are. (A block of
zeros is stored under scale byte 1, the largest values under 252.)"""
import math

import pytest
import torch

import sequence_depth_attention_gb300 as moda
from sequence_depth_attention_gb300 import build as mbuild

import paged_common as pc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mbuild.build()
    moda.load()


# Which of a sequence's n rows have large values; the others' are zeros. Runs of
# 32 rows are units of one warp, and long runs whole CTAs.
PLACES = {
    "large last": lambda n: torch.arange(n) >= n // 2,
    "large first": lambda n: torch.arange(n) < n // 2,
    "every other row": lambda n: torch.arange(n) % 2 == 0,
    "every other 32": lambda n: torch.arange(n) // 32 % 2 == 1,
    "the last one": lambda n: torch.arange(n) == n - 1,
    "the first one": lambda n: torch.arange(n) == 0,
}


@pytest.mark.parametrize("least_rows", [0, 16384], ids=["narrow", "wide"])
@pytest.mark.parametrize("spread", [0.0, 1.0], ids=["equal", "spread"])
@pytest.mark.parametrize("e", [60, 100, 125])
@pytest.mark.parametrize("place", PLACES)
def test_zeros_beside_large_values(monkeypatch, place, e, spread, least_rows):
    """lse is the scores' alone, and o the large rows' share of the weight.

    With weights and values of one sign there is no cancellation, so that the
    formula's own rounding errors bound o relatively: a score is off by ds = (d +
    4) 2^-24 scale sum|q k| (a sum of d products in fp32), a weight by 2^-12 (fp16)
    and 2^-19 (fast exponential, rescalings), where it is large enough to be
    held by fp16 in whole; 2^-31 of the largest weight is lost where it is not
    (2^-32, and as much again where values are so large that fp32 holds the
    weights beside them to few bits). A chain of n additions in fp32 adds n 2^-24,
    twice: l and o."""
    monkeypatch.setattr(pc.Cache, "least_rows", least_rows)
    d, Hk, G, page = 128, 2, 4, 16
    lens = [96, 700, 4000]
    c = pc.Cache("mx4", lens, Hk, d, page, seed=40, device="cuda")
    g = torch.Generator().manual_seed(41)
    q = (torch.randn(3, Hk * G, d, generator=g) * spread).bfloat16().cuda()
    for b, n in enumerate(lens):
        large = PLACES[place](n).cuda()
        p = torch.arange(n, device="cuda")
        at, off = c.table[b].long()[p // page], p % page
        # all values 1 .. 6 times 2^e (codes 2 .. 7), or zeros under scale byte 1
        codes = c.v[at, :, off] & 0x77
        codes = torch.where((codes & 0x70) < 0x20, codes | 0x20, codes)
        codes = torch.where((codes & 0x07) < 0x02, codes | 0x02, codes)
        c.v[at, :, off] = torch.where(large[:, None, None], codes, 0)
        scales = torch.where(large, 127 + e, 1).to(torch.uint8)
        c.vs[at, :, off] = scales[:, None, None].expand(-1, Hk, d // 32)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    scale = d ** -0.5
    o, lse = moda.moda_decode_paged(q, *c.args(), n, scale, **c.scales())
    torch.cuda.synchronize()
    assert moda.moda_get_device_error() == 0
    want, want_lse, _, _ = pc.decode_reference(c, q, lens, None, None, scale)
    for b, n in enumerate(lens):
        qb, k = q[b].double().view(Hk, G, d), c.rows("k", b, n)
        z = qb @ k.transpose(1, 2) * scale
        ds = (d + 4) * pc.HALF_FP32 * scale * (qb.abs() @ k.abs().transpose(1, 2)).amax(-1).reshape(-1)
        assert ((lse[b].double() - want_lse[b]).abs() <= ds + n * pc.HALF_FP32 + 2.0 ** -19 +
                want_lse[b].abs() * 2.0 ** -22).all()
        p = torch.exp(z - want_lse[b].view(Hk, G, 1))[..., PLACES[place](n).cuda()]
        lost = (6 * 2.0 ** (e - 31) * p.amax(-1) * p.shape[-1]).reshape(-1, 1)
        rel = (pc.HALF_BF16 + pc.HALF_FP16 + 2 * (ds + 2.0 ** -19 + n * pc.HALF_FP32))[:, None]
        assert ((o[b].double() - want[b]).abs() <= rel * want[b].abs() + lost).all()


@pytest.mark.parametrize("least_rows", [0, 16384], ids=["narrow", "wide"])
@pytest.mark.parametrize("e", [-79, 60, 125])
def test_depth_slots_beside_scaled_rows(monkeypatch, e, least_rows):
    """Depth slots of ordinary values weigh as much as their scores say beside rows
    of tiny or huge ones (tolerances of test_zeros_beside_large_values)."""
    monkeypatch.setattr(pc.Cache, "least_rows", least_rows)
    d, Hk, G, L = 64, 2, 8, 20
    lens = [64, 333]
    c = pc.Cache("mx4", lens, Hk, d, 16, seed=42, device="cuda")
    c.vs[c.vs != 255] = 127 + e
    g = torch.Generator().manual_seed(43)
    q = torch.randn(2, Hk * G, d, generator=g).bfloat16().cuda()
    kd, vd = (torch.randn(2, Hk, L, d, generator=g).bfloat16().cuda() for _ in range(2))
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    scale = d ** -0.5
    o, lse = moda.moda_decode_paged(q, *c.args(), n, scale, kd=kd, vd=vd, **c.scales())
    torch.cuda.synchronize()
    assert moda.moda_get_device_error() == 0
    want, want_lse, _, tol_lse = pc.decode_reference(c, q, lens, kd, vd, scale)
    assert ((lse.double() - want_lse).abs() <= tol_lse).all()
    for b, m in enumerate(lens):
        qb = q[b].double().view(Hk, G, d)
        k = torch.cat((c.rows("k", b, m), kd[b].double()), 1)
        v = torch.cat((c.rows("v", b, m), vd[b].double()), 1)
        z = qb @ k.transpose(1, 2) * scale
        ds = (d + 4) * pc.HALF_FP32 * scale * (qb.abs() @ k.abs().transpose(1, 2)).amax(-1)
        p = torch.exp(z - want_lse[b].view(Hk, G, 1))
        a = (p @ v.abs()).reshape(-1, d)
        lost = (6 * 2.0 ** (e - 31) * p[..., :m].amax(-1) * m).reshape(-1, 1)
        rel = pc.HALF_FP16 + 2 * (ds.reshape(-1, 1) + 2.0 ** -19 + (m + L) * pc.HALF_FP32)
        assert ((o[b].double() - want[b]).abs() <= pc.HALF_BF16 * want[b].abs() + rel * a + lost).all()


@pytest.mark.parametrize("least_rows", [0, 16384], ids=["narrow", "wide"])
def test_scores_of_zero_values_reach_the_sum(monkeypatch, least_rows):
    """All values zero: o = 0 exactly, lse that of the scores, for one sequence and many."""
    monkeypatch.setattr(pc.Cache, "least_rows", least_rows)
    d, Hk = 64, 1
    for lens in ([1], [5000], [33, 0, 1000, 64] * 20):
        c = pc.Cache("mx4", lens, Hk, d, 32, seed=44, device="cuda")
        c.v.zero_()
        c.vs[c.vs != 255] = 1
        q = torch.randn(len(lens), 5, d, generator=torch.Generator().manual_seed(45)).bfloat16().cuda()
        n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        o, lse = moda.moda_decode_paged(q, *c.args(), n, 0.125, **c.scales())
        torch.cuda.synchronize()
        assert moda.moda_get_device_error() == 0
        _, want, _, tol = pc.decode_reference(c, q, lens, None, None, 0.125)
        assert (o == 0).all()
        empty = n == 0
        assert (lse[empty] == -math.inf).all()
        assert ((lse.double() - want).abs() <= tol)[~empty].all()


@pytest.mark.parametrize("least_rows", [0, 16384], ids=["narrow", "wide"])
@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
@pytest.mark.parametrize("e,ev", [(20, 0), (30, 0), (45, 100), (90, 0), (90, -60)])
def test_scores_of_any_size(monkeypatch, fmt, e, ev, least_rows):
    """Keys of 2^e (and values of 2^ev): the row of the highest score has all of the weight, whatever
    fp32 rounds a score by, as long as no other is as near as that. o is that row
    of V, rounded to bf16 once (and by 2^-12 in fp16 over 4-bit pages, with 2^-19
    for what l and o are rescaled by), lse its score."""
    monkeypatch.setattr(pc.Cache, "least_rows", least_rows)
    d, Hk, G, L = 64, 2, 4, 5
    lens = [1, 40, 700, 3000]
    c = pc.Cache(fmt, lens, Hk, d, 16, seed=46, device="cuda")
    if fmt == "mx4":
        c.ks[c.ks != 255] += e
        c.vs[c.vs != 255] += ev % 256
    else:
        c.k.mul_(2.0 ** e)
        c.v.mul_(2.0 ** ev)
    g = torch.Generator().manual_seed(47)
    q = torch.randn(len(lens), Hk * G, d, generator=g).bfloat16().cuda()
    kd, vd = (torch.randn(len(lens), Hk, L, d, generator=g).bfloat16().cuda() for _ in range(2))
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = moda.moda_decode_paged(q, *c.args(), n, 0.125, kd=kd, vd=vd, **c.scales())
    torch.cuda.synchronize()
    assert moda.moda_get_device_error() == 0
    clear = 0
    for b, m in enumerate(lens):
        k = torch.cat((c.rows("k", b, m), kd[b].double()), 1)
        v = torch.cat((c.rows("v", b, m), vd[b].double()), 1)
        qb = q[b].double().view(Hk, G, d)
        z = qb @ k.transpose(1, 2) * 0.125
        ds = (d + 4) * pc.HALF_FP32 * 0.125 * (qb.abs() @ k.abs().transpose(1, 2)).amax(-1)
        top = z.topk(2, -1)
        alone = (top.values[..., 0] - top.values[..., 1] > 2 * ds + 30).reshape(-1)
        clear += int(alone.sum())
        want = torch.gather(v, 1, top.indices[..., :1].expand(-1, -1, d)).reshape(-1, d)
        assert torch.isfinite(o[b]).all() and torch.isfinite(lse[b]).all()
        tol = (pc.HALF_BF16 + pc.HALF_FP16 + 2.0 ** -19) * want.abs() + (m + L) * 2.0 ** -31 * v.abs().max()
        assert ((o[b].double() - want).abs() <= tol)[alone].all()
        high = top.values[..., 0].reshape(-1)
        assert ((lse[b].double() - high).abs() <= ds.reshape(-1) + high.abs() * 2.0 ** -22 + 2.0 ** -19)[alone].all()
    assert clear >= 24  # of 32 heads
