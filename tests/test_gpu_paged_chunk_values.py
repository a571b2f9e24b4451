"""Chunks of new tokens over values at the ends of their range: sums of the largest 4-bit
values, and the smallest ones."""
import math

import pytest
import torch

import sequence_depth_attention_gb300 as moda
import paged_chunk_common as cc
import paged_common as pc
from test_gpu_paged_chunk import _built, check, chunk, i32, run, settled  # noqa: F401 (_built is a fixture)

pytestmark = pytest.mark.gpu
LARGEST = 252  # of the scale bytes that moda_kv_append writes: values up to 6 * 2^125


def held(c, which):
    """Scale bytes of the rows that sequences own, as a mask."""
    return getattr(c, which) != 255


SHAPES = [  # new tokens, rows before them, G, L
    ([1], [1], 4, 0), ([5, 40], [3, 700], 4, 3), ([70, 2, 1], [0, 5, 16000], 8, 5),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("signs", [False, True])
@pytest.mark.parametrize("new,past,G,L", SHAPES)
def test_sums_of_the_largest_values(new, past, G, L, signs, d):
    """All values 6 * 2^125 (or of both signs), all scores alike (or not): results are finite,
    and right, in tiles that one CTA has and in joined ones."""
    for alike in (True, False):
        c, q, starts, lens, kd, vd = x = chunk("mx4", new, past, G, 1, d, L, 16)
        c.vs[held(c, "vs")] = LARGEST
        if not signs:
            c.v[:] = 0x77
        if alike:
            q[: starts[-1]] = 0
        if L:
            vd[:, : starts[-1]] = torch.where(vd[:, : starts[-1]] < 0, -3e38 if signs else 2e38, 3e38)
        o, lse = run(*x, d ** -0.5)
        assert torch.isfinite(o[: starts[-1]]).all()
        check(*x, d ** -0.5, o, lse)


@pytest.mark.parametrize("d", [64, 128])
def test_a_token_over_the_largest_values_is_a_decode(d):
    lens = [2, 700, 129]
    c, q, starts, _, kd, vd = chunk("mx4", [1] * 3, [n - 1 for n in lens], 16, 4, d, 3, 64)
    c.vs[held(c, "vs")] = torch.randint(240, LARGEST + 1, c.vs.shape, generator=torch.Generator().manual_seed(7),
                                        dtype=torch.uint8).cuda()[held(c, "vs")]
    o, lse = run(c, q, starts, lens, kd, vd, 0.1)
    views = dict(kd=kd.permute(1, 2, 0, 3), vd=vd.permute(1, 2, 0, 3))
    want, wl = moda.moda_decode_paged(q, *c.args(), i32(lens), 0.1, **views, **c.scales())
    settled()
    assert torch.isfinite(o).all() and torch.isfinite(want).all()
    _, _, to, tl = cc.prefill_reference(c, q, starts, lens, kd, vd, 0.1)
    # the decode's own rounding of probabilities (2^-11 and less of the largest product)
    assert ((o.double() - want.double()).abs() <= 3 * to).all() and ((lse.double() - wl.double()).abs() <= 2 * tl).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("low,high", [(0, 40), (20, 60), (90, 130)])
def test_small_values(low, high, d):
    """Scale bytes of 0 to 60 stand for 2^-127 to 2^-67. Of V those up to 26 count as 0, with which
    an average is off by 6 * 2^-101 at most; a product of weight (the largest is at least 1) and
    value may be lost below 2^-100."""
    c, q, starts, lens, kd, vd = chunk("mx4", [5, 40, 1], [3, 700, 5000], 4, 1, d, 0, 16)
    mask = held(c, "vs")
    c.vs[mask] = torch.randint(low, high, c.vs.shape, generator=torch.Generator().manual_seed(8),
                               dtype=torch.uint8).cuda()[mask]
    o, lse = run(c, q, starts, lens, kd, vd, d ** -0.5)
    wo, wl, to, tl = cc.prefill_reference(c, q, starts, lens, kd, vd, d ** -0.5)
    slack = torch.zeros_like(to)
    for b, n in enumerate(lens):
        slack[starts[b] : starts[b + 1]] = 6 * 2.0 ** -101 + n * 2.0 ** -100
    assert ((o.double() - wo).abs() <= to + slack).all() and ((lse.double() - wl).abs() <= tl).all()


@pytest.mark.parametrize("d", [64, 128])
def test_bytes_from_which_on_bf16_holds_infinity(d):
    """Scale bytes of 253 and 254, which no append writes, as bf16 would not hold all their
    codes: a chunk counts with the values that they stand for; NaN (255) stays what it is, where
    it is seen."""
    c, q, starts, lens, kd, vd = x = chunk("mx4", [8], [40], 4, 1, d, 0, 16)
    c.v[:] = 0x22  # 1 * 2^127 under 254
    page = c.table[0].long()
    c.vs[page[0], 0, 3] = 254
    c.vs[page[2], 0, 13, 0] = 255  # row 45: seen by the tokens at rows 45 to 47
    q[:] = 0
    o, lse = run(*x, d ** -0.5)
    want = (2.0 ** 127 / torch.arange(41, 49, dtype=torch.float64, device="cuda")).view(8, 1, 1)
    assert torch.isnan(o[5:, :, :32]).all()
    fine = torch.ones_like(o, dtype=torch.bool)
    fine[5:, :, :32] = False
    err = (o.double() - want).abs() - want * (4 * pc.HALF_BF16)
    assert (err[fine.expand_as(err)] <= 0).all()


@pytest.mark.parametrize("d", [64, 128])
def test_sums_of_as_many_of_the_largest_values_as_the_header_names(d):
    """2^24 rows (of two pages, named again and again), and 128 of smaller scores in front, whose
    share holds blocks with weights of just under 2^8 in all."""
    n, page = 1 << 24, 128
    k, v = (torch.zeros(2, 1, page, d // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((2, 1, page, d // 32), 127, dtype=torch.uint8, device="cuda") for _ in range(2))
    v[:], vs[:] = 0x77, LARGEST
    k[1, :, :, 0] = 2  # 1 in the first element
    table = torch.ones(1, n // page, dtype=torch.int32, device="cuda")
    table[0, 0] = 0
    q = torch.zeros(1, 4, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    scale = 0.686  # 2^0.99 as much weight as the first 128
    o, lse = moda.moda_prefill_paged(q, k, v, table, i32([0, 1]), i32([n]), scale, k_scales=ks, v_scales=vs)
    settled()
    assert (o == 6 * 2.0 ** 125).all()
    want = torch.logsumexp(torch.tensor([math.log(128.0), math.log(n - 128.0) + scale], dtype=torch.float64), 0)
    assert (lse.double().cpu() - want).abs().max() < 2.0 ** -18 * want
