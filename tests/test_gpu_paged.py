"""The paged KV cache on the GPU: append, gather and decode against fp64 forms
(tests/paged_common.py), at the sizes, masks and indexes where they can go
wrong, and a run of them together as a server uses them."""
import math

import pytest
import torch

import sequence_depth_attention_gb300 as moda
from sequence_depth_attention_gb300 import build as mbuild

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


def fused_qkv(N, Hq, Hk, d, seed, gap=0):
    """Views q, k, v of one projection's output, `gap` elements behind each token."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(N, (Hq + 2 * Hk) * d + gap, generator=g).bfloat16().cuda()
    return (x[:, : Hq * d].view(N, Hq, d) if Hq else None,
            x[:, Hq * d : (Hq + Hk) * d].view(N, Hk, d),
            x[:, (Hq + Hk) * d : (Hq + 2 * Hk) * d].view(N, Hk, d))


def tokens(new, lens, pad, seed):
    """seq, pos of the last new[b] rows of every sequence, in random order, padding among them."""
    at = [(b, p) for b, (m, n) in enumerate(zip(new, lens)) for p in range(n - m, n)] + [(-1, 12345)] * pad
    order = torch.randperm(len(at), generator=torch.Generator().manual_seed(seed)).tolist()
    at = [at[i] for i in order]
    return (torch.tensor([s for s, _ in at], dtype=torch.int32, device="cuda"),
            torch.tensor([p for _, p in at], dtype=torch.int32, device="cuda"))


# ------------------------------------------------------------------- append
APPENDS = [
    # fmt, d, rot, interleaved, page, Hq, Hk, rows brought, rows held after, padding
    ("bf16", 128, 128, False, 64, 16, 4, [1], [701], 0),
    ("mx4", 128, 128, False, 16, 16, 4, [1, 1, 1], [1, 17, 160], 2),
    ("bf16", 64, 64, True, 16, 6, 2, [40, 1, 7], [40, 1, 19], 1),
    ("mx4", 64, 32, True, 32, 64, 8, [33, 65], [100, 65], 0),
    ("mx4", 128, 48, False, 128, 3, 1, [131, 5], [131, 300], 3),
    ("bf16", 128, 16, False, 32, 5, 5, [29], [29], 0),
    ("mx4", 64, 0, False, 64, 0, 3, [50, 0, 2], [64, 0, 3], 0),
    ("bf16", 64, 48, True, 128, 0, 1, [9, 9, 9, 9], [9, 130, 255, 257], 4),
    ("mx4", 128, 112, True, 64, 32, 2, [17, 18], [4000, 19], 0),
]


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: "-".join(map(str, c[:7])))
def test_append(case):
    fmt, d, rot, inter, page, Hq, Hk, new, lens, pad = case
    c = pc.Cache(fmt, lens, Hk, d, page, seed=5, device="cuda")
    seq, pos = tokens(new, lens, pad, 6)
    N = seq.numel()
    q, k, v = fused_qkv(N, Hq, Hk, d, 7, gap=8)
    rope = pc.rope_table(max(lens), rot).cuda() if rot else None
    before, q_in = c.bits(), None if q is None else q.clone()
    q_out = torch.full((N, Hq, d), 3.5, dtype=torch.bfloat16, device="cuda") if Hq else None
    k_out = torch.full((N, Hk, d), 3.5, dtype=torch.bfloat16, device="cuda")
    got = moda.moda_kv_append(q, k, v, *c.args(), seq, pos, rope=rope, interleaved=inter, q_out=q_out,
                              k_out=k_out, **c.scales())
    settled()
    assert got[1] is k_out and (q is None or torch.equal(q, q_in))
    real = seq >= 0

    # q_out and k_out: one bf16 rounding of a sum of two products, each product
    # and the sum rounded to fp32: half a bf16 step of the value, and 3 fp32
    # half steps of the products' magnitudes
    for x, out in ((q, q_out), (k, k_out)):
        if x is None:
            continue
        if rot:
            want = pc.turned(x[real], rope, pos[real], inter)
            mags = pc.turned(x[real].abs(), torch.cat((rope[:, : rot // 2].abs(), -rope[:, rot // 2:].abs()), 1),
                             pos[real], inter).abs() + pc.turned(
                x[real].abs(), rope.abs(), pos[real], inter).abs()
        else:
            want = x[real].double()
            mags = torch.zeros_like(want)
        err = (out[real].double() - want).abs()
        assert (err <= pc.HALF_BF16 * want.abs() + 4 * pc.HALF_FP32 * mags).all()
        assert (out[~real] == 3.5).all()
        assert torch.equal(out[real][..., rot:], x[real][..., rot:])

    # the pages: named rows hold the token, every other bit is as it was
    s, p = seq[real].long(), pos[real].long()
    at, off = c.table[s, p // page].long(), p % page
    if fmt == "bf16":
        before[0][at, :, off] = k_out[real]
        before[1][at, :, off] = v[real]
    else:
        kx = pc.turned(k[real], rope, pos[real], inter) if rot else k[real].double()
        for x, codes, scales in ((kx, c.k, c.ks), (v[real].double(), c.v, c.vs)):
            have = pc.mx4_values(codes[at, :, off], scales[at, :, off])
            assert torch.equal(have, pc.mx4_quantised(x))
        for i, t in enumerate((c.k, c.v, c.ks, c.vs)):
            before[i][at, :, off] = t[at, :, off]
    for was, t in zip(before, [t for t in (c.k, c.v, c.ks, c.vs) if t is not None]):
        assert torch.equal(was.view(torch.int16 if was.dtype == torch.bfloat16 else torch.uint8),
                           t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.uint8))


def test_append_large_values_and_ties():
    """4-bit rows of values on and next to every border of every binade, tiny
    and huge blocks, infinities and NaN."""
    d, page, Hk = 64, 16, 1
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0], dtype=torch.float64)
    vals = torch.cat([border, border * (1 + 2 ** -7), border * (1 - 2 ** -8), -border])  # 32 values
    rows = []
    for e in list(range(-133, 126, 7)) + [124, 125]:
        rows.append(torch.cat((vals, vals.flip(0))) * 2.0 ** e)
    rows.append(torch.full((d,), 3.3895313892515355e38, dtype=torch.float64))  # the largest bf16
    rows.append(torch.zeros(d, dtype=torch.float64))
    x = torch.stack(rows)[:, None].bfloat16()
    special = torch.zeros(3, 1, d)
    special[0, 0, 3], special[1, 0, 40], special[2, 0, 63] = math.inf, -math.inf, math.nan
    x = torch.cat((x, special.bfloat16())).cuda()
    N = x.shape[0]
    c = pc.Cache("mx4", [N], Hk, d, page, device="cuda")
    seq, pos = torch.zeros(N, dtype=torch.int32, device="cuda"), torch.arange(N, dtype=torch.int32, device="cuda")
    moda.moda_kv_append(None, x, x, *c.args(), seq, pos, **c.scales())
    k, v = moda.moda_kv_gather(*c.args(), seq, pos, **c.scales())
    settled()
    for got in (c.rows("k", 0, N), c.rows("v", 0, N), k.transpose(0, 1).double(), v.transpose(0, 1).double()):
        want = pc.mx4_quantised(x.double()).transpose(0, 1)
        # the largest magnitudes saturate at 6 * 2^125
        want = want.clamp(-6 * 2.0 ** 125, 6 * 2.0 ** 125)
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(), want.nan_to_num())


def test_append_unturned_elements_keep_infinities():
    """Elements behind the turned part are copied whatever they are."""
    q, k, v = fused_qkv(3, 2, 2, 64, 1)
    for t in (q, k, v):
        t[..., 40], t[..., 41], t[..., 63] = math.inf, -math.inf, math.nan
    c = pc.Cache("bf16", [3], 2, 64, 16, device="cuda")
    i = torch.arange(3, dtype=torch.int32, device="cuda")
    qo, ko = moda.moda_kv_append(q, k, v, *c.args(), torch.zeros_like(i), i, rope=pc.rope_table(3, 32).cuda())
    settled()
    stored = [t[c.table[0, :1].long()][0, :, :3].transpose(0, 1) for t in (c.k, c.v)]
    for a, b in ((qo, q), (ko, k), (stored[0], k), (stored[1], v)):
        a, b = (x[..., 32:].contiguous().view(torch.int16) for x in (a, b))
        assert torch.equal(a, b)
    assert not qo[..., :32].isnan().any()


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
@pytest.mark.parametrize("bad", ["seq", "seq_neg", "pos", "pos_neg", "rope", "page", "page_neg"])
def test_append_and_gather_bad_indexes(fmt, bad):
    """An index out of range leaves its own token out, and nothing else."""
    d, page, Hk, N = 128, 16, 2, 6
    c = pc.Cache(fmt, [32, 32], Hk, d, page, device="cuda")
    q, k, v = fused_qkv(N, 4, Hk, d, 2)
    seq = torch.tensor([0, 1, 0, 1, 0, 1], dtype=torch.int32, device="cuda")
    pos = torch.tensor([0, 1, 2, 19, 20, 21], dtype=torch.int32, device="cuda")
    rope = pc.rope_table(32, d).cuda()
    good = torch.ones(N, dtype=torch.bool, device="cuda")
    table = c.table
    if bad == "seq":
        seq[3] = 2
    elif bad == "seq_neg":
        seq[3] = -2
    elif bad == "pos":
        pos[3] = 32
    elif bad == "pos_neg":
        pos[3] = -1
    elif bad == "rope":
        rope = rope[:21].contiguous()
        good[5] = False
    else:
        table = c.table.clone()
        table[1, 1] = c.num_pages if bad == "page" else -1
        good[5] = False
    if bad != "rope":
        good[3] = False
    before = c.bits()
    qo = torch.full((N, 4, d), 2.0, dtype=torch.bfloat16, device="cuda")
    ko = torch.full((N, Hk, d), 2.0, dtype=torch.bfloat16, device="cuda")
    moda.moda_kv_append(q, k, v, c.k, c.v, table, seq, pos, rope=rope, q_out=qo, k_out=ko, **c.scales())
    settled(INVALID)
    settled()
    assert (qo[~good] == 2).all() and (ko[~good] == 2).all()
    assert not (qo[good] == 2).all(-1).any()
    at, off = c.table[seq[good].long(), pos[good].long() // page].long(), (pos[good] % page).long()
    for was, t in zip(before, [t for t in (c.k, c.v, c.ks, c.vs) if t is not None]):
        was[at, :, off] = t[at, :, off]
        assert torch.equal(was.view(torch.uint8), t.view(torch.uint8))
    kg = torch.full((N, Hk, d), 2.0, dtype=torch.bfloat16, device="cuda")
    vg = kg.clone()
    if bad == "rope":  # the positions themselves are fine
        return
    moda.moda_kv_gather(c.k, c.v, table, seq, pos, k=kg, v=vg, **c.scales())
    settled(INVALID)
    assert (kg[~good] == 2).all() and (vg[~good] == 2).all()
    if fmt == "bf16":
        assert torch.equal(kg[good], ko[good]) and torch.equal(vg[good], v[good])


# ------------------------------------------------------------------- gather
@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
@pytest.mark.parametrize("d,page,Hk", [(128, 16, 3), (64, 128, 1), (64, 32, 8), (128, 64, 4)])
def test_gather(fmt, d, page, Hk):
    lens = [1, 0, 129, 40]
    c = pc.Cache(fmt, lens, Hk, d, page, seed=8, fill=None, device="cuda")
    if fmt == "mx4":  # every scale byte, every code
        g = torch.Generator().manual_seed(9)
        c.ks = torch.randint(0, 256, c.ks.shape, generator=g, dtype=torch.uint8).cuda()
        c.vs = torch.randint(0, 256, c.vs.shape, generator=g, dtype=torch.uint8).cuda()
    seq, pos = tokens(lens, lens, 3, 10)
    seq, pos = torch.cat((seq, seq[:50])), torch.cat((pos, pos[:50]))  # the same rows again
    k = torch.full((seq.numel(), Hk, d), 9.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    moda.moda_kv_gather(*c.args(), seq, pos, k=k, v=v, **c.scales())
    settled()
    for n in range(seq.numel()):
        s, p = int(seq[n]), int(pos[n])
        if s < 0:
            assert (k[n] == 9).all() and (v[n] == 9).all()
            continue
        for got, which in ((k[n], "k"), (v[n], "v")):
            want = c.rows(which, s, p + 1)[:, p].bfloat16()  # inf where bf16 ends
            assert torch.equal(got.isnan(), want.isnan())
            assert torch.equal(got.nan_to_num(nan=7.0), want.nan_to_num(nan=7.0))


# ------------------------------------------------------------------- decode
def depth(B, Hk, L, d, seed):
    if L == 0:
        return None, None
    g = torch.Generator().manual_seed(seed)
    return tuple(torch.randn(B, Hk, L, d, generator=g).bfloat16().cuda() for _ in range(2))


def check_decode(c, q, lens, kd, vd, scale, o, lse):
    ro, rl, to, tl = pc.decode_reference(c, q, lens, kd, vd, scale)
    assert ((o.double() - ro).abs() <= to).all(), ((o.double() - ro).abs() - to).max().item()
    same = rl == lse.double()  # the empty rows' -infinity
    assert (same | ((lse.double() - rl).abs() <= tl)).all()


@pytest.fixture(params=[0, 16384], ids=["narrow", "wide"])
def table_of(request, monkeypatch):
    """Block tables just wide enough for the longest sequence (short batches then
    get a group of CTAs for each segment), and wide ones (the batch is cut into
    equal shares)."""
    monkeypatch.setattr(pc.Cache, "least_rows", request.param)
    return request.param


RAGGED = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 1000]
DECODES = [
    # d, page, Hk, G, L, lens
    (128, 64, 4, 4, 46, [701]),
    (128, 16, 2, 1, 0, RAGGED),
    (128, 32, 1, 16, 17, RAGGED),
    (64, 16, 2, 8, 64, RAGGED),
    (64, 128, 3, 5, 1, RAGGED),
    (128, 128, 1, 9, 130, [0, 0, 300, 2]),
    (64, 64, 8, 3, 0, [0, 5, 0, 0, 4097, 0]),
    (64, 32, 1, 16, 3, [2500, 31, 33]),
    (128, 64, 1, 2, 0, [0]),
    (128, 64, 2, 2, 5, [0, 0]),
    (128, 16, 8, 4, 24, [2000, 1, 600] + [77] * 60),
    (64, 16, 3, 5, 70, [9003]),
    (128, 32, 7, 2, 0, [14001]),
    # narrow tables: 16, 16, 6 (4-bit: 8), 5 (7), 5 (8), 2 (3), one and one CTAs a segment
    (128, 64, 4, 4, 24, [3900, 40]),
    (64, 16, 1, 16, 70, [0, 3800, 1, 127, 2001]),
    (64, 32, 4, 3, 0, RAGGED[1:]),
    (128, 64, 4, 9, 5, [900, 0, 7] + RAGGED[2:]),
    (128, 16, 4, 4, 24, RAGGED),
    (64, 32, 4, 7, 0, RAGGED + RAGGED + [2, 3]),
    (128, 64, 4, 2, 9, [500, 0, 1, 64, 65] * 10),
    (64, 16, 4, 4, 0, [33, 0, 64]),
]


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
@pytest.mark.parametrize("case", DECODES, ids=lambda c: "-".join(map(str, c[:5])) + f"-B{len(c[5])}")
def test_decode(fmt, case, table_of):
    d, page, Hk, G, L, lens = case
    B = len(lens)
    c = pc.Cache(fmt, lens, Hk, d, page, seed=11, device="cuda")
    q = torch.randn(B, Hk * G, d, generator=torch.Generator().manual_seed(12)).bfloat16().cuda()
    kd, vd = depth(B, Hk, L, d, 13)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = moda.moda_decode_paged(q, *c.args(), n, d ** -0.5, kd=kd, vd=vd, **c.scales())
    settled()
    check_decode(c, q, lens, kd, vd, d ** -0.5, o, lse)
    # lse left out, o into the caller's tensor, the workspace full of NaN: the same bits
    ws = torch.full((moda.moda_decode_paged_workspace_bytes(Hk * G, Hk, d) // 4,), math.nan, device="cuda")
    o2, none = moda.moda_decode_paged(q, *c.args(), n, d ** -0.5, kd=kd, vd=vd, workspace=ws,
                                      o=torch.full_like(q, math.nan), want_lse=False, **c.scales())
    settled()
    assert none is None and torch.equal(o, o2)


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
def test_decode_depth_views(fmt, table_of):
    """The depth slots in place in layer-major tensors [L, B, Hk, d], and with gaps."""
    d, Hk, L, lens = 128, 2, 7, [40, 0, 100]
    c = pc.Cache(fmt, lens, Hk, d, 16, seed=14, device="cuda")
    q = torch.randn(3, 8, d, generator=torch.Generator().manual_seed(15)).bfloat16().cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(16)
    lm = [torch.randn(L, 3, Hk, d, generator=g).bfloat16().cuda() for _ in range(2)]
    wide = [torch.randn(3, Hk, L + 3, 2 * d, generator=g).bfloat16().cuda() for _ in range(2)]
    for kd, vd in ([x.permute(1, 2, 0, 3) for x in lm], [x[:, :, 1 : L + 1, :d] for x in wide]):
        o, lse = moda.moda_decode_paged(q, *c.args(), n, 0.1, kd=kd, vd=vd, **c.scales())
        settled()
        check_decode(c, q, lens, kd, vd, 0.1, o, lse)


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
@pytest.mark.parametrize("mul", [1e-3, 30.0])
def test_decode_flat_and_peaked(fmt, mul, table_of):
    """Scores from all alike to one key taking all the weight."""
    d, Hk, lens = 128, 2, [900, 64, 3]
    c = pc.Cache(fmt, lens, Hk, d, 32, seed=17, device="cuda")
    q = (torch.randn(3, 8, d, generator=torch.Generator().manual_seed(18)) * mul).bfloat16().cuda()
    kd, vd = depth(3, Hk, 24, d, 19)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = moda.moda_decode_paged(q, *c.args(), n, d ** -0.5, kd=kd, vd=vd, **c.scales())
    settled()
    check_decode(c, q, lens, kd, vd, d ** -0.5, o, lse)


def test_decode_mx4_scales_far_apart(table_of):
    """Key and value blocks of very different magnitudes: rows whose values are
    2^40 larger have next to no weight, and queries far from 1. The others'
    part must not be lost beside them."""
    d, Hk, G, lens = 128, 2, 4, [500, 130]
    c = pc.Cache("mx4", lens, Hk, d, 16, seed=20, device="cuda")
    g = torch.Generator().manual_seed(21)
    q = torch.randn(2, Hk * G, d, generator=g).bfloat16().cuda()
    for b, n in enumerate(lens):
        for p in (3, 64, n - 2):
            page, off = int(c.table[b, p // 16]), p % 16
            c.vs[page, :, off] = 127 + 40
            # a key that every query scores far below the others: codes against the
            # signs of the group's first query, large scale
            c.k[page, :, off], c.ks[page, :, off] = 0, 127
            for h in range(Hk):
                sign = (q[b, h * G] > 0)
                code = torch.where(sign, 15, 7).to(torch.uint8)  # -6 / +6
                c.k[page, h, off] = code[0::2] | (code[1::2] << 4)
                c.ks[page, h, off] = 130
    q = q.view(2, Hk, G, d)[:, :, :1].expand(-1, -1, G, -1).reshape(2, Hk * G, d).contiguous()
    for mul, scale in ((1.0, d ** -0.5), (2.0 ** 60, 2.0 ** -60 * d ** -0.5), (2.0 ** -60, 2.0 ** 60 * d ** -0.5)):
        n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        qq = (q.float() * mul).bfloat16()
        o, lse = moda.moda_decode_paged(qq, *c.args(), n, scale, **c.scales())
        settled()
        check_decode(c, qq, lens, None, None, scale, o, lse)


def test_decode_mx4_nan_block(table_of):
    """A block stored as NaN makes its head's columns NaN; the other heads are untouched."""
    d, Hk, lens = 64, 2, [50]
    c = pc.Cache("mx4", lens, Hk, d, 16, seed=22, device="cuda")
    c.v[c.table[0, 1], 1, 5, 16:] = 0
    c.vs[c.table[0, 1], 1, 5, 1] = 255
    q = torch.randn(1, 4, d, generator=torch.Generator().manual_seed(23)).bfloat16().cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = moda.moda_decode_paged(q, *c.args(), n, 0.125, **c.scales())
    settled()
    assert o[0, 2:, 32:].isnan().all() and not o[0, :2].isnan().any()
    ro, _, to, _ = pc.decode_reference(c, q, lens, None, None, 0.125)
    assert ((o.double() - ro).abs() <= to)[0, :2].all()
    c.k[c.table[0, 2], 0, 3, :16] = 0
    c.ks[c.table[0, 2], 0, 3, 0] = 255
    o, lse = moda.moda_decode_paged(q, *c.args(), n, 0.125, **c.scales())
    settled()
    assert o[0, :2].isnan().all() and lse[0, :2].isnan().all()


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
def test_decode_bad_lengths_and_pages(fmt):
    d, Hk, lens = 64, 2, [40, 64, 20]
    c = pc.Cache(fmt, lens, Hk, d, 16, seed=24, fill=None, width=4, device="cuda")
    c.table[0, 3] = c.table[0, 0]
    q = torch.randn(3, 4, d, generator=torch.Generator().manual_seed(25)).bfloat16().cuda()
    # too long is taken as the table's width, negative as empty
    n = torch.tensor([40, 1000, -3], dtype=torch.int32, device="cuda")
    o, lse = moda.moda_decode_paged(q, *c.args(), n, 0.125, **c.scales())
    settled(INVALID)
    check_decode(c, q, [40, 64, 0], None, None, 0.125, o, lse)
    # a page that is none: latched; the other sequences are right
    for bad in (-1, c.num_pages, 2 ** 31 - 1):
        table = c.table.clone()
        table[1, 2] = bad
        n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        o, lse = moda.moda_decode_paged(q, c.k, c.v, table, n, 0.125, **c.scales())
        settled(INVALID)
        ro, rl, to, tl = pc.decode_reference(c, q, lens, None, None, 0.125)
        ok = (o.double() - ro).abs() <= to
        assert ok[0].all() and ok[2].all()
    settled()


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
def test_offsets_past_32_bits(fmt):
    """Rows whose element offset in the pool is beyond 2^31 (bf16: beyond 4 GiB too)."""
    d, Hk, page, lens = 128, 4, 128, [300, 5]
    c = pc.Cache(fmt, lens, Hk, d, page, seed=26, device="cuda")
    pages = (2 ** 31 + 2 ** 28) // (Hk * page * d)  # pools of 2.4 G elements
    shift = pages - c.num_pages
    big = []
    for t in (c.k, c.v, c.ks, c.vs):
        x = None
        if t is not None:
            x = torch.zeros((pages, *t.shape[1:]), dtype=t.dtype, device="cuda")
            x[shift:] = t
        big.append(x)
    table = torch.where(c.table >= 0, c.table + shift, c.table)
    scales = dict(k_scales=big[2], v_scales=big[3])
    q, k, v = fused_qkv(2, 16, Hk, d, 27)
    seq = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    pos = torch.tensor([299, 4], dtype=torch.int32, device="cuda")
    rope = pc.rope_table(300, d).cuda()
    qo, _ = moda.moda_kv_append(q, k, v, *c.args(), seq, pos, rope=rope, **c.scales())
    qb, _ = moda.moda_kv_append(q, k, v, big[0], big[1], table, seq, pos, rope=rope, **scales)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    a = moda.moda_decode_paged(qo, *c.args(), n, d ** -0.5, **c.scales())
    b = moda.moda_decode_paged(qb, big[0], big[1], table, n, d ** -0.5, **scales)
    ka = moda.moda_kv_gather(*c.args(), seq, pos, **c.scales())
    kb = moda.moda_kv_gather(big[0], big[1], table, seq, pos, **scales)
    settled()
    for x, y in zip(a + ka, b + kb):
        assert torch.equal(x, y)
    check_decode(c, qo, lens, None, None, d ** -0.5, *a)


# -------------------------------------------------------- streams and graphs
@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
def test_decode_on_streams_and_in_graphs(fmt, table_of):
    """Two calls at once with a workspace each; a captured step (append and
    decode) replayed on new inputs; two graphs that share a workspace, in turn."""
    d, Hk, lens = 128, 4, [3000, 700, 1, 64]
    scale = d ** -0.5
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cs = [pc.Cache(fmt, lens, Hk, d, 16, seed=30 + i, device="cuda") for i in range(2)]
    qs = [torch.randn(4, 16, d, generator=torch.Generator().manual_seed(40 + i)).bfloat16().cuda() for i in range(2)]
    kd, vd = depth(4, Hk, 24, d, 50)
    alone = [moda.moda_decode_paged(q, *c.args(), n, scale, kd=kd, vd=vd, **c.scales()) for c, q in zip(cs, qs)]
    settled()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for rep in range(4):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(moda.moda_decode_paged(qs[i], *cs[i].args(), n, scale, kd=kd, vd=vd,
                                                     **cs[i].scales()))
    settled()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, alone[i][0]) and torch.equal(lse, alone[i][1])

    # one step captured: append one token per sequence, then attend
    c = cs[0]
    q, k, v = fused_qkv(4, 16, Hk, d, 60)
    seq = torch.arange(4, dtype=torch.int32, device="cuda")
    pos = n - 1
    rope = pc.rope_table(3000, d).cuda()
    ws = torch.empty(moda.moda_decode_paged_workspace_bytes(16, Hk, d) // 4, device="cuda")
    out = [(torch.empty(4, 16, d, dtype=torch.bfloat16, device="cuda"), torch.empty(4, 16, device="cuda"))
           for _ in range(2)]
    qo = torch.empty_like(out[0][0])
    ko = torch.empty(4, Hk, d, dtype=torch.bfloat16, device="cuda")

    def step(i):
        moda.moda_kv_append(q, k, v, *cs[i].args(), seq, pos, rope=rope, q_out=qo, k_out=ko, **cs[i].scales())
        moda.moda_decode_paged(qo, *cs[i].args(), n, scale, kd=kd, vd=vd, o=out[i][0], lse=out[i][1],
                               workspace=ws, **cs[i].scales())

    side = torch.cuda.Stream()
    graphs = []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            step(i)
            side.synchronize()
            with torch.cuda.graph(graph, stream=side):
                step(i)
        graphs.append(graph)
    for rep in range(3):
        base = q._base if q._base is not None else q
        base.copy_(torch.randn(base.shape, generator=torch.Generator().manual_seed(70 + rep)).bfloat16())
        if rep == 2:  # the lengths are read when the graph runs
            n.copy_(torch.tensor([2999, 1, 0, 63], dtype=torch.int32))
            pos.copy_((n - 1).clamp(min=0))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        replayed = [(o.clone(), lse.clone()) for o, lse in out]
        for i in range(2):
            step(i)
            torch.cuda.synchronize()
            assert torch.equal(out[i][0], replayed[i][0]) and torch.equal(out[i][1], replayed[i][1])
    settled()


# ------------------------------------------------------------- all together
@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
def test_prompt_then_steps(fmt, table_of):
    """Two requests: prompts through moda_kv_append and moda_fwd_layer_major,
    the keys' depth slots through what k_out gives, then single tokens through
    append and decode_paged; every row against one fp64 pass over the whole
    sequence (for 4-bit pages: over the values that the pages hold)."""
    d, Hk, G, L, page = 64, 2, 4, 3, 16
    Hq, scale, steps = Hk * G, d ** -0.5, 5
    prompts = [37, 80]
    total = [p + steps for p in prompts]
    c = pc.Cache(fmt, total, Hk, d, page, seed=80, device="cuda")
    rope = pc.rope_table(max(total), d).cuda()
    xs = [fused_qkv(t, Hq, Hk, d, 81 + b) for b, t in enumerate(total)]
    dep = [depth(t, Hk, L, d, 90 + b) for b, t in enumerate(total)]  # [T, Hk, L, d]

    def rows(b, i):  # the token's views as a batch of one
        return [t[i : i + 1] for t in xs[b]]

    # prompts: both requests' tokens in one append, then each its own attention
    seq = torch.cat([torch.full((p,), b, dtype=torch.int32) for b, p in enumerate(prompts)]).cuda()
    pos = torch.cat([torch.arange(p, dtype=torch.int32) for p in prompts]).cuda()
    q, k, v = (torch.cat([xs[b][i][: prompts[b]] for b in range(2)]) for i in range(3))
    qo, ko = moda.moda_kv_append(q, k, v, *c.args(), seq, pos, rope=rope, **c.scales())
    at = 0
    for b, p in enumerate(prompts):
        kl, vl = (t[:p].permute(2, 0, 1, 3).contiguous() for t in dep[b])  # [L, T, Hk, d]
        o, lse = moda.moda_fwd_layer_major(qo[at : at + p], ko[at : at + p], v[at : at + p].contiguous(),
                                           kl, vl, scale)
        settled()
        turned = [pc.turned(xs[b][i][:p], rope, torch.arange(p, device="cuda"), False) for i in range(2)]
        for t in range(p):
            kk = torch.cat((turned[1][: t + 1].transpose(0, 1), dep[b][0][t].double()), 1)
            vv = torch.cat((xs[b][2][: t + 1].double().transpose(0, 1), dep[b][1][t].double()), 1)
            z = turned[0][t].view(Hk, G, d) @ kk.transpose(1, 2) * scale
            want = (torch.softmax(z, -1) @ vv).view(Hq, d)
            assert (o[t].double() - want).abs().max() <= 2e-2  # moda_fwd's documented accuracy
        at += p
    # steps: one token of each request at a time
    for i in range(steps):
        n = torch.tensor([p + i + 1 for p in prompts], dtype=torch.int32, device="cuda")
        q, k, v = (torch.cat([rows(b, prompts[b] + i)[j] for b in range(2)]) for j in range(3))
        seq = torch.arange(2, dtype=torch.int32, device="cuda")
        qo, ko = moda.moda_kv_append(q, k, v, *c.args(), seq, n - 1, rope=rope, **c.scales())
        kd = torch.stack([dep[b][0][prompts[b] + i] for b in range(2)])
        vd = torch.stack([dep[b][1][prompts[b] + i] for b in range(2)])
        o, lse = moda.moda_decode_paged(qo, *c.args(), n, scale, kd=kd, vd=vd, **c.scales())
        settled()
        check_decode(c, qo, n.tolist(), kd, vd, scale, o, lse)
        if fmt == "bf16":  # and against the sequence itself, turned in fp64
            for b in range(2):
                t = prompts[b] + i
                p = torch.arange(t + 1, device="cuda")
                kk = pc.turned(xs[b][1][: t + 1], rope, p, False).transpose(0, 1)
                qq = pc.turned(xs[b][0][t : t + 1], rope, p[t:], False)[0].view(Hk, G, d)
                kk = torch.cat((kk, kd[b].double()), 1)
                vv = torch.cat((xs[b][2][: t + 1].double().transpose(0, 1), vd[b].double()), 1)
                want = (torch.softmax(qq @ kk.transpose(1, 2) * scale, -1) @ vv).view(Hq, d)
                assert (o[b].double() - want).abs().max() <= 2e-2
    # the whole of both requests read back
    seq = torch.cat([torch.full((t,), b, dtype=torch.int32) for b, t in enumerate(total)]).cuda()
    pos = torch.cat([torch.arange(t, dtype=torch.int32) for t in total]).cuda()
    kg, vg = moda.moda_kv_gather(*c.args(), seq, pos, **c.scales())
    settled()
    want_v = torch.cat([xs[b][2] for b in range(2)])
    if fmt == "bf16":
        assert torch.equal(vg, want_v)
    else:
        assert torch.equal(vg.double(), pc.mx4_quantised(want_v.double()))
        want_k = torch.cat([pc.turned(xs[b][1], rope, torch.arange(total[b], device="cuda"), False)
                            for b in range(2)])
        assert torch.equal(kg.double(), pc.mx4_quantised(want_k))


# --------------------------------------------------------- wide, many, often
@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
@pytest.mark.parametrize("B,Hk,G,L", [(3000, 1, 2, 0), (700, 4, 16, 3), (257, 2, 5, 17)])
def test_decode_many_sequences(fmt, B, Hk, G, L):
    """More sequences than threads of a CTA, empty ones among them, segments
    shorter than a unit and cut anywhere."""
    d, page = 64, 16
    g = torch.Generator().manual_seed(100 + B)
    lens = torch.randint(0, 90, (B,), generator=g)
    lens[torch.rand(B, generator=g) < 0.3] = 0
    lens[B // 2] = 2500
    lens = lens.tolist()
    c = pc.Cache(fmt, lens, Hk, d, page, seed=101, device="cuda")
    q = torch.randn(B, Hk * G, d, generator=g).bfloat16().cuda()
    kd, vd = depth(B, Hk, L, d, 102)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = moda.moda_decode_paged(q, *c.args(), n, 0.125, kd=kd, vd=vd, **c.scales())
    settled()
    check_decode(c, q, lens, kd, vd, 0.125, o, lse)


def test_decode_paged_against_moda_decode():
    """One sequence through the dense cache's decode and through pages."""
    d, Hk, G, L, n = 128, 4, 4, 46, 5000
    c = pc.Cache("bf16", [n], Hk, d, 64, seed=110, device="cuda")
    k, v = (c.rows(w, 0, n).transpose(0, 1).contiguous().bfloat16() for w in ("k", "v"))
    q = torch.randn(1, Hk * G, d, generator=torch.Generator().manual_seed(111)).bfloat16().cuda()
    kd, vd = depth(1, Hk, L, d, 112)
    o, lse = moda.moda_decode_paged(q, *c.args(), torch.tensor([n], dtype=torch.int32, device="cuda"),
                                    d ** -0.5, kd=kd, vd=vd)
    od, lsed = moda.moda_decode(q[0], k, v, kd[0], vd[0], d ** -0.5)
    settled()
    ro, rl, to, tl = pc.decode_reference(c, q, [n], kd, vd, d ** -0.5)
    # each is within its tolerance of the same values
    assert ((o - od).abs().double() <= 2 * to).all() and ((lse - lsed).abs().double() <= 2 * tl).all()


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
def test_append_many_heads(fmt):
    """More heads than a warp's or a CTA's, of odd numbers."""
    d, Hk, Hq, N = 64, 37, 37 * 3, 70
    c = pc.Cache(fmt, [N, 3], Hk, d, 32, seed=120, device="cuda")
    q, k, v = fused_qkv(N, Hq, Hk, d, 121)
    seq = torch.zeros(N, dtype=torch.int32, device="cuda")
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    rope = pc.rope_table(N, d).cuda()
    qo, ko = moda.moda_kv_append(q, k, v, *c.args(), seq, pos, rope=rope, **c.scales())
    kg, vg = moda.moda_kv_gather(*c.args(), seq, pos, **c.scales())
    settled()
    for x, out in ((q, qo), (k, ko)):
        want = pc.turned(x, rope, pos, False)
        size = x.double().abs().amax(dim=(1, 2), keepdim=True) * 2
        assert ((out.double() - want).abs() <= pc.HALF_BF16 * want.abs() + 4 * pc.HALF_FP32 * size).all()
    if fmt == "bf16":
        assert torch.equal(kg, ko) and torch.equal(vg, v)
    else:
        assert torch.equal(kg.double(), pc.mx4_quantised(pc.turned(k, rope, pos, False)))
        assert torch.equal(vg.double(), pc.mx4_quantised(v.double()))


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
def test_calls_follow_one_another_without_waits(fmt):
    """Every call reads what the one before it in the stream wrote, tensors and
    workspace used again at once; the bits of the same calls with a
    synchronisation after each, three times over."""
    d, Hk, G, L, steps = 128, 4, 4, 24, 30
    Hq, scale = Hk * G, d ** -0.5
    total = [400, 33, 1000]
    rope = pc.rope_table(1000 + steps, d).cuda()
    q, k, v = fused_qkv(3, Hq, Hk, d, 130)
    base = q._base
    seq = torch.arange(3, dtype=torch.int32, device="cuda")
    ws = torch.empty(moda.moda_decode_paged_workspace_bytes(Hq, Hk, d) // 4, device="cuda")
    qo = torch.empty(3, Hq, d, dtype=torch.bfloat16, device="cuda")
    ko = torch.empty(3, Hk, d, dtype=torch.bfloat16, device="cuda")
    kb, vb = torch.empty_like(ko), torch.empty_like(ko)
    kd, vd = depth(3, Hk, L, d, 131)
    start = base.clone()

    def run(wait):
        c = pc.Cache(fmt, [t + steps for t in total], Hk, d, 16, seed=132, device="cuda")
        base.copy_(start)
        n = torch.tensor(total, dtype=torch.int32, device="cuda")
        got = []
        o, lse = torch.empty_like(qo), torch.empty(3, Hq, device="cuda")
        for _ in range(steps):
            moda.moda_kv_append(q, k, v, *c.args(), seq, n, rope=rope, q_out=qo, k_out=ko, **c.scales())
            wait()
            moda.moda_kv_gather(*c.args(), seq, n, k=kb, v=vb, **c.scales())
            wait()
            n.add_(1)
            moda.moda_decode_paged(qo, *c.args(), n, scale, kd=kd, vd=vd, o=o, lse=lse, workspace=ws,
                                   **c.scales())
            wait()
            got += [o.clone(), lse.clone(), kb.clone(), vb.clone()]
            # the next step's rows depend on this one's result
            base.view(3, -1)[:, : Hq * d].copy_((o.float() * 3).view(3, -1).bfloat16())
            base.view(3, -1)[:, Hq * d : (Hq + Hk) * d].copy_(kb.view(3, -1))
        torch.cuda.synchronize()
        return got

    want = run(torch.cuda.synchronize)
    for _ in range(3):
        for a, b in zip(run(lambda: None), want):
            assert torch.equal(a, b)
    settled()


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
def test_what_a_call_allocates_belongs_to_its_stream(fmt, monkeypatch):
    """Outputs and workspace of a call on a stream of its own come from that
    stream's memory: what the current stream's pool hands out may still be in
    use there, and would be handed out again while the call runs."""
    d, Hk, lens = 64, 2, [70, 5]
    c = pc.Cache(fmt, lens, Hk, d, 16, seed=3, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    seq = torch.arange(2, dtype=torch.int32, device="cuda")
    q, k, v = fused_qkv(2, 8, Hk, d, 4)
    want = (moda.moda_kv_append(q, k, v, *c.args(), seq, n - 1, **c.scales()),
            moda.moda_kv_gather(*c.args(), seq, n - 1, **c.scales()),
            moda.moda_decode_paged(q.contiguous(), *c.args(), n, 0.1, **c.scales()))
    qc, pos = q.contiguous(), n - 1
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on, empty = [], torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: (on.append(torch.cuda.current_stream()), empty(*a, **kw))[1])
    for stream in (side, side.cuda_stream, torch.cuda.default_stream().cuda_stream):
        on.clear()
        got = (moda.moda_kv_append(q, k, v, *c.args(), seq, pos, stream=stream, **c.scales()),
               moda.moda_kv_gather(*c.args(), seq, pos, stream=stream, **c.scales()),
               moda.moda_decode_paged(qc, *c.args(), n, 0.1, stream=stream, **c.scales()))
        assert len(on) == 7
        assert {s.cuda_stream for s in on} == {getattr(stream, "cuda_stream", stream)}
        settled()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
def test_captured_among_copies_and_other_streams(fmt, table_of):
    """A step captured where what comes before each call is not a kernel (a
    copy, a fill) or is two streams that meet; replayed on new inputs."""
    d, Hk, lens = 64, 2, [130, 17, 1]
    c = pc.Cache(fmt, lens, Hk, d, 16, seed=13, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    seq, pos, scale = torch.arange(3, dtype=torch.int32, device="cuda"), n - 1, d ** -0.5
    q, k, v = (torch.zeros(3, h, d, dtype=torch.bfloat16, device="cuda") for h in (4, Hk, Hk))
    new = [torch.zeros_like(t) for t in (q, k, v)]
    qo, o, kg, vg = torch.empty_like(q), torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ko, lse = torch.empty_like(k), torch.empty(3, 4, device="cuda")
    ws = torch.empty(moda.moda_decode_paged_workspace_bytes(4, Hk, d) // 4, device="cuda")
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def step():
        for t, x in zip((q, k, v), new):
            t.copy_(x)  # the append's predecessor is a copy
        moda.moda_kv_append(q, k, v, *c.args(), seq, pos, q_out=qo, k_out=ko, **c.scales())
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            kg.zero_()
            moda.moda_kv_gather(*c.args(), seq, pos, k=kg, v=vg, **c.scales())
        o.zero_()
        moda.moda_decode_paged(qo, *c.args(), n, scale, o=o, lse=lse, workspace=ws, **c.scales())
        torch.cuda.current_stream().wait_stream(side)
        # two streams end here, and the next call waits for both
        moda.moda_kv_append(None, kg, vg, *c.args(), seq, pos, k_out=ko, **c.scales())

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(main):
        step()
        main.synchronize()
        with torch.cuda.graph(graph, stream=main):
            step()
    for rep in range(3):
        for i, t in enumerate(new):
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(5 * rep + i)).bfloat16())
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        held = [t.clone() for t in (o, lse, kg, vg, ko)]
        with torch.cuda.stream(main):
            step()
        torch.cuda.synchronize()
        for a, b in zip(held, (o, lse, kg, vg, ko)):
            assert torch.equal(a, b)
        if fmt == "bf16":
            assert torch.equal(kg, new[1]) and torch.equal(vg, new[2])
        check_decode(c, new[0], lens, None, None, scale, o, lse)
    settled()


@pytest.mark.parametrize("G", [1, 8, 16])
def test_depth_slots_weigh_in_two_parts_over_4_bit_pages(G, table_of):
    """Where the depth slots hold nearly all of the weight, o is right to its
    own rounding and the sums' (pc.decode_reference without the rounding of a
    probability: two bf16 parts leave 2^-16 of it)."""
    d, Hk, L = 128, 2, 40
    lens = [33, 64]
    c = pc.Cache("mx4", lens, Hk, d, 16, seed=23, device="cuda")
    c.ks.fill_(96), c.vs.fill_(96)  # 2^-31: the rows' scores are 0, their values nothing
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.randn(2, Hk * G, d, generator=torch.Generator().manual_seed(24)).bfloat16().cuda()
    kd, vd = depth(2, Hk, L, d, 25)
    kd, vd = kd * 2, vd.abs()  # sums without cancellation
    scale = d ** -0.5
    o, lse = moda.moda_decode_paged(q, *c.args(), n, scale, kd=kd, vd=vd, **c.scales())
    settled()
    # the fill rows beyond the sequences hold no NaN here, and are not reached
    want, _, tol, _ = pc.decode_reference(c, q, lens, kd, vd, scale)
    # a = sum p |v| = o up to the rows' 2^-31: take HALF_BF16 of it off twice, give 2^-16 twice
    tight = tol - 2 * (pc.HALF_BF16 - 2.0 ** -16) * want.abs() + 2.0 ** -30
    assert ((o.double() - want).abs() <= tight).all()


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
def test_bad_lengths_and_pages_of_many(fmt):
    """test_decode_bad_lengths_and_pages with as many sequences as are cut into
    shares however narrow the table is, and one at a time."""
    d, Hk, lens, many = 64, 2, [40, 64, 20], 110
    c = pc.Cache(fmt, lens, Hk, d, 16, seed=24, fill=None, width=4, device="cuda")
    c.table[0, 3] = c.table[0, 0]
    q = torch.randn(3, 4, d, generator=torch.Generator().manual_seed(25)).bfloat16().cuda()
    n = torch.tensor([40, 1000, -3], dtype=torch.int32, device="cuda")
    ro, rl, to, tl = pc.decode_reference(c, q, [40, 64, 0], None, None, 0.125)
    o, lse = moda.moda_decode_paged(q.repeat(many, 1, 1), c.k, c.v, c.table.repeat(many, 1), n.repeat(many),
                                    0.125, **c.scales())
    settled(INVALID)
    assert ((o.double() - ro.repeat(many, 1, 1)).abs() <= to.repeat(many, 1, 1)).all()
    assert (o.view(many, 3, 4, d)[:, 2] == 0).all() and (lse.view(many, 3, 4)[:, 2] == -math.inf).all()
    wide = torch.full((3, 1024), -7, dtype=torch.int32, device="cuda")
    wide[:, :4] = c.table
    for b, bad, table in ((0, False, c.table), (1, True, c.table), (2, True, c.table), (2, True, wide)):
        o, lse = moda.moda_decode_paged(q[b : b + 1], c.k, c.v, table[b : b + 1], n[b : b + 1], 0.125, **c.scales())
        settled(INVALID if bad else 0)
        assert ((o.double() - ro[b]).abs() <= to[b]).all()
        assert b != 2 or (o == 0).all() and (lse == -math.inf).all()
    table = c.table.repeat(many, 1)
    table[1::3, 2] = c.num_pages
    lens = torch.tensor(lens, dtype=torch.int32, device="cuda").repeat(many)
    o, _ = moda.moda_decode_paged(q.repeat(many, 1, 1), c.k, c.v, table, lens, 0.125, **c.scales())
    settled(INVALID)
    ro, _, to, _ = pc.decode_reference(c, q, [40, 64, 20], None, None, 0.125)
    ok = ((o.double() - ro.repeat(many, 1, 1)).abs() <= to.repeat(many, 1, 1)).view(many, 3, -1).all(-1)
    assert ok[:, 0].all() and ok[:, 2].all()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (128, 48)])
def test_turned_keys_on_and_next_to_borders(d, rot, inter):
    """4-bit rows of K whose turned values lie on the borders between codes and
    between scales, and off them by 2^-12 to 2^-30 of the other half of the pair:
    every code is the exact value's (cosines and sines are powers of two, so that
    fp64 holds it), also where most of a value cancels."""
    g = torch.Generator().manual_seed(50 + rot + inter)
    border = torch.tensor([0.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 6.0, 3.0], dtype=torch.float64)
    N, Hk, page = 600, 2, 16
    pick = lambda: border[torch.randint(0, len(border), (N, Hk, d), generator=g)]  # noqa: E731
    sign = lambda: 1.0 - 2.0 * torch.randint(0, 2, (N, Hk, d), generator=g)  # noqa: E731
    k = pick() * sign() * torch.exp2(torch.randint(-3, 4, (N, Hk, 1), generator=g).double())
    k[::3, :, : d // 2] = k[::3, :, d // 2:]  # equal halves, which cancel where cos = -sin
    cos = torch.tensor([1.0, 0.5, -1.0, 2.0])[torch.randint(0, 4, (N, rot // 2), generator=g)]
    sin = torch.tensor([0.0, 2.0 ** -12, -2.0 ** -22, 2.0 ** -23, -2.0 ** -24, 2.0 ** -30, 1.0, -0.5])[
        torch.randint(0, 8, (N, rot // 2), generator=g)]
    rope = torch.cat((cos, sin), 1).cuda()
    k = k.bfloat16().cuda()
    c = pc.Cache("mx4", [N], Hk, d, page, device="cuda")
    seq, pos = torch.zeros(N, dtype=torch.int32, device="cuda"), torch.arange(N, dtype=torch.int32, device="cuda")
    moda.moda_kv_append(None, k, k, *c.args(), seq, pos, rope=rope, interleaved=inter, **c.scales())
    settled()
    want = pc.mx4_quantised(pc.turned(k, rope, pos, inter)).transpose(0, 1)
    assert torch.equal(c.rows("k", 0, N), want)
    assert torch.equal(c.rows("v", 0, N), pc.mx4_quantised(k.double()).transpose(0, 1))
