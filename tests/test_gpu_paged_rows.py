"""The paged decode held to the arithmetic that include/moda.h states
(paged_tight.py), and every row of V at its own weight."""
import pytest
import torch

import sequence_depth_attention_gb300 as moda
from sequence_depth_attention_gb300 import build as mbuild

import paged_common as pc
import paged_tight as pt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mbuild.build()
    moda.load()


@pytest.fixture(params=[0, 16384], ids=["narrow", "wide"])
def table_of(request, monkeypatch):
    """Tables just wide enough (clusters for short batches) and wide ones (equal shares)."""
    monkeypatch.setattr(pc.Cache, "least_rows", request.param)
    return request.param


def queries(B, Hq, d, seed):
    return torch.randn(B, Hq, d, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


def depth(B, Hk, L, d, seed):
    if L == 0:
        return None, None
    g = torch.Generator().manual_seed(seed)
    return tuple(torch.randn(B, Hk, L, d, generator=g).bfloat16().cuda() for _ in range(2))


def decode(c, q, kd, vd, scale):
    n = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    o, _ = moda.moda_decode_paged(q, *c.args(), n, scale, kd=kd, vd=vd, **c.scales())
    torch.cuda.synchronize()
    assert moda.moda_get_device_error() == 0
    return o


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
@pytest.mark.parametrize("d,page,Hk,G,n", [
    (128, 16, 2, 4, 1000), (128, 64, 1, 8, 4097), (128, 128, 2, 16, 2047), (64, 32, 4, 1, 777),
    (64, 16, 1, 9, 3000), (64, 64, 3, 7, 130), (128, 32, 4, 2, 31), (128, 16, 1, 1, 9003),
])
def test_every_row_arrives_at_its_weight(fmt, d, page, Hk, G, n, table_of):
    """Each column of o is one row's value times its weight: a row left out, read
    twice or taken for another shows whatever the length."""
    c = pc.Cache(fmt, [n] * -(-n // (Hk * d)), Hk, d, page, seed=50, device="cuda")
    row = pt.single_rows(c, 51)
    q = queries(len(c.lens), Hk * G, d, 52)
    o = decode(c, q, None, None, d ** -0.5)
    for b in range(len(c.lens)):
        want, tol = pt.one(c, b, n, q, None, None, d ** -0.5)
        got = o[b].double().view(Hk, G, d)
        assert ((got - want).abs() <= tol).all(), row[b][((got - want).abs() > tol).any(1)].tolist()[:20]


RAGGED = [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 1000]


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
@pytest.mark.parametrize("G", [1, 3, 8, 16])
@pytest.mark.parametrize("d,page,Hk,L,lens", [
    (128, 16, 2, 0, RAGGED), (64, 64, 3, 17, RAGGED), (128, 32, 4, 24, [300, 2] * 20), (64, 16, 1, 70, [3001]),
    (128, 64, 1, 46, [701]),
])
def test_accuracy_as_documented(fmt, G, d, page, Hk, L, lens, table_of):
    """Values of one sign: no cancellation hides a weight's rounding."""
    c = pc.Cache(fmt, lens, Hk, d, page, seed=53, device="cuda")
    if fmt == "bf16":
        c.v = c.v.abs()
    else:
        c.v = c.v & 0x77
    q = queries(len(lens), Hk * G, d, 54)
    kd, vd = depth(len(lens), Hk, L, d, 55)
    if L:
        vd = vd.abs()
    o = decode(c, q, kd, vd, d ** -0.5)
    for b, n in enumerate(lens):
        want, tol = pt.one(c, b, n, q, kd, vd, d ** -0.5)
        assert ((o[b].double().view(Hk, G, d) - want).abs() <= tol).all()


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
@pytest.mark.parametrize("G", [1, 3, 5, 7, 9, 11, 13, 15])
def test_odd_head_counts_in_clusters(fmt, G, table_of):
    """d = 64 and odd G: the columns that a cluster joins do not fill its warps."""
    lens = [500, 1, 0, 64, 333]
    c = pc.Cache(fmt, lens, 1, 64, 16, seed=56, device="cuda")
    q = queries(len(lens), G, 64, 57)
    o = decode(c, q, None, None, 0.125)
    for b, n in enumerate(lens):
        if n == 0:
            assert (o[b] == 0).all()
            continue
        want, tol = pt.one(c, b, n, q, None, None, 0.125)
        assert ((o[b].double().view(1, G, 64) - want).abs() <= tol).all()
