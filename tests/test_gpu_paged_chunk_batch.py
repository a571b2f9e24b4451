"""Chunks of new tokens in batches most of whose sequences have none: a table of all
requests of a server, of which a few take part in a step."""
import math

import pytest
import torch

import sequence_depth_attention_gb300 as moda
from test_gpu_paged_chunk import _built, check, chunk, i32, run, settled  # noqa: F401 (_built is a fixture)

pytestmark = pytest.mark.gpu


def spread(x, B, at):
    """The chunk x of len(at) sequences as sequences at[i] of B; the others have no tokens,
    every second one rows all the same (that no page holds: none of them is looked at)."""
    c, q, starts, lens, kd, vd = x
    table = torch.full((B, c.max_pages), -7, dtype=torch.int32, device="cuda")
    table[torch.tensor(at, device="cuda")] = c.table
    c.table = table
    rows = torch.zeros(B, dtype=torch.int32)
    rows[1::2] = c.max_pages * c.page
    s = torch.zeros(B + 1, dtype=torch.int32)
    for i, b in enumerate(at):
        rows[b] = lens[i]
        s[b + 1 :] = starts[i + 1]
    return c, q, s, rows, kd, vd


BATCHES = [  # sequences, those with tokens
    (7, [6]), (512, [0, 511]), (513, [1, 2, 512]), (700, [0, 31, 32, 33, 600]), (1500, [5, 6, 7, 8, 1022, 1499]),
    (4096, [0, 4095]), (5000, [17, 18, 4000, 4001]),
]


@pytest.mark.parametrize("fmt,d", [("bf16", 128), ("bf16", 64), ("mx4", 128)])
@pytest.mark.parametrize("B,at", BATCHES, ids=lambda x: str(x) if isinstance(x, int) else f"{len(x)}")
def test_few_of_many_sequences(fmt, d, B, at):
    n = len(at)
    new = [(1, 40, 3, 9, 2, 17)[i % 6] for i in range(n)]
    past = [(300, 0, 1000, 128, 77, 5)[i % 6] for i in range(n)]
    x = chunk(fmt, new, past, 4, 1, d, 3, 32, pad=2)
    c, q, starts, lens, kd, vd = x
    held = c.table.clone()
    _, _, s, rows, _, _ = spread(x, B, at)
    o = torch.full(q.shape, 3.5, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 3.5, dtype=torch.float32, device="cuda")
    moda.moda_prefill_paged(q, *c.args(), s.cuda(), rows.cuda(), d ** -0.5, kd=kd, vd=vd, o=o, lse=lse, **c.scales())
    settled()
    c.table = held
    check(c, q, starts, lens, kd, vd, d ** -0.5, o, lse)


def test_a_batch_of_empty_sequences_takes_no_time():
    """Two sequences of 65536, whose shares of the work meet in one CTA: what lies between
    them is passed over at once (0.2 ms; one by one 6 ms)."""
    x = chunk("bf16", [8, 8], [992, 992], 4, 1, 128, 0, 16)
    c, q, starts, lens, kd, vd = x
    held = c.table.clone()
    _, _, s, rows, _, _ = spread(x, 65536, [0, 65535])
    s, rows = s.cuda(), rows.cuda()
    best = math.inf
    for _ in range(5):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        a.record()
        o, lse = moda.moda_prefill_paged(q, *c.args(), s, rows, 0.1)
        b.record()
        settled()
        best = min(best, a.elapsed_time(b))
    c.table = held
    check(c, q, starts, lens, kd, vd, 0.1, o, lse)
    assert best < 2.0, f"{best:.2f} ms"


@pytest.mark.parametrize("fmt,d", [("bf16", 128), ("bf16", 64), ("mx4", 128), ("mx4", 64)])
def test_infinite_values_before_many_short_tiles(fmt, d):
    """Tiles of two halves whose border holds infinities and NaN, each with a run of tiles of
    one half behind it in the same CTA's share: what a tile had taken out is told apart from
    what the tiles behind it had, or had not, for both halves."""
    G, L = 4, 2
    P = 128 // G
    run_of = [2 * P] + [1] * 300
    new = run_of * 10
    past = [3] * len(new)
    x = chunk(fmt, new, past, G, 1, d, L, 16)
    c, q, starts, lens, kd, vd = x
    clean, clean_lse = run(*x, d ** -0.5)
    tables = c.table[torch.arange(0, len(new), len(run_of), device="cuda")].long()
    row = 3 + P // 2  # seen by the tokens from P / 2 on: some of the first half, all of the second
    page, off = tables[:, row // 16], row % 16
    if fmt == "bf16":
        for col, value in ((5, math.nan), (6, math.inf), (7, -math.inf)):
            c.v[page, 0, off, col] = value
        cols = slice(5, 8)
    else:
        c.vs[page, 0, off, 0] = 255
        cols = slice(0, 32)
    last = torch.tensor(starts[0 : len(new) : len(run_of)], device="cuda") + 2 * P - 1
    vd[1, last, 0, d - 1] = math.inf  # and of one token of the second half in a slot of its own
    hit = torch.zeros(q.shape, dtype=torch.bool, device="cuda")
    for first in starts[0 : len(new) : len(run_of)]:
        hit[first + P // 2 : first + 2 * P, :, cols] = True
        hit[first + 2 * P - 1, :, d - 1] = True
    for _ in range(20):
        o, lse = run(*x, d ** -0.5)
        assert torch.equal(lse, clean_lse) and torch.equal(o[~hit], clean[~hit])
        assert not torch.isfinite(o[hit]).any()
        if fmt == "bf16":
            for first in starts[0 : len(new) : len(run_of)]:
                seen = o[first + P // 2 : first + 2 * P]
                assert torch.isnan(seen[..., 5]).all() and (seen[..., 6] == math.inf).all()
                assert (seen[..., 7] == -math.inf).all()
        assert (o[last, :, d - 1] == math.inf).all()
