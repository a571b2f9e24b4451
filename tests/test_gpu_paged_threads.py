"""The calls over chunks and selected pages from several host threads, a stream and a workspace
each: results are those of one call after another."""
import threading

import pytest
import torch

import sequence_depth_attention_gb300 as moda
import paged_chunk_common as cc
from test_gpu_paged_chunk import _built, chunk, i32, settled  # noqa: F401 (_built is a fixture)

pytestmark = pytest.mark.gpu


def program(i):
    """A thread's calls over its own cache, from inputs to outputs; every third has 4-bit pages, and
    sizes differ."""
    fmt, d = ("mx4" if i % 3 == 2 else "bf16"), (64, 128)[i % 2]
    Hk, G, L, S = 2, (4, 8, 1)[i % 3], 3, 5
    new, past = [4, 0, 30 + i], [300, 17, 1000 * i]
    c, q, starts, lens, kd, vd = chunk(fmt, new, past, Hk * G, Hk, d, L, 16, seed=i)
    at = [(b, t) for b in range(3) for t in range(past[b], lens[b])]
    seq, pos = (i32([x[j] for x in at]) for j in (0, 1))
    full = torch.nan_to_num(cc.page_means(c).bfloat16())
    st, ln = i32(starts), i32(lens)
    dk, dv = (x.permute(1, 2, 0, 3) for x in (kd, vd))

    def call():
        o, lse = moda.moda_prefill_paged(q, *c.args(), st, ln, 0.1, kd=kd, vd=vd, **c.scales())
        means = moda.moda_page_means(*c.args(), seq, pos, full.clone(), **c.scales())
        pages, rows = moda.moda_select_pages(q.contiguous(), means, *c.args(), seq, pos, S, **c.scales())
        o2, lse2 = moda.moda_decode_selected(q.contiguous(), c.k, c.v, pages, rows, 0.1, kd=dk, vd=dv, **c.scales())
        return o, lse, means, pages, rows, o2, lse2

    return call


def test_calls_from_several_threads():
    calls = [program(i) for i in range(6)]
    want = [call() for call in calls]
    settled()
    got, failed, start = [None] * len(calls), [], threading.Barrier(len(calls))

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait(60)
                got[i] = [calls[i]() for _ in range(50)]
        except Exception as e:  # noqa: BLE001 (told to the main thread)
            failed.append(f"{i}: {e}")

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    settled()
    for w, runs in zip(want, got):
        for g in runs:
            assert all(torch.equal(x, y) for x, y in zip(w, g))
