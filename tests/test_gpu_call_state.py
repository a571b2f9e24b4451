"""Calls of one kernel that need different amounts of shared memory, from two host threads
at once and in one captured graph: a call must not take away what another one needs."""
import ctypes
import sys
import threading

import pytest
import torch

import sequence_depth_attention_gb300 as moda
from sequence_depth_attention_gb300 import build as mbuild

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mbuild.build()
    moda.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def select(max_pages, seed):
    """A choice over a table of max_pages pages: a maker of outputs, and of the call into given
    ones on the current stream."""
    Hk, G, d, page, S, held = 2, 4, 64, 16, 8, 300
    g = torch.Generator().manual_seed(seed)
    table = torch.full((1, max_pages), -7, dtype=torch.int32)
    table[0, :held] = torch.randperm(held, generator=g).to(torch.int32)
    table = table.cuda()
    q = torch.randn(1, Hk * G, d, generator=g).bfloat16().cuda()
    means = torch.randn(held, Hk, d, generator=g).bfloat16().cuda()
    k = torch.zeros(held, Hk, page, d, dtype=torch.bfloat16, device="cuda")
    seq, pos = i32([0]), i32([held * page - 1])

    def fresh():
        return tuple(torch.full(s, 99, dtype=torch.int32, device="cuda") for s in ((1, Hk, S), (1, Hk)))

    def bind(out):
        return lambda: moda.moda_select_pages(q, means, k, k, table, seq, pos, S, pages=out[0], rows=out[1])

    return fresh, bind


def mass(L, seed):
    """The same for the depth slots' mass, by the library's function itself: what Python does
    around it keeps two calls apart."""
    T, Hk, G, d = 64, 1, 16, 128
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(T, Hk * G, d, generator=g).bfloat16().cuda()
    kd = torch.randn(Hk, T, L, d, generator=g).bfloat16().cuda()
    lse = torch.full((T, Hk * G), 8.0, device="cuda")
    work = torch.empty(moda.moda_depth_mass_workspace_bytes(T, Hk, L) // 4, device="cuda")

    def fresh():
        return (torch.full((Hk, L), 99.0, device="cuda"),)

    def bind(out):
        f = moda.load().moda_depth_mass
        vp = ctypes.c_void_p
        tensors = q, kd, lse, out[0], work
        ptr = [vp(x.data_ptr()) for x in tensors]
        args = (*ptr[:3], T, Hk * G, Hk, d, L, ctypes.c_float(d ** -0.5), *ptr[3:], work.numel() * 4,
                vp(torch.cuda.current_stream().cuda_stream))

        def call():
            st = f(*args)
            assert st == 0, moda.moda_status_string(st)

        call.keeps = tensors
        return call

    return fresh, bind


# the kernel, and what makes one call need more shared memory than the other
KERNELS = [(select, (32768, 9000)), (mass, (1024, 8))]


def of_each_size(make, sizes):
    makers = [make(n, i) for i, n in enumerate(sizes)]
    want, got = ([fresh() for fresh, _ in makers] for _ in range(2))
    for (_, bind), out in zip(makers, want):
        bind(out)()
    torch.cuda.synchronize()
    return [bind for _, bind in makers], want, got


def settled(want, got):
    torch.cuda.synchronize()
    assert moda.moda_get_device_error() == 0
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("make,sizes", KERNELS, ids=lambda x: getattr(x, "__name__", None))
def test_two_sizes_in_one_graph(make, sizes):
    binds, want, got = of_each_size(make, sizes)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for bind, out in zip(binds, got):  # the larger first
            bind(out)()
    binds[1](want[1])()
    for _ in range(2):
        graph.replay()
    settled(want, got)


@pytest.mark.parametrize("make,sizes", KERNELS, ids=lambda x: getattr(x, "__name__", None))
def test_two_sizes_from_several_threads(make, sizes):
    binds, want, got = of_each_size(make, [sizes[i % 2] for i in range(6)])
    start, failed = threading.Barrier(len(binds)), []

    def run(bind, out, size):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                call = bind(out)
                start.wait(60)
                for _ in range(10000):
                    call()
        except Exception as e:  # noqa: BLE001 (told to the main thread)
            failed.append(f"{make.__name__}({size}): {e}")

    threads = [threading.Thread(target=run, args=(bind, out, sizes[i % 2]))
               for i, (bind, out) in enumerate(zip(binds, got))]
    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-5)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    assert not failed
    settled(want, got)
