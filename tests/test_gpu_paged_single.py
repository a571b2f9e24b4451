"""The smallest appends through the C ABI on real tensors: one token without
queries, rotation or k_out, whose strides are never stepped."""
import ctypes

import pytest
import torch

import sequence_depth_attention_gb300 as moda
from sequence_depth_attention_gb300 import binding
from sequence_depth_attention_gb300 import build as mbuild

import paged_common as pc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mbuild.build()
    return binding.load()


@pytest.mark.parametrize("fmt", ["bf16", "mx4"])
@pytest.mark.parametrize("d,Hk,page", [(64, 2, 16), (128, 1, 128)])
def test_one_token_without_queries(lib, fmt, d, Hk, page):
    c = pc.Cache(fmt, [5], Hk, d, page, seed=1, device="cuda")
    k, v = (torch.randn(1, Hk, d, generator=torch.Generator().manual_seed(2 + i)).bfloat16().cuda() for i in range(2))
    seq, pos = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((1,), 4, dtype=torch.int32, device="cuda")
    before = c.bits()
    cache = binding._PagedKv(binding.MODA_KV_MX4 if fmt == "mx4" else binding.MODA_KV_BF16, c.num_pages, page, Hk, d,
                             1, c.max_pages, *(t.data_ptr() if t is not None else None
                                               for t in (c.k, c.v, c.ks, c.vs)), c.table.data_ptr())
    stream = torch.cuda.current_stream().cuda_stream
    rc = lib.moda_kv_append(None, k.data_ptr(), v.data_ptr(), 0, 3, 5, None, 0, 0, 0, seq.data_ptr(), pos.data_ptr(),
                            1, 0, ctypes.byref(cache), None, None, stream)
    torch.cuda.synchronize()
    assert rc == 0 and moda.moda_get_device_error() == 0
    hold = (lambda x: x.double()) if fmt == "bf16" else (lambda x: pc.mx4_quantised(x.double()))
    for which, x in (("k", k), ("v", v)):
        assert torch.equal(c.rows(which, 0, 5)[:, 4], hold(x[0]))
    # every other row is as it was
    at = int(c.table[0, 0])
    for was, t in zip(before, [t for t in (c.k, c.v, c.ks, c.vs) if t is not None]):
        was[at, :, 4] = t[at, :, 4]
        assert torch.equal(was.view(torch.uint8), t.view(torch.uint8))
