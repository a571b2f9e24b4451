"""Counts that do not fit the library's 32-bit arguments: refused by name, before anything is
allocated or called, not cut to what their low bits say."""
import pytest

import sequence_depth_attention_gb300 as moda

from test_abi_paged_args import ways  # noqa: F401 (a fixture)
from test_abi_paged_more import arguments, more  # noqa: F401 (a fixture)


@pytest.mark.parametrize("name", ["S", "sink", "recent"])
@pytest.mark.parametrize("x", [2**31, 2**32, 2**32 + 1, -2**31 - 1, -2**32, -2**32 + 2, 2**63, 2**64 + 1, 1e10])
def test_counts_of_more_than_32_bits(more, name, x):  # noqa: F811
    rec, ext = more
    a = dict(arguments("select", False), pages=None, rows=None)
    a[name] = x
    rec.seen = None
    assert ext.select(*a.values()) is None
    with pytest.raises(ValueError, match=name):
        moda.moda_select_pages(**a)
    assert rec.seen is None
