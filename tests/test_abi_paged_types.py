"""What is no tensor is refused as such, by name, in every argument of the paged calls."""
import numpy as np
import pytest

from test_abi_paged_args import CALLS, SLOW, arguments, ways  # noqa: F401 (a fixture)

import torch


@pytest.mark.parametrize("call,mx4", CALLS)
def test_what_is_no_tensor(ways, call, mx4):  # noqa: F811
    rec, _ = ways
    base = arguments(call, mx4)
    for name, t in base.items():
        if not isinstance(t, torch.Tensor):
            continue
        for x in ([1.0], 3, "x", np.zeros(tuple(t.shape), np.float32)):
            rec.seen = None
            with pytest.raises(TypeError, match=name):
                SLOW[call](**dict(base, **{name: x}))
            assert rec.seen is None
