"""Pages that are not in the pool among pages whose scores are no better: by their place."""
import math

import pytest
import torch

from test_gpu_page_select import INVALID, _built, bare, choose, i32, normal  # noqa: F401 (_built is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("worst", [-math.inf, math.nan])
@pytest.mark.parametrize("pages", [20, 600])
def test_a_missing_page_counts_as_minus_infinity(worst, pages):
    """Three pages with finite scores, one missing, the others at -infinity (or NaN, which counts
    as that): the three first, then the first places of the rest, the missing page's among them."""
    d, page, missing = 64, 16, 2
    c = bare([pages * page], 1, d, page)
    q = torch.ones(1, 4, d, dtype=torch.bfloat16, device="cuda")
    means = normal(c.num_pages, 1, d, seed=5)
    means[:, :, 7] = worst
    finite = [6, 11, 14]
    ids = c.table[0].clone()
    means[ids[finite].long()] = 1.0
    c.table[0, missing] = c.num_pages
    for S, want in ((4, [6, 11, 14]), (6, [0, 1, 6, 11, 14]), (7, [0, 1, 2, 6, 11, 14]), (8, [0, 1, 2, 3, 6, 11, 14])):
        got, rows = choose(c, q, means, i32([0]), i32([pages * page - 1]), S, 0, 1, want=INVALID)
        expect = [-1 if i == missing else ids[i].item() for i in want + [pages - 1]]
        assert got[0, 0].tolist() == expect and rows[0, 0] == S * page
