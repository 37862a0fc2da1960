"""GPU tests of the matrices' gradient where the rows that count lie past 2^31 elements.  Every other row
holds other values, so that one of them in the sum, or a row left out of it, shows.

Tolerance: 2 (n + 4) u of the sum of the magnitudes, n = 700 the rows in the sum (test_gpu_expert_product):
9e-5 of it, where one row in 700 is worth 1.4e-3."""
import numpy as np
import pytest
import torch

from _gpu_helpers import DEV
from expert_slot_cache_amd import binding
from test_gpu_expert_large import fresh
from test_gpu_expert_product import sum_err
from test_gpu_operators import dev

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
M, LAST = 1_100_000, 700


@pytest.mark.parametrize("N,K", [(2048, 64), (64, 2048)])
@pytest.mark.parametrize("by", ["offsets", "zeros"])
def test_a_matrix_gradient_of_rows_far_down(N, K, by):
    assert M * max(N, K) > 1 << 31 and (M - LAST) * max(N, K) > 1 << 31
    d, x = fresh(M, N, seed=1).abs_(), fresh(M, K, seed=2).abs_()
    if by == "zeros":                                  # the whole length is summed
        d[:-LAST] = 0
    a, b = d[-LAST:].double(), x[-LAST:].double()
    want = a.t().contiguous() @ b                      # of positive values: the magnitudes' sum, too
    for off in (None,) if by == "zeros" else ([M - LAST, M], [0, 0, M - LAST, M, M]):
        G = 1 if off is None else len(off) - 1
        g = 0 if G == 1 else 2
        if G > 1:
            off[1] = off[2] = M - LAST                 # group 0 has the other rows
            off[3] = off[4] = M
        dw = torch.full((G, N, K), 7.0, device=DEV)
        db = torch.full((G, N), 7.0, device=DEV)
        offsets = None if off is None else dev(np.int32(off))
        binding.expert_product_backward(d, x, None, d_w=dw, offsets=offsets)
        binding.activation_backward(d, None, None, d_bias=db, offsets=offsets)
        assert ((dw[g].double() - want).abs() <= want * sum_err(LAST)).all(), off
        total = a.sum(0)
        assert ((db[g].double() - total).abs() <= total * sum_err(LAST)).all(), off
        if G > 1:
            assert not bool(dw[1].any()) and not bool(dw[3].any()) and not bool(db[[1, 3]].any())
