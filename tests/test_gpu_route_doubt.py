"""GPU tests of the grouped router where fp32 cannot tell groups apart: sums of choices that cancel
(tolerances and oracle of test_gpu_route_groups; ids one by one)."""
import numpy as np
import pytest
import torch

from _gpu_helpers import DEV
from expert_slot_cache_amd import binding
from test_gpu_operators import dev
from test_gpu_route_groups import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [16.0, 1e3, 1e5])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,groups,each,kept,K", [(400, 2, 2, 1, 2), (200, 8, 4, 3, 4), (100, 8, 64, 4, 10), (60, 32, 3, 9, 8),
                                                 (60, 64, 16, 20, 12)])
def test_sums_that_cancel(T, groups, each, kept, K, score, size):
    """A group's two largest choices are near +size and -size: their sum is a difference of scores, and
    what each lost in fp32 goes by its size.  Scores differ by about that."""
    rng = np.random.default_rng(groups + each)
    bias = np.full((groups, each), -3 * size, np.float32)
    bias[:, 0], bias[:, 1] = size, -size
    place = np.argsort(rng.random((groups, each)), axis=1)
    near = rng.normal(size=(T, 1, each)) + size * 2.0 ** -22 * rng.normal(size=(T, groups, each))
    z = np.take_along_axis(near, place[None].repeat(T, 0), 2).astype(np.float32).reshape(T, -1)
    bias = np.take_along_axis(bias, place, 1).reshape(-1)
    check(dev(z), bias, K, score=score, renorm=False, n_groups=groups, kept=kept, group_top=2)


def test_two_groups_whose_sums_cancel():
    z = np.float32([[-0.03002781, 0.17396595, -0.03002714, 0.17396444]])
    bias = np.float32([16, -16, 16, -16])
    ids = torch.zeros(1, 2, dtype=torch.int32, device=DEV)
    binding.route_groups(dev(z), ids, torch.zeros(1, 2, device=DEV), bias=dev(bias), score="sigmoid", n_groups=2, kept_groups=1,
                         group_top=2)
    assert ids.tolist() == [[0, 1]]                    # 1.03587574 against 1.03587554
