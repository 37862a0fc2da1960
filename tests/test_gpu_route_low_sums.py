"""GPU tests of the grouped router where two choices of a group add up to less than fp32's lowest value
(tolerances and oracle of test_gpu_route_groups; ids one by one)."""
import numpy as np
import pytest

from test_gpu_operators import INF, dev
from test_gpu_route_groups import check

pytestmark = pytest.mark.gpu


def test_negative_sums_that_run_over_fp32():
    """Biases near fp32's lowest value: two of them have no sum in fp32, and differ in fp64."""
    rng = np.random.default_rng(4)
    bias = np.full(32, -2.0e38, np.float32)
    bias += (rng.integers(0, 1000, 32) * 2.0 ** 110).astype(np.float32)
    check(dev(rng.normal(size=(9, 32)).astype(np.float32)), bias, 3, score="sigmoid", renorm=False, n_groups=8, kept=3, group_top=2)


@pytest.mark.parametrize("value", [float(np.finfo(np.float32).min), -2e38])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_a_group_of_low_biases_goes_before_a_masked_one(score, value):
    """Groups: all -inf, all near the lowest value, live, all -inf.  The second and the third are kept."""
    bias = np.zeros((4, 8), np.float32)
    bias[[0, 3]] = -INF
    bias[1] = value
    z = np.random.default_rng(2).normal(size=(40, 32)).astype(np.float32)
    for top in (1, 2):
        check(dev(z), bias.reshape(-1), 10, score=score, renorm=False, n_groups=4, kept=2, group_top=top)
