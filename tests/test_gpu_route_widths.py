"""GPU tests of the router and its gradient at every width of its selection, those of 17 to 32
experts and the borders of 16, 32, 64 .. among them."""
import pytest

import test_gpu_operators as ops

pytestmark = pytest.mark.gpu

WIDTHS = [(50, 17, 5), (33, 31, 31), (64, 32, 4), (40, 24, 8), (21, 16, 16), (9, 2, 1), (30, 3, 2), (19, 33, 33),
          (25, 63, 12), (17, 65, 9), (12, 127, 20), (11, 129, 40), (10, 255, 64), (15, 257, 6), (9, 511, 11), (9, 513, 12),
          (8, 1025, 5), (9, 2049, 9)]


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,K", WIDTHS)
def test_route_at(T, E, K, kind, renorm):
    ops.test_route(T, E, K, kind, renorm)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,K", WIDTHS)
def test_route_backward_at(T, E, K, kind, renorm):
    ops.test_route_backward(T, E, K, kind, renorm)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,K", [(60, 31, 20), (90, 17, 17), (70, 32, 6), (41, 2, 2), (33, 15, 9), (28, 255, 30), (20, 513, 64)])
def test_route_of_many_equal_logits_at(T, E, K, kind):
    ops.test_route_of_many_equal_logits(T, E, K, kind)
