"""GPU tests of the combine's gradient with 1, 4 and 16 waves to a token."""
import pytest

import test_gpu_operators as ops

pytestmark = pytest.mark.gpu

# 16 waves below 256 and rows above 256 pieces; 4 below 1280 and above 64, or where two thirds of
# the steps of 256 pieces are filled and a token's rows are more than 1024 pieces; one else.  Both
# sides of each border, both types.
WAVES = [(255, 8, 2056, "bf16"), (255, 8, 2048, "bf16"), (256, 8, 2056, "bf16"), (31, 60, 1032, "f32"), (300, 8, 512, "bf16"),
         (300, 8, 520, "bf16"), (300, 3, 257, "f32"), (1279, 4, 768, "bf16"), (1280, 4, 768, "bf16"), (1300, 8, 1360, "bf16"),
         (1300, 8, 1368, "bf16"), (1300, 2, 2728, "bf16"), (1300, 2, 2740, "bf16"), (641, 12, 1028, "f32"),
         (1300, 3, 2740, "bf16"), (1300, 4, 2048, "bf16"), (1300, 5, 2048, "bf16"), (1300, 1, 8192, "bf16"),
         (1300, 1, 8200, "bf16"), (3, 8, 12400, "f32")]


@pytest.mark.parametrize("T,K,H,kind", WAVES)
def test_gradient_at_each_count_of_waves(T, K, H, kind):
    ops.test_combine_rows_backward(T, K, 70, H, kind)
