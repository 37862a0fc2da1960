"""GPU tests of the grouped router with experts out of service (tolerances and oracle of
test_gpu_route_groups; ids one by one)."""
import numpy as np
import pytest

from test_gpu_operators import INF, dev
from test_gpu_route_groups import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("live", [8, 9, 10, 11])
@pytest.mark.parametrize("value", [-INF, float(np.finfo(np.float32).min)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,kept", [(64, 1, 1), (64, 8, 4), (512, 8, 4), (1024, 16, 3)])
def test_experts_out_of_service(E, groups, kept, score, value, live):
    """Whole columns without service, by logit or by bias, so that K = 8, 9, .. experts are left."""
    rng = np.random.default_rng(E + live)
    z = rng.normal(size=(70, E)).astype(np.float32)
    bias = (0.1 * rng.normal(size=E)).astype(np.float32)
    out = rng.permutation(E)[live:]
    masked = bias.copy()
    masked[out] = value
    for top in (1, 2):
        kw = dict(score=score, renorm=True, n_groups=groups, kept=kept, group_top=top)
        check(dev(z), masked, 8, **kw)
        z2 = z.copy()
        z2[:, out] = -INF
        check(dev(z2), bias, 8, **kw)
        check(dev(z2), None, 8, **kw)
