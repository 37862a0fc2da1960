"""CPU pins of oracle/experts.py: the router against oracle/rows.py and hand cases, every gradient
against differences."""
import math

import numpy as np
import pytest

from oracle import experts as oe
from oracle import rows as orows


@pytest.mark.parametrize("renorm", [False, True])
def test_softmax_without_bias_is_the_plain_router(renorm):
    z = np.random.default_rng(1).normal(size=(30, 24))
    z[3] = -np.inf
    z[4, ::2] = -np.inf
    z[5, 7] = np.nan
    z[6, [2, 9]] = np.inf
    ids, w = oe.route_groups(z, None, 6, score="softmax", renorm=renorm)
    ref_ids, ref_w = orows.route(z, 6, renorm)
    assert np.array_equal(ids, ref_ids) and np.allclose(w, ref_w, rtol=1e-13, atol=1e-300)


def test_groups_by_hand():
    # sigmoid(0) = 0.5 everywhere: the bias alone orders.  Groups of three: tops 0.9, 0.6 + 0.5, 0.8
    z = np.zeros((1, 9))
    bias = np.array([0.4, -9, -9, 0.1, 0.0, -9, 0.3, -0.2, -9])
    run = lambda **k: oe.route_groups(z, bias, 2, score="sigmoid", renorm=False, n_groups=3, **k)[0][0].tolist()   # noqa: E731
    assert run(kept=1, group_top=1) == [0, 1]          # 0.9 is the largest single choice
    assert run(kept=1, group_top=2) == [3, 4]          # 0.6 + 0.5 against 0.9 - 8.5 and 0.8 + 0.3
    assert run(kept=2, group_top=1) == [0, 6]
    assert run(kept=3, group_top=1) == [0, 6]
    z[0, 3] = -np.inf                                  # masked: group 1 counts expert 4 alone
    assert run(kept=1, group_top=2) == [6, 7]
    z[0, 4] = z[0, 5] = np.nan                         # a group of masked experts comes last
    assert run(kept=2, group_top=2) == [0, 6]
    assert oe.route_groups(z, bias, 9, score="sigmoid", renorm=True, n_groups=3, kept=3)[0][0].tolist() == [0, 6, 7, 1, 2, 8, 3, 4, 5]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_is_the_differences(score, renorm):
    rng = np.random.default_rng(7)
    z, bias, d_w = rng.normal(size=(4, 12)), 0.3 * rng.normal(size=12), rng.normal(size=(4, 5))
    kw = dict(score=score, renorm=renorm, scale=2.5)
    ids, w = oe.route_groups(z, bias, 5, n_groups=4, kept=3, group_top=2, **kw)

    def loss(v):                                       # at the ids chosen: they do not move
        total = 0.0
        for t in range(4):
            s = oe.scores(v[t], score)[ids[t]]
            total += (2.5 * (s / s.sum() if renorm else s) * d_w[t]).sum()
        return total

    g = oe.route_groups_grad(z, ids, w, d_w, score=score, renorm=renorm, scale=2.5)
    for t, e in [(0, ids[0, 0]), (1, ids[1, 4]), (2, ids[2, 2]), (3, 0), (0, 11)]:
        up, dn = z.copy(), z.copy()
        up[t, e] += 1e-5
        dn[t, e] -= 1e-5
        assert math.isclose((loss(up) - loss(dn)) / 2e-5, g[t, e], rel_tol=1e-6, abs_tol=1e-8)


@pytest.mark.parametrize("act", oe.ACTS)
def test_product_gradients_are_the_differences(act):
    rng = np.random.default_rng(9)
    M, G, N, K = 7, 3, 6, 5
    offsets = [1, 3, 3, 6]                             # row 0 and row 6 lie in no group, group 1 has none
    x, w, bias = rng.normal(size=(M, K)), rng.normal(size=(G, N, K)), rng.normal(size=(G, N))
    cols = N // 2 if act == "swiglu" else N
    d_out = rng.normal(size=(M, cols))

    def loss(x, w, bias):
        return np.nansum(oe.product(x, w, offsets, bias, None, act)[0] * d_out)

    out, h = oe.product(x, w, offsets, bias, None, act)
    assert np.isnan(out[[0, 6]]).all() and not np.isnan(out[1:6]).any()
    d_pre, d_bias = oe.activation_grad(d_out, np.nan_to_num(h), offsets, N, act)
    d_x, d_w = oe.product_grad(np.nan_to_num(d_pre), x, w, offsets)
    assert (d_w[1] == 0).all() and (d_bias[1] == 0).all()
    for name, v, g in [("x", x, d_x), ("w", w, d_w), ("bias", bias, d_bias)]:
        for i in rng.permutation(v.size)[:12]:
            at = np.unravel_index(i, v.shape)
            if name == "x" and at[0] in (0, 6):
                continue
            args = dict(x=x, w=w, bias=bias)
            up, dn = v.copy(), v.copy()
            up[at] += 1e-6
            dn[at] -= 1e-6
            diff = (loss(**dict(args, **{name: up})) - loss(**dict(args, **{name: dn}))) / 2e-6
            assert math.isclose(diff, g[at], rel_tol=1e-5, abs_tol=1e-7), (name, at)
