"""CPU pins of oracle/rows.py (the operators around the experts): e4m3 against torch's
type, gradients against differences, the sort against a sort of tuples, the router
against oracle/router.py."""
import numpy as np
import pytest
import torch

from oracle import router as orouter
from oracle import rows as orows


def test_e4m3_values_and_rounding_are_torchs():
    codes = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(orows.e4m3_widen(codes), ref, equal_nan=True)
    rng = np.random.default_rng(1)
    v = np.concatenate([rng.uniform(-448, 448, 4000), rng.normal(0, 0.02, 4000), ref[np.isfinite(ref)],
                        np.arange(-64, 64) * 2.0 ** -11]).astype(np.float32)
    got = torch.from_numpy(v).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(orows.e4m3_round(v), got)
    # halfway cases go to the even code
    assert orows.e4m3_round(np.array([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10])).tolist() == [16.0, 20.0, 0.0, 2.0 ** -8]


def test_block_scale_cases():
    assert orows.block_scale(np.zeros(3)) == 1.0
    assert orows.block_scale(np.array([448.0, -1.0])) == 1.0
    assert orows.block_scale(np.array([448.1])) == 2.0
    assert orows.block_scale(np.array([-224.0, np.inf, np.nan])) == 0.5
    assert orows.block_scale(np.array([1e-45])) == 2.0 ** -126


def test_route_equals_the_router_oracle_and_its_edges():
    rng = np.random.default_rng(2)
    z = rng.normal(size=(20, 12))
    z[3, 4] = z[3, 9]
    ids, w = orows.route(z, 5, False)
    p = orouter.softmax(z)
    assert np.array_equal(ids, orouter.top_k(z, 5))
    assert np.allclose(w, np.take_along_axis(p, ids.astype(np.int64), 1), rtol=1e-13)
    assert np.allclose(orows.route(z, 5, True)[1].sum(1), 1.0, rtol=1e-13)
    inf = np.inf
    ids, w = orows.route(np.array([[-inf, -inf, -inf], [0.0, inf, inf], [np.nan, 1.0, -inf]]), 2, False)
    assert ids.tolist() == [[0, 1], [1, 2], [1, 0]] and w.tolist() == [[0, 0], [0.5, 0.5], [1, 0]]


@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(renorm):
    rng = np.random.default_rng(3)
    z, dw = rng.normal(size=(4, 9)), rng.normal(size=(4, 3))
    ids, w = orows.route(z, 3, renorm)
    g = orows.route_grad(z, ids, w, dw, renorm)
    h = 1e-5
    for t in range(4):
        for e in range(9):
            up, down = z.copy(), z.copy()
            up[t, e] += h
            down[t, e] -= h
            (iu, wu), (idn, wd) = orows.route(up, 3, renorm), orows.route(down, 3, renorm)
            assert np.array_equal(iu, ids) and np.array_equal(idn, ids)
            # central difference: error about h^2 = 1e-10
            assert abs((((wu - wd) * dw).sum() / (2 * h)) - g[t, e]) < 1e-8


def test_sort_pairs_is_a_stable_sort():
    rng = np.random.default_rng(4)
    ids = rng.integers(-1, 7, (13, 4)).astype(np.int32)
    offsets, rows = orows.sort_pairs(ids, 6)
    order = sorted((int(ids[t, k]), t, k) for t in range(13) for k in range(4) if 0 <= ids[t, k] < 6)
    assert [int(rows[t, k]) for _, t, k in order] == list(range(len(order)))
    assert int((rows < 0).sum()) == 52 - len(order)
    assert offsets.tolist() == [sum(i < e for i, _, _ in order) for e in range(7)]


def test_combine_gradient_against_differences():
    rng = np.random.default_rng(5)
    ids = rng.integers(-1, 4, (5, 3)).astype(np.int32)
    _, rows = orows.sort_pairs(ids, 4)
    ys, w, d = rng.normal(size=(15, 6)), rng.normal(size=(5, 3)), rng.normal(size=(5, 6))
    d_ys, d_w = orows.combine_grad(d, ys, rows, w)
    # combine is linear in ys and in w: differences are exact but for rounding
    vy, vw = rng.normal(size=ys.shape), rng.normal(size=w.shape)
    base = (orows.combine(ys, rows, w) * d).sum()
    assert abs((orows.combine(ys + vy, rows, w) * d).sum() - base - (d_ys * vy).sum()) < 1e-10
    assert abs((orows.combine(ys, rows, w + vw) * d).sum() - base - (d_w * vw).sum()) < 1e-10


def test_scaled_product_by_hand():
    x = orows.widen_rows(np.ones((3, 130)), np.array([[1.0, 2.0], [0.5, 1.0], [1.0, 1.0]]))
    w = orows.widen_matrix(np.ones((129, 130)), np.array([[1.0, 10.0], [2.0, 3.0]]))
    out = orows.scaled_product(x, [w, w], [0, 0, 2])
    assert out[0, 0] == 128 + 2 * 2 * 10 and out[0, 128] == 256 + 2 * 2 * 3
    assert out[1, 0] == 64 + 20 and np.isnan(out[2]).all()
