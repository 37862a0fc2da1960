"""CPU pins of oracle/experts.py at NaN and the infinities: each activation and slope as its formula has it."""
import numpy as np
import pytest

from oracle import experts as oe

H = np.array([[np.nan, np.inf, -np.inf, 0.0, -0.0, 2.0, -2.0, 1.0]])


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
def test_nan_stays_nan(act):
    with np.errstate(invalid="ignore"):
        a, s = oe.activate(H, act)[0], oe.slope(H, act)[0]
    assert np.isnan(a[0]) and a[1] == np.inf
    assert not np.isnan(a[3:]).any() and not np.isnan(s[3:]).any()
    assert np.isnan(s[0]) == (act != "none")
    if act == "relu":
        assert a.tolist()[2:] == [0, 0, 0, 2, 0, 1] and s.tolist()[1:] == [1, 0, 0, 0, 1, 0, 1]


def test_nan_in_either_half_of_swiglu():
    h = np.array([[np.nan, 1.0, 1.0, np.nan]])
    assert np.isnan(oe.activate(h, "swiglu")).all()
    d, _ = oe.activation_grad(np.ones((1, 2)), h, None, 4, "swiglu")
    assert np.isnan(d).tolist() == [[True, True, True, False]]
