"""CPU tests of where the grouped router's fp32 leaves an order open (csrc/route_doubt.hpp), against
exact fractions."""
import os
import shutil
import subprocess
from fractions import Fraction

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "expert_slot_cache_amd", "csrc")
INF = float("inf")
LOWEST = float(np.finfo(np.float32).min)


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path_factory.mktemp("doubt") / "route_doubt_driver")
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC,
                    os.path.join(ROOT, "tests", "native", "route_doubt_driver.cpp"), "-o", exe], check=True)

    def ask(lines):
        text = "".join(" ".join(str(v) for v in line) + "\n" for line in lines)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split("\n")[:-1]
        return [tuple(float.fromhex(v) if "x" in v else float(v) for v in line.split()) for line in out]
    return ask


def f32(v):
    return float(np.float32(v))


@pytest.mark.parametrize("pairs", [0, 1])
@pytest.mark.parametrize("size", [0.0, 0.5, 16.0, 1e3, 1e5, 1e30])
def test_what_a_group_s_sum_may_be_off(driver, size, pairs):
    """Choices score + bias, each score off by off / 2: the bound holds, and so it does where the two
    biases cancel, also after one more rounding (the sum and the bound are added)."""
    rng = np.random.default_rng(int(size) % 1000 + pairs)
    off = 2.0 ** -21
    lines, want = [], []
    for _ in range(3000):
        s = rng.random(2)
        signs = [1, -1] if rng.random() < 0.7 else [1, 1]
        b = [f32(sign * size * (1 + 1e-3 * rng.random())) for sign in signs]
        moved = [f32(v + off / 2 * 0.98 * rng.choice([-1, 1])) for v in s]
        c = [float(np.float32(m) + np.float32(v)) for m, v in zip(moved, b)]
        one, two = max(c), min(c)
        exact = [Fraction(v) + Fraction(w) for v, w in zip(s, b)]
        want.append(sum(exact) / 2 if pairs else exact[c.index(one)])
        lines.append((repr(one), repr(two), pairs, repr(off)))
    for (value, bound), true in zip(driver(lines), want):
        low, high = np.float32(value) - np.float32(bound), np.float32(value) + np.float32(bound)
        assert Fraction(float(low)) <= true <= Fraction(float(high))


def test_sums_of_infinite_and_lowest_choices(driver):
    got = driver([(INF, 1.0, 1, 1e-6), (INF, -INF, 1, 1e-6), (-INF, -INF, 1, 1e-6), (LOWEST, LOWEST, 1, 1e-6),
                  (3e38, 3e38, 1, 1e-6), (1.0, LOWEST, 1, 1e-6), (0.5, -INF, 1, 0.0), (INF, -1.0, 0, 1e-6), (-INF, -INF, 0, 1e-6)])
    assert [v for v, _ in got] == [INF, INF, -INF, LOWEST, f32(3e38), LOWEST / 2, 0.25, INF, -INF]
    assert [bound for _, bound in got[:3]] == [0, 0, 0] and all(np.isfinite(bound) for _, bound in got)


def test_choices_next_to_masked_ones_are_in_no_doubt(driver):
    off = 2.0 ** -21
    near = lambda *pairs: [v for v, in driver([(repr(x), repr(y), 2, repr(off)) for x, y in pairs])]      # noqa: E731
    assert near((0.5, -INF), (-1e5, -INF), (LOWEST, -INF), (-INF, -INF), (INF, 1.0), (INF, LOWEST), (INF, -INF), (INF, INF),
                (0.5, LOWEST), (2e38, -2e38)) == [0] * 10
    assert near((0.5, 0.5), (0.0, -0.0), (0.5, 0.5 - off), (0.5 + 2 * off, 0.5), (1e5, f32(1e5 - 0.01)), (1e5, f32(1e5 - 0.04)),
                (LOWEST, LOWEST)) == [1, 1, 1, 0, 1, 0, 1]
