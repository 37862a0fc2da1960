"""CPU test of the expert products' launches (csrc/product_tile.hpp): every workgroup has a place, few
places are empty, and no dimension has 2^32 lanes or more than the hardware counts."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_grids(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "grid_driver")
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", "-I", os.path.join(ROOT, "expert_slot_cache_amd", "csrc"),
                    os.path.join(ROOT, "tests", "native", "grid_driver.cpp"), "-o", exe], check=True)
    sizes = [(n, waves) for waves in (1, 2, 4, 8) for p in (0, 3, 20, 22, 23, 24, 25, 26, 27) for n in
             (2 ** p - 8, 2 ** p, 2 ** p + 8, 3 * 2 ** p // 2) if n > 0]
    text = "".join(f"{n} {w}\n" for n, w in sizes)
    out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split("\n")[:-1]
    assert len(out) == len(sizes)
    for (n, waves), line in zip(sizes, out):
        x, y = (int(v) for v in line.split())
        assert n <= x * y < n + 8 * y + y, (n, waves)
        assert x * 64 * waves < 1 << 32 and y < 1 << 16 and x * y < 1 << 31
        assert y == 1 or x % 8 == 0
        assert (y == 1) == (n * 64 * waves < 1 << 32)
