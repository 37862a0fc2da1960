"""CPU test that the expert products' rules (csrc/product_tile.hpp) have no kernel built that no sizes reach,
and that a format known to the compiler takes the tiles that the same format at run time takes."""
import os
import shutil
import subprocess

import pytest

from test_expert_tiles import tile  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_tile_that_is_built_is_taken(tile, tmp_path):  # noqa: F811
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "expert_tiles_built_driver")
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", "-I", os.path.join(ROOT, "expert_slot_cache_amd", "csrc"),
                    os.path.join(ROOT, "tests", "native", "expert_tiles_built_driver.cpp"), "-o", exe], check=True)
    sizes = [(s, b, M, G, N) for s in (0, 1) for b in (0, 1) for G in (1, 8, 64) for M in (1, 40, 300, 600, 2048, 8192, 65536)
             for N in (64, 1024, 8192)]
    text = "".join(f"{s} {b} {M} {G} {N} {int(G > 1)}\n" for s, b, M, G, N in sizes)
    out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
    built, taken = out.split("end\n")
    built = {tuple(int(v) for v in line.split()) for line in built.split("\n")[:-1]}
    taken = [tuple(int(v) for v in line.split()) for line in taken.split("\n")[:-1]]
    assert len(taken) == len(sizes)
    assert built == {(s, b, *t) for (s, b, *_), t in zip(sizes, taken)}
    assert len(built) == 6 + 6 + 3 + 4                 # bf16 both ways, fp32 plain, fp32 SwiGLU
    for (s, b, M, G, N), t in list(zip(sizes, taken))[::5]:
        assert tile("s" if s else "p", b, M, G, N, 0, G > 1)[:2] == t
