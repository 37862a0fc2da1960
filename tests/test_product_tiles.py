"""CPU tests of the rule that picks a product's tile (csrc/product_tile.hpp): each case that
tests/test_gpu_product_stages.py stands on takes the tile it is listed under, its rows use every
stage of the ring again, and no tile of the rule is left out."""
import os
import re
import shutil
import subprocess

import pytest

import test_gpu_product_stages as stages

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "expert_slot_cache_amd", "csrc")


@pytest.fixture(scope="module")
def tile(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path_factory.mktemp("tile") / "product_tile_driver")
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC,
                    os.path.join(ROOT, "tests", "native", "product_tile_driver.cpp"), "-o", exe], check=True)

    def ask(swiglu, M, G, N):
        r = subprocess.run([exe], input=f"{int(swiglu)} {M} {G} {N} {int(G > 1)}\n", capture_output=True, text=True, check=True)
        return tuple(int(v) for v in r.stdout.split())
    return ask


def _rule_tiles():
    text = open(os.path.join(CSRC, "product_tile.hpp")).read()
    return {tuple(int(v) for v in m) for m in re.findall(r"Tile<(\d+), (\d+), (\d+), (\d+)>", text)}


def test_every_tile_has_cases_that_use_its_stages_again(tile):
    seen = set()
    for swiglu, table in ((False, stages.PRODUCTS), (True, stages.GATED)):
        for want, cases in table.items():
            kinds = set()
            for M, G, N, K in cases:
                TW, TT, waves, S = tile(swiglu, M, G, 2 * N if swiglu else N)
                assert (TW, TT) == want, (swiglu, M, G, N)
                seen.add((TW, TT, waves, S))
                blocks = -(-K // 128)
                assert blocks > S + 1, (swiglu, M, G, N, K)
                # scales four blocks at a time: two groups of four, each used again
                kinds.add("fours" if blocks % 4 == 0 and blocks >= 12 else "ones")
                kinds.add("short" if K % 128 else "whole")
            assert kinds == {"fours", "ones", "short", "whole"}, want
    assert seen == _rule_tiles()


@pytest.mark.parametrize("swiglu,M,G,N,want", [
    (False, 32768, 64, 4096, (256, 128)), (False, 1023, 64, 4096, (128, 16)), (False, 1024, 64, 4096, (128, 64)),
    (False, 2048, 64, 4096, (256, 128)), (False, 1, 1, 16, (32, 16)), (False, 1024, 1, 1024, (64, 32)),
    (True, 8, 64, 2048, (256, 16)), (True, 384, 64, 2048, (256, 32)), (True, 1024, 64, 2048, (256, 64)),
    (True, 2048, 64, 2048, (256, 128)), (True, 2000, 1, 2048, (256, 64)), (True, 1000, 1, 2048, (256, 32))])
def test_tiles_at_the_rule_s_borders(tile, swiglu, M, G, N, want):
    assert tile(swiglu, M, G, N)[:2] == want
