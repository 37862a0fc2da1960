"""CPU tests of the rules that pick an expert product's tile (csrc/product_tile.hpp): each case of
tests/test_gpu_expert_tiles.py takes the tile it is listed under, products use every stage of the ring
again, and no tile of the rules is left out."""
import os
import re
import shutil
import subprocess

import pytest

import test_gpu_expert_tiles as cases

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "expert_slot_cache_amd", "csrc")


@pytest.fixture(scope="module")
def tile(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path_factory.mktemp("tile") / "expert_tile_driver")
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC,
                    os.path.join(ROOT, "tests", "native", "expert_tile_driver.cpp"), "-o", exe], check=True)

    def ask(rule, bf16, M, G, N, K, offsets):
        r = subprocess.run([exe], input=f"{rule} {int(bf16)} {M} {G} {N} {K} {int(offsets)}\n", capture_output=True, text=True,
                           check=True)
        return tuple(int(v) for v in r.stdout.split())
    return ask


def test_every_tile_has_cases_that_use_its_stages_again(tile):
    seen = set()
    for rules, bf16, table in (("ps", True, cases.BF16), ("ps", False, cases.F32), ("s", False, cases.F32_SWIGLU)):
        for want, shapes in table.items():
            kinds = set()
            for M, G, N, K in shapes:
                for rule in rules:                     # plain, SwiGLU
                    for offsets in {G > 1, True}:      # with holes a single group has offsets too
                        PA, PB, RB, S, _ = tile(rule, bf16, M, G, N, K, offsets)
                        assert (PA, PB) == want, (bf16, M, G, N)
                    seen.add((PA, PB))
                    depth = RB // (2 if bf16 else 4)
                    assert -(-K // depth) > S + 1, (M, G, N, K)
                kinds.add("short" if K % depth else "whole")
            assert kinds == {"short", "whole"}, want
    for want, shapes in cases.MATRICES.items():
        for M, G, N, K in shapes:
            PA, PB, _, _, parts = tile("m", True, M, G, N, K, True)
            assert (PA, PB, parts) == want, (M, G, N, K)
            seen.add((PA, PB))
    text = open(os.path.join(CSRC, "product_tile.hpp")).read()
    assert seen == {(int(a), int(b)) for a, b in re.findall(r"CoreTile<(\d+), (\d+), ", text)}


@pytest.mark.parametrize("bf16,M,G,N,want", [
    (True, 384 * 64, 64, 2048, (256, 256)), (True, 383 * 64, 64, 2048, (256, 128)), (True, 128 * 64, 64, 2048, (256, 128)),
    (True, 127 * 64, 64, 2048, (128, 64)), (True, 48 * 64, 64, 2048, (128, 64)), (True, 47 * 64, 64, 2048, (64, 64)),
    (True, 32 * 64, 64, 2048, (64, 64)), (True, 31 * 64, 64, 2048, (64, 32)), (True, 333, 1, 1000, (64, 32)),
    (False, 333, 1, 1000, (32, 32)), (False, 1024, 64, 1024, (64, 32)),
    (True, 1, 1, 4096, (32, 32)), (True, 1, 1, 8192, (64, 32)), (True, 2048, 1, 4096, (256, 128)),
    (False, 768 * 8, 8, 4096, (64, 64)), (False, 1, 1, 16, (32, 32))])
def test_tiles_at_the_rule_s_borders(tile, bf16, M, G, N, want):
    assert tile("p", bf16, M, G, N, 0, G > 1)[:2] == want


@pytest.mark.parametrize("M,G,N,K,parts", [(16384, 1, 64, 2048, 8), (4095, 1, 64, 2048, 1), (4096, 1, 64, 2048, 2),
                                           (1 << 24, 1, 64, 128, 16), (16384, 1, 1024, 1024, 2)])
def test_parts_of_a_matrix_gradient(tile, M, G, N, K, parts):
    assert tile("m", True, M, G, N, K, False)[4] == parts
