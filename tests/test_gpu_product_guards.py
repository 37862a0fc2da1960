"""GPU tests that a product writes inside its outputs alone, whatever the offsets hold."""
import numpy as np
import pytest
import torch

import test_gpu_operators as ops
from _gpu_helpers import DEV
from expert_slot_cache_amd import binding

pytestmark = pytest.mark.gpu

GUARD = 300        # rows before and behind: more than the largest tile has


def guarded(rows, cols, dtype):
    """(the whole, its middle rows): the rows around the middle hold 0x5a in every byte."""
    size = torch.empty(0, dtype=dtype).element_size()
    whole = torch.full((rows + 2 * GUARD, cols * size), 0x5A, dtype=torch.uint8, device=DEV)
    return whole, whole[GUARD:GUARD + rows].view(dtype)


def untouched(whole, rows):
    return bool((whole[:GUARD] == 0x5A).all()) and bool((whole[GUARD + rows:] == 0x5A).all())


def offsets_of(M, G, seed):
    """Offsets of G groups of M rows that are as they should be, and ones that are not."""
    rng = np.random.default_rng(seed)
    rising = ops.offsets_for(M, G, seed)
    falling = rising[::-1].copy()
    mixed = rng.permutation(rising)
    outside = rng.integers(-(1 << 31), 1 << 31, G + 1).astype(np.int32)
    a_little = (rising + rng.integers(-3, 4, G + 1)).astype(np.int32)
    saw = np.where(np.arange(G + 1) % 2 == 0, 0, M).astype(np.int32)
    high, low = np.full(G + 1, M + 1, np.int32), np.full(G + 1, -1, np.int32)
    return dict(rising=rising, falling=falling, mixed=mixed, outside=outside, a_little=a_little, saw=saw, high=high, low=low)


# (rows, groups, columns, depth): several groups to a lane (more than 64), and every tile
CASES = [(40, 4, 64, 128), (90, 200, 96, 272), (200, 30, 1030, 144), (700, 30, 700, 144), (3500, 20, 1100, 144), (700, 3, 512, 144)]
GATED = [(40, 4, 256, 128), (90, 200, 256, 272), (300, 30, 1536, 144), (700, 30, 1280, 144), (3500, 20, 1280, 144)]


@pytest.mark.parametrize("M,G,N,K,out_type", [(*c, kind) for kind in ("f32", "bf16") for c in CASES] +
                         [(*c, "swiglu") for c in GATED])
def test_rows_around_the_outputs_stay(M, G, N, K, out_type):
    gated = out_type == "swiglu"
    x, w = ops.codes_for((M, K), M).to(DEV), ops.codes_for((G, N, K), N).to(DEV)
    xs = ops.dev(ops.scales_for((M, -(-K // 128)), 1))
    ws = ops.dev(ops.scales_for((G, -(-N // 128), -(-K // 128)), 2))
    for name, offsets in offsets_of(M, G, M + G).items():
        if gated:
            whole, out = guarded(M, N // 2, ops.F8)
            whole_s, scales = guarded(M, N // 256, torch.float32)
        else:
            whole, out = guarded(M, N, ops.TYPES[out_type])
            whole_s, scales = None, None
        binding.scaled_product(x, xs, w, ws, out, offsets=ops.dev(offsets), swiglu_scales=scales)
        assert untouched(whole, M), name
        assert whole_s is None or untouched(whole_s, M), name
        if name == "rising":                           # every row lies in a group here
            assert not bool((out.view(torch.uint8) == 0x5A).all(dim=1).any())
