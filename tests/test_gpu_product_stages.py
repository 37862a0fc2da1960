"""GPU tests of the products in the middle of long rows: each tile with more blocks of 128 than its
ring has stages, so that every stage and every place of the scales is used again, with and
without a short last block.  tests/test_product_tiles.py holds the tile of each case."""
import numpy as np
import pytest
import torch

import test_gpu_operators as ops
from _gpu_helpers import DEV
from expert_slot_cache_amd import binding

pytestmark = pytest.mark.gpu

# (tile's matrix rows, rows) -> (rows, groups, columns, depth): depths of a multiple of four blocks, whose
# scales are copied four at a time by the tiles of 64 rows and more, and others
PRODUCTS = {
    (256, 128): [(3500, 20, 1100, 1536), (3500, 20, 1100, 1168)],
    (128, 64): [(700, 30, 700, 1536), (700, 30, 700, 1168)],
    (128, 16): [(200, 30, 1030, 1536), (200, 30, 1030, 1168)],
    (64, 32): [(700, 3, 512, 1536), (700, 3, 512, 1168)],
    (32, 16): [(17, 1, 100, 1536), (40, 3, 257, 2064)],
}
# the same with SwiGLU, the columns being those of its output
GATED = {
    (256, 128): [(3500, 20, 640, 1536), (3500, 20, 640, 1168)],
    (256, 64): [(700, 30, 640, 1536), (700, 30, 640, 1168)],
    (256, 32): [(300, 30, 768, 1536), (300, 30, 768, 1168)],
    (256, 16): [(8, 64, 256, 1536), (180, 2, 256, 1168)],
}


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("case", [c for cases in PRODUCTS.values() for c in cases], ids=str)
def test_product_of_long_rows(case, kind):
    ops.test_scaled_product(*case, kind)


@pytest.mark.parametrize("case", [c for cases in GATED.values() for c in cases], ids=str)
def test_swiglu_of_long_rows(case):
    ops.test_scaled_product_swiglu(*case)


def off16(t):
    """t's values at an address that is not a multiple of 16."""
    out = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:].view(t.shape)
    out.copy_(t)
    assert out.data_ptr() % 16 == 4 and out.is_contiguous()
    return out


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("M,G,N,K", [(3500, 20, 1280, 1536), (700, 30, 1280, 1536)])
def test_scales_on_no_16_bytes_give_the_same_bits(M, G, N, K, swiglu):
    p = ops.Product(M, G, N, K, M, ops.offsets_for(M, G, M))
    results = []
    for moved in (False, True):
        xs, ws = (off16(p.xs), off16(p.ws)) if moved else (p.xs, p.ws)
        out = torch.zeros((M, N // 2 if swiglu else N), device=DEV).to(ops.F8 if swiglu else torch.float32)
        scales = torch.zeros((M, N // 256), device=DEV) if swiglu else None
        binding.scaled_product(p.x, xs, p.w, ws, out, offsets=ops.dev(p.offsets), swiglu_scales=scales)
        results.append((out.view(torch.uint8), scales))
    (a, sa), (b, sb) = results
    assert torch.equal(a, b) and (not swiglu or torch.equal(sa, sb))
    assert np.isfinite(ops.host(p.xs)).all() and bool(a.any())
