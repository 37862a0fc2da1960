"""GPU tests of the bias' gradient over many rows of a group.

Tolerance: u = 2^-24 is half a step of fp32.  A tile's sums are fp32, over at most 64 rows in
chains of 8 and 8 additions; the tiles' sums are added in 64 bits and rounded once.  So a sum is off
by at most (8 + 8 + 1 + 1) u of the sum of the magnitudes, however many rows there are."""
import numpy as np
import pytest
import torch

from _gpu_helpers import DEV
from expert_slot_cache_amd import binding
from test_gpu_operators import TYPES, U, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [16, 40])
def test_large_tiles_first(N):
    """Eight tiles of 2^24 and then tiles of 1: a chain in fp32 loses every one of them."""
    tiles = 1 << 14
    d = torch.zeros(tiles * 64, N, device=DEV)
    d[::64] = 1.0
    d[:8 * 64:64] = 2.0 ** 24
    db = torch.empty(1, N, device=DEV)
    binding.activation_backward(d, None, None, d_bias=db)
    total = d.double().sum(0)
    assert ((db[0].double() - total).abs() <= 18 * U * total).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["none", "relu"])
def test_many_rows(kind, act):
    M, N = 1_500_001, 48
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)
    d = torch.rand(M, N, generator=gen, device=DEV).to(TYPES[kind])
    off = [5, 6, 900_000, 900_000, M - 3]
    db = torch.empty(4, N, device=DEV)
    binding.activation_backward(d, torch.ones_like(d) if act == "relu" else None, None, d_bias=db, act=act,
                                offsets=dev(np.int32(off)))
    for g in range(4):
        total = d[off[g]:off[g + 1]].double().sum(0)
        assert ((db[g].double() - total).abs() <= 18 * U * total).all(), g
