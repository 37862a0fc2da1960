"""GPU tests of expert products so wide, with so many groups, that their tiles are more than one
dimension of a launch holds (2^32 lanes): each is exact or within a rounding, so that a tile left out
or taken twice shows (tolerances of test_gpu_expert_product)."""
import numpy as np
import pytest
import torch

from _gpu_helpers import DEV
from expert_slot_cache_amd import binding
from test_gpu_expert_product import sum_err
from test_gpu_operators import HALF, dev

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def random(*shape, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return torch.randn(*shape, generator=gen, device=DEV).to(BF16)


def test_many_wide_matrices():
    """4096 groups of one row, 262144 columns: 4224 x 4096 tiles forward, 2^23 workgroups of 512 back."""
    G, N, K = 4096, 1 << 18, 8
    base = random(N, K, seed=1)
    power = 2.0 ** (torch.arange(G, device=DEV) % 5 - 2)                 # of a group's matrix: exact in bf16
    w = torch.empty(G, N, K, dtype=BF16, device=DEV)
    for g in range(G):
        torch.mul(base, power[g].to(BF16), out=w[g])
    x, off = random(G, K, seed=2), dev(np.arange(G + 1, dtype=np.int32))
    out = torch.full((G, N), 7.0, dtype=BF16, device=DEV)
    binding.expert_product(x, w, out, offsets=off)
    b = base.double()
    for r in range(0, G, 256):
        rows = x[r:r + 256].double() * power[r:r + 256, None]
        want = rows @ b.t().contiguous()
        size = rows.abs() @ b.abs().t().contiguous() * sum_err(K)
        assert ((out[r:r + 256].double() - want).abs() <= size + (want.abs() + size) * HALF["bf16"]).all(), r
    # back, with the output as its gradient: a group's one row times its one row
    d_w = w.fill_(7.0)
    binding.expert_product_backward(out, x, None, d_w=d_w, offsets=off)
    for g in range(G):
        want = out[g].float()[:, None] * x[g].float()[None]              # 8 bits by 8: exact in fp32
        assert torch.equal(d_w[g], want.to(BF16)), g
