"""GPU tests that the expert products and their gradients write inside their outputs alone, whatever
the offsets hold."""
import numpy as np
import pytest
import torch

import test_gpu_operators as ops
from expert_slot_cache_amd import binding
from test_gpu_expert_product import Guarded, rows_for
from test_gpu_product_guards import offsets_of

pytestmark = pytest.mark.gpu

CASES = [(40, 4, 64, 128), (90, 200, 96, 272), (700, 30, 272, 144), (1500, 3, 528, 256), (3000, 20, 512, 144)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("M,G,N,K", CASES)
def test_memory_around_the_outputs_stays(M, G, N, K, kind):
    x, w, dp = rows_for((M, K), 1, kind), rows_for((G, N, K), 2, kind), rows_for((M, N), 3, kind)
    for name, offsets in offsets_of(M, G, M + G).items():
        off = ops.dev(offsets)
        outs = []
        for act in ("none", "swiglu"):
            cols = N // 2 if act == "swiglu" else N
            o, p = Guarded((M, cols), kind), Guarded((M, N), kind)
            binding.expert_product(x, w, o.t, pre=p.t, act=act, offsets=off)
            d, b = Guarded((M, N), kind), Guarded((G, N), "f32")
            binding.activation_backward(rows_for((M, cols), 4, kind), dp, d.t, d_bias=b.t, act=act, offsets=off)
            outs += [o, p, d, b]
        dx, dw = Guarded((M, K), kind), Guarded((G, N, K), "f32")
        binding.expert_product_backward(dp, x, w, d_x=dx.t, d_w=dw.t, offsets=off)
        for o in outs + [dx, dw]:
            o.check(name)


def test_every_row_of_groups_that_cover_all_is_written():
    M, G, N, K = 1000, 9, 96, 64
    off = np.sort(np.random.default_rng(1).integers(0, M + 1, G + 1)).astype(np.int32)
    off[0], off[-1] = 0, M
    for kind in ("f32", "bf16"):
        out = torch.full((M, N), float("nan"), dtype=ops.TYPES[kind], device="cuda")
        binding.expert_product(rows_for((M, K), 1, kind), rows_for((G, N, K), 2, kind), out, offsets=ops.dev(off))
        assert not bool(torch.isnan(out).any())
