"""GPU tests of the expert products and their gradients where offsets into the arrays pass 32 bits: rows
far down and the last of many matrices, against float64 (tolerances of test_gpu_expert_product)."""
import numpy as np
import pytest
import torch

from _gpu_helpers import DEV
from expert_slot_cache_amd import binding
from oracle import experts as oe
from test_gpu_expert_product import sum_err
from test_gpu_operators import HALF, U, dev, host, within

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def fresh(*shape, seed=0):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return torch.randn(*shape, generator=gen, device=DEV, dtype=BF16)


def test_rows_far_down():
    M, N, K, last = 1_100_000, 2048, 64, 700           # 2.25 * 2^30 values of a row array
    assert M * N > 1 << 31
    x, w = fresh(M, K, seed=1), fresh(1, N, K, seed=2)
    out = torch.empty(M, N, dtype=BF16, device=DEV)
    binding.expert_product(x, w, out)
    xs, ws = host(x[-last:]), host(w)
    ref, _ = oe.product(xs, ws, None)
    bound = (np.abs(xs) @ np.abs(ws[0]).T) * sum_err(K)
    within(host(out[-last:]), ref, bound + (np.abs(ref) + bound) * HALF["bf16"], "out")
    # back: the output as its own gradient
    dp = torch.empty_like(out)
    db = torch.empty(1, N, device=DEV)
    binding.activation_backward(out, out, dp, d_bias=db, act="relu")
    assert torch.equal(dp[-last:], torch.where(out[-last:] > 0, out[-last:], 0))
    total = sum(torch.where(out[i:i + 100_000] > 0, out[i:i + 100_000], 0).double().sum(0) for i in range(0, M, 100_000))
    # a thread adds 8 rows, 8 threads a column, 8 slices of the M / 64 tiles: fewer than M / 512 + 80 additions in a chain
    assert ((db[0].double() - total).abs() <= total * (M / 64 / 8 + 80) * U).all()
    dx = torch.empty_like(x)
    binding.expert_product_backward(dp, None, w, d_x=dx)
    d = host(dp[-last:])
    ref = d @ ws[0]
    bound = (np.abs(d) @ np.abs(ws[0])) * sum_err(N)
    within(host(dx[-last:]), ref, bound + (np.abs(ref) + bound) * HALF["bf16"], "d_x")
    dw = torch.empty(1, N, K, device=DEV)
    binding.expert_product_backward(dp, x, None, d_w=dw)
    want, size = torch.zeros(N, K, dtype=torch.float64, device=DEV), torch.zeros(N, K, dtype=torch.float64, device=DEV)
    for i in range(0, M, 100_000):
        a, b = dp[i:i + 100_000].double().t().contiguous(), x[i:i + 100_000].double()
        want += a @ b
        size += a.abs() @ b.abs()
    assert ((dw[0].double() - want).abs() <= size * sum_err(M)).all()


def test_the_last_of_many_matrices():
    G, N, K, M = 136, 4096, 4096, 40
    assert G * N * K > 1 << 31
    w = torch.zeros(G, N, K, dtype=BF16, device=DEV)
    w[-1] = fresh(N, K, seed=3)
    x, dp = fresh(M, K, seed=4), fresh(M, N, seed=5)
    off = dev(np.int32([0] * G + [M]))
    out, dx = torch.empty(M, N, dtype=BF16, device=DEV), torch.empty(M, K, dtype=BF16, device=DEV)
    binding.expert_product(x, w, out, offsets=off)
    binding.expert_product_backward(dp, None, w, d_x=dx, offsets=off)
    xs, ds, ws = host(x), host(dp), host(w[-1])
    for got, ref, size, n in ((out, xs @ ws.T, np.abs(xs) @ np.abs(ws).T, K), (dx, ds @ ws, np.abs(ds) @ np.abs(ws), N)):
        bound = size * sum_err(n)
        within(host(got), ref, bound + (np.abs(ref) + bound) * HALF["bf16"])
    w.fill_(7.0)                                       # now the gradient
    binding.expert_product_backward(dp, x, None, d_w=w, offsets=off)
    assert not bool(w[:-1].any())
    ref, bound = ds.T @ xs, (np.abs(ds).T @ np.abs(xs)) * sum_err(M)
    within(host(w[-1]), ref, bound + (np.abs(ref) + bound) * HALF["bf16"], "d_w")
