"""GPU tests of NaN and infinities through the expert products' epilogue and back: what goes in as NaN
leaves as NaN, and an infinity as the activation's formula has it (inf - inf and 0 inf are NaN)."""
import numpy as np
import pytest
import torch

from _gpu_helpers import DEV
from expert_slot_cache_amd import binding
from oracle import experts as oe
from test_gpu_expert_product import act_err, rows_for, slope_err
from test_gpu_operators import HALF, TYPES, U, dev, host

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
VALUES = [NAN, INF, -INF, 0.0, -0.0, 1.0, -3.0, 2.0 ** 99, -(2.0 ** 99), -80.0, 80.0, 0.5]


def same(got, ref, bound, what):
    """NaN for NaN, each infinity itself, and the others within the bound."""
    assert np.array_equal(np.isnan(got), np.isnan(ref)), (what, got, ref)
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), what
    live = ~inf & ~np.isnan(ref)
    assert (np.abs(got[live] - ref[live]) <= bound[live]).all(), what


def grid(act):
    """Every value in every column; for SwiGLU every pair of gate and up."""
    n = len(VALUES)
    if act != "swiglu":
        return np.float32(VALUES + VALUES[:4])[None]                     # 16 columns
    pairs = np.float32([(a, b) for a in VALUES for b in VALUES] + [(1, 1)] * (-n * n % 8))
    return np.concatenate([pairs[:, 0], pairs[:, 1]])[None]


def finite(a):
    return np.where(np.isfinite(a), a, 0.0)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("act", oe.ACTS)
def test_forward(act, kind):
    h = grid(act).astype(np.float64)
    N, M = h.shape[1], 5
    cols = N // 2 if act == "swiglu" else N
    # rows of zeros: h is the bias
    out, pre = torch.empty(M, cols, device=DEV), torch.empty(M, N, dtype=TYPES[kind], device=DEV)
    binding.expert_product(torch.zeros(M, 16, dtype=TYPES[kind], device=DEV), torch.ones(1, N, 16, dtype=TYPES[kind], device=DEV),
                           out, bias=dev(h.astype(np.float32)), pre=pre, act=act)
    with np.errstate(all="ignore"):
        ref = oe.activate(h, act)
        if act == "swiglu":
            g, u = h[:, :cols], h[:, cols:]
            bound = act_err(g, 0, "silu") * np.abs(u) + np.abs(ref) * 3 * U
            # a product past fp32's largest value is an infinity
            ref = np.where(np.abs(ref) > np.finfo(np.float32).max, np.sign(ref) * INF, ref)
        else:
            bound = act_err(h, 0, act) + np.abs(ref) * 3 * U
    for r in range(M):
        same(host(out)[r:r + 1], ref, finite(bound), (act, r))
        same(host(pre)[r:r + 1], h, np.abs(finite(h)) * HALF[kind], "pre")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("act", oe.ACTS)
def test_backward(act, kind):
    h = host(dev(grid(act), kind))
    M, N = 4, h.shape[1]
    cols = N // 2 if act == "swiglu" else N
    h = h.repeat(M, 0)
    d = np.float64([1.5, 0.0, NAN, -INF])[:, None].repeat(cols, 1)
    d_pre, d_bias = torch.empty(M, N, dtype=TYPES[kind], device=DEV), torch.empty(1, N, device=DEV)
    args = (dev(d.astype(np.float32)), dev(h.astype(np.float32), kind))
    binding.activation_backward(*args, d_pre, d_bias=d_bias, act=act)
    with np.errstate(all="ignore"):
        ref, _ = oe.activation_grad(d, h, None, N, act)
        if act == "swiglu":
            g, u = h[:, :cols], h[:, cols:]
            e = np.concatenate([np.abs(d * u) * (slope_err(g, "silu") + np.abs(oe.slope(g, "silu")) * 3 * U),
                                np.abs(d) * (act_err(g, 0, "silu") + np.abs(oe.activate(g, "silu")) * 3 * U)], axis=1)
        else:
            e = np.abs(d) * (slope_err(h, act) + np.abs(oe.slope(h, act)) * 2 * U)
        e = e + np.abs(ref) * HALF[kind]
    same(host(d_pre), ref, finite(e), act)
    assert bool(torch.isnan(d_bias).all())             # of the row whose gradient is NaN


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("act", oe.ACTS)
@pytest.mark.parametrize("M,G,N,K", [(7, 2, 48, 40), (200, 3, 272, 136), (1601, 8, 2576, 360)])
def test_a_row_of_nan_stays_in_its_row(act, kind, M, G, N, K):
    """A NaN in a row of x makes that row NaN, one in a matrix its column of its group's rows, and
    they leave every other output's bits as they are: the products and all gradients."""
    x, w, b = rows_for((M, K), 1, kind), rows_for((G, N, K), 2, kind, 0.1), rows_for((G, N), 3, "f32")
    off = np.linspace(0, M, G + 1).astype(np.int32)
    cols = N // 2 if act == "swiglu" else N
    run = lambda x, w, b: [t := torch.empty(M, cols, dtype=TYPES[kind], device=DEV),             # noqa: E731
                           binding.expert_product(x, w, t, bias=b, act=act, offsets=dev(off))][0]
    good = run(x, w, b)
    row, group, col = int(off[1]), 1, N - 3            # the second group's first row
    bad = x.clone()
    bad[row, K - 1] = NAN
    got = run(bad, w, b)
    assert bool(torch.isnan(got[row]).all())
    keep = torch.arange(M, device=DEV) != row
    assert torch.equal(got[keep], good[keep])
    at = col - cols if act == "swiglu" else col
    for which in ("matrix", "bias"):
        bad_w, bad_b = w.clone(), b.clone()
        if which == "matrix":
            bad_w[group, col, 0] = NAN
        else:
            bad_b[group, col] = NAN
        got = run(x, bad_w, bad_b)
        mine = slice(int(off[group]), int(off[group + 1]))
        assert bool(torch.isnan(got[mine, at]).all()), which
        got[mine, at] = good[mine, at]
        assert torch.equal(got, good), which
    # back: a NaN in d_pre reaches its row of d_x and its row of its group's d_w alone
    dp = rows_for((M, N), 4, kind)
    def back(dp):
        dx, dw = torch.empty_like(x), torch.empty(G, N, K, device=DEV)
        binding.expert_product_backward(dp, x, w, d_x=dx, d_w=dw, offsets=dev(off))
        return dx, dw
    dx, dw = back(dp)
    bad = dp.clone()
    bad[row, col] = NAN
    dx2, dw2 = back(bad)
    assert bool(torch.isnan(dx2[row]).all()) and torch.equal(dx2[keep], dx[keep])
    assert bool(torch.isnan(dw2[group, col]).all())
    dw2[group, col] = dw[group, col]
    assert torch.equal(dw2, dw)
