"""GPU tests of the grouped router and its gradient against oracle/experts.py in float64.  Ids are
held to the oracle's one by one, those included whose choices differ by less than fp32 holds.

Tolerances: u = 2^-24 is half a step of fp32.  A score's exponential is off by (|l| + 1) 2 u of
itself, its sum and quotient by E u + 3 u; products and sums after that by a few u."""
import numpy as np
import pytest
import torch

from _gpu_helpers import DEV
from expert_slot_cache_amd import binding
from oracle import experts as oe
from test_gpu_operators import HALF, INF, TYPES, U, dev, host, logits_for, within

pytestmark = pytest.mark.gpu


def run(lg, bias, K, **kw):
    T = lg.shape[0]
    ids = torch.full((T, K), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T, K), 9.0, device=DEV)
    binding.route_groups(lg, ids, w, bias=bias, **kw)
    return ids, w


def span_of(z):
    """The largest finite |l| that is no stand-in for -inf, twice: a difference of two."""
    fin = np.where(np.isfinite(z), z, 0)
    return np.where(np.abs(fin) < 1e30, np.abs(fin), 0).max() * 2


def check(lg, bias, K, *, score, renorm, n_groups, kept, group_top, scale=1.0, what=""):
    ids, w = run(lg, None if bias is None else dev(bias), K, score=score, renorm=renorm, n_groups=n_groups, kept_groups=kept,
                 group_top=group_top, scale=scale)
    z = host(lg)
    ref_ids, ref_w = oe.route_groups(z, bias, K, score=score, renorm=renorm, n_groups=n_groups, kept=kept, group_top=group_top,
                                     scale=scale)
    assert np.array_equal(ids.cpu().numpy(), ref_ids), what
    # a score below 2^-126 (|l| > 87) has no normal number: 2^-126 absolute, of the scale
    within(host(w), ref_w, np.abs(ref_w) * (2 * span_of(z) + lg.shape[1] + K + 16) * U + scale * 2.0 ** -125, what)


# T, E, K, groups, kept, group_top
CASES = [(1, 8, 2, 4, 2, 2), (4, 64, 8, 8, 4, 2), (9, 60, 6, 5, 2, 2), (33, 256, 8, 8, 4, 2), (17, 512, 10, 8, 4, 1),
         (9, 512, 12, 64, 7, 2), (8, 505, 7, 5, 1, 2), (11, 48, 12, 6, 6, 2), (16, 160, 6, 8, 3, 2), (9, 7, 7, 7, 7, 1),
         (9, 40, 5, 20, 5, 2), (8, 1024, 9, 32, 11, 2), (8, 1000, 64, 10, 4, 2), (8, 4096, 64, 64, 8, 2), (8, 4095, 3, 1, 1, 1),
         (130, 128, 8, 1, 1, 1), (21, 6, 1, 6, 1, 2), (300, 32, 4, 4, 2, 2)]


@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,K,groups,kept,top", CASES)
def test_route_groups(T, E, K, groups, kept, top, kind, score, renorm):
    pad = E + 3 if T % 2 else E                        # rows apart, on no 16 bytes
    lg = torch.full((T, pad), 9.0, dtype=TYPES[kind], device=DEV)[:, :E]
    lg.copy_(dev(logits_for(T, E, E + K), kind))
    rng = np.random.default_rng(E)
    bias = (0.1 * rng.normal(size=E)).astype(np.float32)
    kw = dict(score=score, renorm=renorm, n_groups=groups, kept=kept, group_top=top, scale=2.5)
    check(lg, bias, K, what="bias", **kw)
    check(lg, None, K, what="no bias", **kw)
    bias[rng.integers(0, E, 3)] = [-INF, np.nan, INF]
    check(lg, bias, K, what="bias with infinities", **kw)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K,groups,kept", [(61, 8, 6, 4, 3), (200, 64, 20, 8, 5), (97, 132, 12, 4, 2), (150, 512, 10, 16, 3),
                                              (33, 1024, 30, 8, 2)])
def test_many_equal_choices(T, E, K, groups, kept, score, kind):
    """Logits and biases of a few values: the lower group and the lower id at every tie."""
    rng = np.random.default_rng(T)
    few = np.array([-INF, -2.0, -0.0, 0.0, 1.0, 1.0, 3.0, np.nan], np.float32)
    z = few[rng.integers(0, len(few), (T, E))]
    z[::3] = few[rng.integers(2, 5, (len(z[::3]), E))]
    lg = dev(z, kind)
    for bias in (None, np.zeros(E, np.float32), np.float32([0.0, 0.25])[rng.integers(0, 2, E)]):
        for top in (1, 2):
            check(lg, bias, K, score=score, renorm=True, n_groups=groups, kept=kept, group_top=top, what=(bias is None, top))


@pytest.mark.parametrize("T,E,K,groups,kept", [(40, 64, 8, 8, 4), (40, 160, 10, 10, 3), (20, 512, 12, 1, 1), (12, 2000, 40, 20, 7)])
def test_choices_nearer_than_fp32_holds(T, E, K, groups, kept):
    """Sigmoids of 9 to 20 are all but 1: in fp32 many are equal, in fp64 none.  And softmax scores
    that differ in their last digits."""
    rng = np.random.default_rng(E)
    z = rng.uniform(9, 20, (T, E)).astype(np.float32)
    near = (1 + np.arange(E) * 2.0 ** -22).astype(np.float32)[rng.permutation(E)][None, :].repeat(T, 0)
    bias = np.full(E, 0.5, np.float32)
    a_little = (bias + 2.0 ** -22 * rng.integers(-2, 3, E)).astype(np.float32)
    for top in (1, 2):
        kw = dict(renorm=False, n_groups=groups, kept=kept, group_top=top)
        check(dev(z), bias, K, score="sigmoid", **kw)
        check(dev(z), a_little, K, score="sigmoid", **kw)
        check(dev(z), None, K, score="sigmoid", **kw)
        check(dev(near), bias, K, score="softmax", **kw)
        check(dev(near), a_little, K, score="sigmoid", **kw)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,K,groups,kept", [(64, 64, 8, 8, 4), (64, 64, 8, 1, 1), (24, 512, 9, 8, 3), (9, 1024, 64, 1, 1),
                                              (9, 1024, 63, 4, 3), (33, 20, 19, 1, 1), (33, 20, 20, 1, 1)])
def test_pairs_of_near_choices(T, E, K, groups, kept, score):
    """Experts in pairs whose choices differ by the rounding of their fp32 biases, pairs well apart: the
    order inside a pair, at the border of the chosen ones too, is that of fp64."""
    rng = np.random.default_rng(E + K)
    z = np.empty((T, E), np.float32)
    bias = np.empty(E, np.float32)
    one = rng.normal(size=E).astype(np.float32)        # the same logits for every token, in another order of pairs
    s = oe.scores(one.astype(np.float64), score)
    target = np.repeat(rng.permutation(E // 2 + E % 2) * 0.02, 2)[:E]
    bias[:] = (target - s).astype(np.float32)
    z[:] = one
    turned = rng.random(T) < 0.5                       # softmax: a shift of all logits changes no score
    z[turned] += np.float32(1.0) if score == "softmax" else np.float32(0.0)
    for top in (1, 2):
        check(dev(z), bias, K, score=score, renorm=True, n_groups=groups, kept=kept, group_top=top)


def test_group_sums_that_run_over_fp32():
    """Biases near fp32's largest value: two of them have no sum in fp32, and differ in fp64."""
    rng = np.random.default_rng(4)
    bias = np.full(32, 2.0e38, np.float32)
    bias += (rng.integers(0, 1000, 32) * 2.0 ** 110).astype(np.float32)
    assert np.isfinite(bias).all() and np.isinf(bias[0] + bias[1])
    check(dev(rng.normal(size=(9, 32)).astype(np.float32)), bias, 3, score="sigmoid", renorm=False, n_groups=8, kept=3, group_top=2)


@pytest.mark.parametrize("renorm", [False, True])
def test_scores_far_below_fp32(renorm):
    """Sigmoids of -60 to -200: renormalised weights keep their ratios."""
    rng = np.random.default_rng(3)
    z = rng.uniform(-200, -60, (20, 32)).astype(np.float32)
    check(dev(z), None, 6, score="sigmoid", renorm=renorm, n_groups=4, kept=2, group_top=1)


@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 64, 8), (9, 7, 7), (130, 60, 6), (65, 128, 8), (33, 200, 10), (9, 512, 10),
                                   (8, 1000, 33), (11, 2048, 64), (8, 4095, 3), (300, 33, 4)])
def test_route_groups_backward(T, E, K, kind, score, renorm):
    z = logits_for(T, E, 3 * E + K)
    pad = E + 5 if T % 2 else E
    lg = torch.full((T, pad), 9.0, dtype=TYPES[kind], device=DEV)[:, :E]
    lg.copy_(dev(z, kind))
    z = host(lg)
    rng = np.random.default_rng(E)
    kw = dict(score=score, renorm=renorm, scale=2.5)
    ids, w = oe.route_groups(z, None, K, **kw)
    if T > 8 and K >= 2:
        ids[8, 1] = ids[8, 0]                          # the same expert twice
        ids[0, K - 1] = E                              # and one that is none
        ids[7, 0] = -1
    w, dw = w.astype(np.float32), rng.normal(size=(T, K)).astype(np.float32)
    buf = torch.full((T, pad), 5.0, dtype=TYPES[kind], device=DEV)
    out = buf[:, :E]
    needed = score == "sigmoid" or not renorm
    binding.route_groups_backward(lg if needed else None, dev(ids), dev(w), dev(dw), out, **kw)
    assert (buf[:, E:] == 5.0).all()
    ref = oe.route_groups_grad(z, ids, w, dw, **kw)
    keep = (ids >= 0) & (ids < E)
    total = (np.abs(w * dw) * keep).sum(1)             # S and what it is subtracted from
    size = np.zeros_like(ref)
    for t in range(T):
        if score == "softmax" and not renorm:
            s = oe.scores(np.where(np.isnan(z[t]), -INF, z[t]), score)
            size[t] = s * (2.5 * np.abs(dw[t]).sum() + total[t])
        else:
            np.add.at(size[t], ids[t][keep[t]], (np.abs(w[t]) * (np.abs(dw[t]) + total[t]))[keep[t]])
    within(host(out), ref, size * (2 * span_of(z) + E + 2 * K + 16) * U + np.abs(ref) * HALF[kind] + 2.0 ** -125, "d_logits")


def test_no_groups_no_bias_softmax_is_the_plain_router():
    lg = dev(logits_for(64, 96, 5))
    ids, w = run(lg, None, 6)
    ids0, w0 = torch.empty_like(ids), torch.empty_like(w)
    binding.route(lg, ids0, w0)
    assert torch.equal(ids, ids0)
    within(host(w), host(w0), host(w0) * 16 * U)


def test_captured_and_on_another_stream():
    """A graph of the router and its gradient, replayed on changing logits, with eager calls of the
    same on another stream in between: every replay gives the eager result's bits."""
    T, E, K = 70, 128, 8
    kw = dict(score="sigmoid", renorm=True, scale=2.5)
    bias = dev((0.1 * np.random.default_rng(1).normal(size=E)).astype(np.float32))
    lg, dw = torch.zeros(T, E, device=DEV), torch.randn(T, K, device=DEV)
    ids, w, dl = torch.zeros(T, K, dtype=torch.int32, device=DEV), torch.zeros(T, K, device=DEV), torch.zeros(T, E, device=DEV)

    def both(lg, ids, w, dl):
        binding.route_groups(lg, ids, w, bias=bias, n_groups=8, kept_groups=4, group_top=2, **kw)
        binding.route_groups_backward(lg, ids, w, dw, dl, **kw)

    both(lg, ids, w, dl)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(lg, ids, w, dl)
    side = torch.cuda.Stream()
    for i in range(5):
        # from the second replay on every other token's choices are near each other
        z = logits_for(T, E, 50 + i)
        if i:
            z[::2] = np.random.default_rng(i).uniform(9, 20, (T // 2, E))
        lg.copy_(dev(z))
        torch.cuda.synchronize()
        graph.replay()
        mine = [torch.empty_like(v) for v in (ids, w, dl)]
        with torch.cuda.stream(side):
            both(lg, *mine)
        torch.cuda.synchronize()
        for a, b in zip((ids, w, dl), mine):
            assert torch.equal(a.view(torch.int32), b.view(torch.int32)), i
