"""GPU test of a mixture-of-experts layer through its operators as a training step runs them: grouped
router, sort, both expert products, combine, and back through every gradient, against the same layer
in float64 by torch's autograd on the CPU (at the experts that were chosen).

Tolerance: every stage adds at most 2 (n + 4) u of the sum of magnitudes of its n terms (u = 2^-24),
and passes on what reaches it by at most the magnitudes themselves (slopes of silu below 1.13, of a
share of the scores below 1).  So each result is off by less than the sum of the stages' factors, times
the same chain on magnitudes, which is the layer with every tensor replaced by its absolute value and
silu by 1.13 |h|: computed beside it."""
import numpy as np
import pytest
import torch

from _gpu_helpers import DEV
from expert_slot_cache_amd import binding
from oracle import experts as oe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def reference(t, ids, d_out, K, scale, magnitudes):
    """(out, gradients by name) in float64; with magnitudes an upper bound of each one's terms."""
    v = {k: a.double().cpu() for k, a in t.items()}
    d = d_out.double().cpu()
    if magnitudes:
        v = {k: a.abs() for k, a in v.items()}
        d = d.abs()
    leaves = {k: a.requires_grad_() for k, a in v.items()}
    silu = (lambda h: 1.13 * h) if magnitudes else torch.nn.functional.silu
    T = v["x"].shape[0]
    ids = ids.long().cpu()
    if magnitudes:                                     # shares of about 1/K each, their slopes below the shares
        z = (v["x"] @ v["router"].T).gather(1, ids)
        share = scale * (1.0 + z)
    else:
        s = torch.sigmoid((v["x"] @ v["router"].T).gather(1, ids))
        share = scale * s / s.sum(1, keepdim=True)
    out = v["x"].clone()
    half = v["w13"].shape[1] // 2
    for k in range(K):
        for i in range(T):
            e = int(ids[i, k])
            h = v["w13"][e] @ v["x"][i] + v["b13"][e]
            y = v["w2"][e] @ (silu(h[:half]) * h[half:]) + v["b2"][e]
            out[i] = out[i] + share[i, k] * y
    (out * d).sum().backward()
    return out.detach(), {k: a.grad for k, a in leaves.items()}


def test_a_layer_and_its_gradients():
    T, E, K, H, I, scale = 23, 8, 2, 64, 48, 1.5
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)
    make = lambda *s: torch.randn(*s, generator=gen, device=DEV)      # noqa: E731
    t = dict(x=make(T, H), router=0.2 * make(E, H), w13=0.1 * make(E, 2 * I, H), b13=0.1 * make(E, 2 * I), w2=0.1 * make(E, H, I),
             b2=0.1 * make(E, H))
    balance, d_out = 0.1 * make(E), make(T, H)
    new = lambda *s: torch.full(s, 7.0, device=DEV)                    # noqa: E731
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device=DEV)     # noqa: E731
    R = T * K

    logits, ids, w = new(T, E), i32(T, K), new(T, K)
    binding.expert_product(t["x"], t["router"][None], logits)
    route = dict(score="sigmoid", renorm=True, scale=scale)
    binding.route_groups(logits, ids, w, bias=balance, n_groups=4, kept_groups=2, group_top=2, **route)
    xs, offsets, rows = new(R, H), i32(E + 1), i32(T, K)
    binding.sort_tokens(t["x"], ids, xs, offsets, rows)
    act, pre, ys, out = new(R, I), new(R, 2 * I), new(R, H), new(T, H)
    binding.expert_product(xs, t["w13"], act, bias=t["b13"], pre=pre, act="swiglu", offsets=offsets)
    binding.expert_product(act, t["w2"], ys, bias=t["b2"], offsets=offsets)
    binding.combine_rows(ys, rows, out, topk_w=w, resid=t["x"])

    d_ys, d_w, d_act, d_pre, d_xs = new(R, H), new(T, K), new(R, I), new(R, 2 * I), new(R, H)
    g = {k: torch.empty_like(v) for k, v in t.items()}
    binding.combine_rows_backward(d_out, ys, rows, w, d_ys, d_w)
    binding.activation_backward(d_ys, None, None, d_bias=g["b2"], offsets=offsets)
    binding.expert_product_backward(d_ys, act, t["w2"], d_x=d_act, d_w=g["w2"], offsets=offsets)
    binding.activation_backward(d_act, pre, d_pre, d_bias=g["b13"], act="swiglu", offsets=offsets)
    binding.expert_product_backward(d_pre, xs, t["w13"], d_x=d_xs, d_w=g["w13"], offsets=offsets)
    d_logits, d_router_x = new(T, E), new(T, H)
    binding.route_groups_backward(logits, ids, w, d_w, d_logits, **route)
    binding.expert_product_backward(d_logits, t["x"], t["router"][None], d_x=d_router_x, d_w=g["router"][None])
    # x is reached through the residual, the experts and the router
    binding.combine_rows(d_xs, rows, g["x"], resid=d_out)
    g["x"] += d_router_x

    z = (t["x"].double() @ t["router"].double().T).cpu().numpy()
    ref_ids, _ = oe.route_groups(z, balance.cpu().numpy(), K, score="sigmoid", renorm=True, n_groups=4, kept=2, group_top=2)
    assert np.array_equal(ids.cpu().numpy(), ref_ids)
    ref, ref_g = reference(t, ids, d_out, K, scale, False)
    mag, mag_g = reference(t, ids, d_out, K, scale, True)
    stages = 2 * (2 * (H + 4) + 2 * (I + 4) + 2 * (2 * I + 4) + 2 * (H + 4) + 2 * (R + 4) + 40) * U
    assert ((out.cpu().double() - ref).abs() <= stages * mag).all()
    for k in g:
        worst = ((g[k].cpu().double() - ref_g[k]).abs() / mag_g[k].clamp(min=1e-30)).max().item()
        assert worst <= stages, (k, worst, stages)
