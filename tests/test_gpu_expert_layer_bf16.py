"""GPU test of a mixture-of-experts layer that trains, written as a user writes it, forward and all the
way back, in fp32 and in bf16: the same calls, against the layer in float64 by torch's autograd on the
CPU (at the experts that were chosen).

Tolerance.  Every input is a positive value, and the bound is a chain of magnitudes beside the
reference: every tensor its absolute value, silu (1.13 + |h| / 2) |h| (its derivative is above that of silu and
the change of that derivative with h, |h| silu''(h) <= |h| / 2), a share of the scores scale (1 + the sum of
the token's chosen logits) (its derivatives are above the share's: both are at most scale).  A stage adds 2 (n + 4) u of
the magnitudes of its n terms; a tensor kept in bf16 adds 2^-8 of them.  The longest way has ROUNDED
such tensors: pre, act, ys, out (forward) and d_ys, d_act, d_pre, d_xs or d_logits, and the result; what reaches a gradient
over two ways (its own and the values kept for it) counts twice."""
import numpy as np
import pytest
import torch

from _gpu_helpers import DEV
from expert_slot_cache_amd import binding as b
from oracle import experts as oe

pytestmark = pytest.mark.gpu

U, ROUNDED = 2.0 ** -24, 9
T, E, K, H, I, SCALE = 29, 8, 2, 64, 48, 1.5
CHOICE = dict(n_groups=4, kept_groups=2, group_top=2)
ROUTE = dict(score="sigmoid", renorm=True, scale=SCALE)


def layer(t, balance, d_out, kind):
    """(out, ids, the gradients by name) by the library's operators."""
    new = lambda *s: torch.full(s, 7.0, dtype=kind, device=DEV)          # noqa: E731
    f32 = lambda *s: torch.full(s, 7.0, device=DEV)                      # noqa: E731
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device=DEV)       # noqa: E731
    x, router, R = t["x"], t["router"], T * K
    logits, ids, w = f32(T, E), i32(T, K), f32(T, K)
    b.expert_product(x, router[None], logits)
    b.route_groups(logits, ids, w, bias=balance, **CHOICE, **ROUTE)
    xs, offsets, rows = new(R, H), i32(E + 1), i32(T, K)
    b.sort_tokens(x, ids, xs, offsets, rows)
    act, pre, ys, out = new(R, I), new(R, 2 * I), new(R, H), new(T, H)
    b.expert_product(xs, t["w13"], act, bias=t["b13"], pre=pre, act="swiglu", offsets=offsets)
    b.expert_product(act, t["w2"], ys, bias=t["b2"], offsets=offsets)
    b.combine_rows(ys, rows, out, topk_w=w, resid=x)

    g = {k: torch.full_like(v, 7.0) for k, v in t.items()}
    d_ys, d_w, d_act, d_pre, d_xs = new(R, H), f32(T, K), new(R, I), new(R, 2 * I), new(R, H)
    b.combine_rows_backward(d_out, ys, rows, w, d_ys, d_w)
    b.activation_backward(d_ys, None, None, d_bias=g["b2"], offsets=offsets)
    b.expert_product_backward(d_ys, act, t["w2"], d_x=d_act, d_w=g["w2"], offsets=offsets)
    b.activation_backward(d_act, pre, d_pre, d_bias=g["b13"], act="swiglu", offsets=offsets)
    b.expert_product_backward(d_pre, xs, t["w13"], d_x=d_xs, d_w=g["w13"], offsets=offsets)
    d_logits, d_rows, d_x = f32(T, E), new(T, E), new(T, H)
    b.route_groups_backward(logits, ids, w, d_w, d_logits, **ROUTE)
    b.activation_backward(d_logits, None, d_rows)                        # to the rows' format
    b.expert_product_backward(d_rows, x, router[None], d_x=d_x, d_w=g["router"][None])
    b.combine_rows(d_xs, rows, g["x"], resid=d_out)
    g["x"] += d_x
    return out, ids, g


def reference(t, ids, d_out, magnitudes):
    v = {k: a.double().cpu().requires_grad_() for k, a in t.items()}
    silu = (lambda h: (1.13 + h / 2) * h) if magnitudes else torch.nn.functional.silu
    ids = ids.long().cpu()
    z = (v["x"] @ v["router"].T).gather(1, ids)
    if magnitudes:
        share = SCALE * (1 + z.sum(1, keepdim=True)).expand(-1, K)
    else:
        s = torch.sigmoid(z)
        share = SCALE * s / s.sum(1, keepdim=True)
    out = v["x"].clone()
    for k in range(K):
        for i in range(T):
            e = int(ids[i, k])
            h = v["w13"][e] @ v["x"][i] + v["b13"][e]
            y = v["w2"][e] @ (silu(h[:I]) * h[I:]) + v["b2"][e]
            out = out + torch.zeros_like(out).index_add(0, torch.tensor([i]), (share[i, k] * y)[None])
    (out * d_out.double().cpu()).sum().backward()
    return out.detach(), {k: a.grad for k, a in v.items()}


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_a_layer_that_trains(kind):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)
    make = lambda *s: torch.rand(*s, generator=gen, device=DEV)          # noqa: E731
    t = dict(x=make(T, H), router=make(E, H) / H, w13=make(E, 2 * I, H) / H, w2=make(E, H, I) / I)
    t = {k: v.to(kind) for k, v in t.items()} | dict(b13=make(E, 2 * I), b2=make(E, H))
    balance, d_out = 0.1 * make(E), make(T, H).to(kind)
    out, ids, g = layer(t, balance, d_out, kind)
    z = (t["x"].double() @ t["router"].double().T).cpu().numpy()
    ref_ids, _ = oe.route_groups(z, balance.cpu().numpy(), K, score="sigmoid", renorm=True, n_groups=4, kept=2, group_top=2)
    assert np.array_equal(ids.cpu().numpy(), ref_ids)
    ref, ref_g = reference(t, ids, d_out, False)
    mag, mag_g = reference(t, ids, d_out, True)
    stages = 2 * (2 * (H + 4) + 2 * (I + 4) + 2 * (2 * I + 4) + 2 * (H + 4) + 2 * (T * K + 4) + 40) * U
    if kind is torch.bfloat16:
        stages += 2 * ROUNDED * 2.0 ** -8
    assert ((out.cpu().double() - ref).abs() <= stages * mag).all()
    for k in g:
        assert g[k].dtype is t[k].dtype
        worst = ((g[k].cpu().double() - ref_g[k]).abs() / mag_g[k].clamp(min=1e-30)).max().item()
        assert worst <= stages, (k, worst, stages)
